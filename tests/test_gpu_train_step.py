"""The operators together, as a training step uses them: a tied embedding and
LM head around a layer of experts, gradients written into flat buffers, the
gradient-norm clip over both, Muon on the expert blocks, AdamW on the table.

    x = s E[ids];  u = x W1_e (rows sorted by expert);  a = max(u, 0)
    h = x + a W2_e;  loss = mean over labelled rows of CE(h E^T)

Bound, relative to the norm of each gradient.  Every product's element is off
by (K + 1) 2^-23 sum|a||b| <= (K + 1) 2^-23 sqrt(K) |a||b| typically, with
K <= 300, over at most 6 products in a row: 6 * 301 * 2^-23 * sqrt(300) =
3.8e-3 in fp32.  bf16 adds a rounding of 2^-8 at each of the at most 8 places
where a value is stored, 3.1e-2, and the inputs of the reference are the same
bf16 values."""

import pytest
import torch

import muon_newton_schulz_amd as M
from muon_newton_schulz_amd import workloads as W
from train_ops_util import DT, same_bits

pytestmark = pytest.mark.gpu

N, V, D, F, E = 200, 300, 64, 96, 5
SCALE = 8.0


class Step:
    """Parameters, flat gradient buffers, workspaces and one step."""

    def __init__(self, gpu, dt, seed):
        g = torch.Generator(device=gpu)
        g.manual_seed(seed)
        t = DT[dt]
        self.dt = dt
        r = lambda *s: torch.randn(*s, generator=g, device=gpu)  # noqa: E731
        # expert blocks [E, D, F] and [E, F, D] in one flat buffer, as Muon takes them
        n1, n2 = E * D * F, E * F * D
        self.params = (r(n1 + n2) * 0.15).to(t)
        self.grads = torch.empty_like(self.params)
        self.w1, self.w2 = self.params[:n1].view(E, D, F), self.params[n1:].view(E, F, D)
        self.dw1, self.dw2 = self.grads[:n1].view(E, D, F), self.grads[n1:].view(E, F, D)
        mats = [(e * D * F, D, F) for e in range(E)] + [(n1 + e * F * D, F, D) for e in range(E)]
        self.plan = M.muon_plan_create(mats, n1 + n2, dt, dt, dt)
        self.mom = torch.zeros(n1 + n2, device=gpu)
        self.mws = self.plan.alloc_workspace(gpu)
        # the table: AdamW, fp32 master where the parameters are bf16
        self.table = (r(V, D) * 0.1).to(t)
        self.master = self.table.float() if dt == "bf16" else None
        self.dtable = torch.empty_like(self.table)
        self.m, self.v = torch.zeros(V * D, device=gpu), torch.zeros(V * D, device=gpu)
        self.clip = torch.zeros(16, dtype=torch.uint8, device=gpu)
        self.clip_ws = torch.empty(M.grad_norm_clip_workspace_size(2), dtype=torch.uint8,
                                   device=gpu)
        # a batch: ids with padding, labels with ignored rows, rows by expert
        self.ids = torch.randint(-20, V, (N,), generator=g, device=gpu)
        self.targets = torch.randint(-60, V, (N,), generator=g, device=gpu)
        self.offsets = torch.tensor([0, 40, 40, 111, 150, N], dtype=torch.int32, device=gpu)
        self.dloss = torch.full((N,), 1.0 / int((self.targets >= 0).sum()), device=gpu)
        e = lambda *s: torch.empty(*s, dtype=t, device=gpu)  # noqa: E731
        self.x, self.u, self.y, self.h = e(N, D), e(N, F), e(N, D), e(N, D)
        self.dh, self.da, self.dx = e(N, D), e(N, F), e(N, D)
        self.loss, self.lse = torch.empty(N, device=gpu), torch.empty(N, device=gpu)
        need = max(M.lm_loss_workspace_size(N, V, D, dt), M.embed_backward_workspace_size(N, V, D))
        self.ws = torch.empty(need, dtype=torch.uint8, device=gpu)
        self.hp, self.ahp = W.MuonHParams(), W.AdamWHParams()

    def gradients(self):
        M.embed_forward(self.table, self.ids, SCALE, out=self.x)
        M.expert_matmul(self.x, self.w1, self.offsets, out=self.u)
        a = self.u.clamp(min=0)
        M.expert_matmul(a, self.w2, self.offsets, out=self.y)
        torch.add(self.x, self.y, out=self.h)
        M.lm_loss_forward(self.h, self.table, self.targets, loss=self.loss, lse=self.lse,
                          workspace=self.ws)
        # the head's part of the table gradient first, the embedding's on top
        M.lm_loss_backward(self.h, self.table, self.targets, self.lse, self.dloss,
                           dhidden=self.dh, dweight=self.dtable, workspace=self.ws)
        M.expert_wgrad(a, self.dh, self.offsets, self.dw2)
        M.expert_matmul(self.dh, self.w2, self.offsets, trans=True, out=self.da)
        self.da.mul_(self.u > 0)
        M.expert_wgrad(self.x, self.da, self.offsets, self.dw1)
        M.expert_matmul(self.da, self.w1, self.offsets, trans=True, out=self.dx)
        self.dx.add_(self.dh)
        M.embed_backward(self.dx, self.ids, self.dtable, SCALE, accumulate=True, workspace=self.ws)

    def step(self):
        self.gradients()
        flat = self.dtable.view(-1)
        M.grad_norm_clip([self.grads, flat], 1.0, out=self.clip, workspace=self.clip_ws)
        M.muon_step(self.plan, self.params, self.grads, self.mom, self.mws, self.hp,
                    clip=self.clip)
        master = None if self.master is None else self.master.view(-1)
        M.adamw_step(self.table.view(-1), master, flat, self.m, self.v, self.ahp, 1,
                     clip=self.clip)

    def tensors(self):
        out = [self.params, self.grads, self.mom, self.table, self.dtable, self.m, self.v,
               self.loss, self.lse, self.clip.view(torch.float32)]
        return out + ([self.master] if self.master is not None else [])


def _reference(s):
    """Gradients by autograd in fp64 from the step's parameters."""
    table = s.table.double().requires_grad_()
    w1, w2 = s.w1.double().requires_grad_(), s.w2.double().requires_grad_()
    ok = s.ids >= 0
    x = torch.where(ok[:, None], table[s.ids.clamp(min=0)] * SCALE, torch.zeros((), device=table.device,
                                                                               dtype=torch.float64))
    b = s.offsets.tolist()
    y = torch.cat([(x[b[e]:b[e + 1]] @ w1[e]).clamp(min=0) @ w2[e] for e in range(E)])
    logits = (x + y) @ table.t()
    loss = torch.logsumexp(logits, 1) - logits.gather(1, s.targets.clamp(min=0)[:, None])[:, 0]
    loss = torch.where(s.targets >= 0, loss, torch.zeros_like(loss))
    (loss * s.dloss.double()).sum().backward()
    return loss.detach(), table.grad, w1.grad, w2.grad


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_step_against_fp64_autograd(gpu, dt):
    s = Step(gpu, dt, 3)
    loss, dt_ref, d1, d2 = _reference(s)
    before = s.table.clone(), s.params.clone()
    s.step()
    torch.cuda.synchronize()
    tol = 3.8e-3 + (3.1e-2 if dt == "bf16" else 0.0)
    for got, want in ((s.dtable, dt_ref), (s.dw1, d1), (s.dw2, d2)):
        assert float((got.double() - want).norm()) <= tol * float(want.norm())
    assert float((s.loss.double() - loss).norm()) <= tol * float(loss.norm())
    # an expert without rows got zeros, and the step saw these gradients
    assert not bool(s.dw1[1].any()) and not bool(s.dw2[1].any())
    c = M.read_clip_state(s.clip)
    norm = float((s.dtable.double().norm() ** 2 + s.grads.double().norm() ** 2).sqrt())
    assert not c["skip"] and abs(c["norm"] - norm) <= 1e-5 * norm
    assert not torch.equal(s.table, before[0]) and not torch.equal(s.params, before[1])
    assert bool(s.table.float().isfinite().all()) and bool(s.params.float().isfinite().all())


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_captured_step_replays_bitwise(gpu, dt):
    eager = Step(gpu, dt, 4)
    ref = []
    for _ in range(3):
        eager.step()
        torch.cuda.synchronize()
        ref.append([t.clone() for t in eager.tensors()])
    cap = Step(gpu, dt, 4)
    start = [t.clone() for t in cap.tensors()]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            cap.step()
    torch.cuda.synchronize()
    for t, s0 in zip(cap.tensors(), start):
        t.copy_(s0)
    torch.cuda.synchronize()
    gen = torch.Generator(device=gpu)
    gen.manual_seed(1)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        torch.randn(1 << 20, generator=gen, device=gpu).mul_(2.0)  # eager work between
        torch.cuda.synchronize()
        for a, b in zip(cap.tensors(), ref[k]):
            assert same_bits(a, b), k


def test_two_streams_at_once(gpu):
    # each stream with its own tensors and workspaces
    ref = Step(gpu, "bf16", 5)
    ref.gradients()
    steps = [Step(gpu, "bf16", 5), Step(gpu, "bf16", 5)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.gradients()
    torch.cuda.synchronize()
    for s in steps:
        assert same_bits(s.grads, ref.grads) and same_bits(s.dtable, ref.dtable)
        assert same_bits(s.loss, ref.loss)
