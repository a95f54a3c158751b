"""The losses of fine-tuning together, as a step uses them: the token losses of
the head feed a policy and a preference loss, whose gradients are the head's
dloss; a teacher's lists add theirs to the same table gradient; AdamW steps the
table.

    nll = CE(h E^T, targets);  L = sum_s a_s policy_s(nll) + sum_i b_i pref_i(nll)
                                   + sum_t c_t KL_t(h E^T / T, lists)

Bound, relative to the norm of each gradient.  Two products in a row, each
element off by (K + 1) 2^-23 sqrt(K) of the sizes of its terms typically, K <=
300: 2 * 301 * 2^-23 * sqrt(300) = 1.3e-3 in fp32.  bf16 adds a rounding of 2^-8
at each of at most 3 places where a value is stored, 1.2e-2, and the inputs of
the reference are the same bf16 values."""

import pytest
import torch

import muon_newton_schulz_amd as M
from muon_newton_schulz_amd import workloads as W
from train_ops_util import DT, same_bits

pytestmark = pytest.mark.gpu

N, V, D, K, S = 260, 300, 64, 12, 8
T = 1.7
POLICY = dict(clip_low=0.2, clip_high=0.28, kl_weight=0.1)
PREFERENCE = dict(beta=0.3, smoothing=0.1)


class Step:
    """Inputs, gradients, workspaces and one step."""

    def __init__(self, gpu, dt, seed):
        g = torch.Generator(device=gpu)
        g.manual_seed(seed)
        t = DT[dt]
        r = lambda *s: torch.randn(*s, generator=g, device=gpu)  # noqa: E731
        self.dt = dt
        self.table = (r(V, D) * 0.2).to(t)
        self.master = self.table.float() if dt == "bf16" else None
        self.h = r(N, D).to(t)
        # prompts have no targets; the last rows are padding behind the sequences
        self.targets = torch.randint(-90, V, (N,), generator=g, device=gpu)
        self.mask = self.targets >= 0
        self.offsets = torch.tensor([0, 31, 31, 75, 76, 140, 180, 233, 250], dtype=torch.int32,
                                    device=gpu)
        base = M.lm_loss_forward(self.h, self.table, self.targets)[0]
        self.old, self.ref = base + r(N) * 0.2, base + r(N) * 0.3
        self.adv = r(S)
        self.a, self.b = r(S) * 0.1, r(S // 2) * 0.1
        self.ids = torch.randint(-30, V, (N, K), generator=g, device=gpu)
        self.teacher = r(N, K).to(t)
        self.c = torch.rand(N, generator=g, device=gpu) / N
        self.c[250:] = 0.0
        e = lambda *s: torch.zeros(*s, device=gpu)  # noqa: E731
        self.dpol, self.dpre = e(N), e(N)
        self.dh, self.dh2 = torch.empty_like(self.h), torch.empty_like(self.h)
        self.dtable = torch.empty_like(self.table)
        self.m, self.v = e(V * D), e(V * D)
        need = max(M.lm_loss_workspace_size(N, V, D, dt),
                   M.distill_loss_workspace_size(N, V, D, K, dt),
                   M.sequence_loss_workspace_size(N, S))
        self.ws = torch.empty(need, dtype=torch.uint8, device=gpu)
        self.out = []

    def step(self):
        nll, lse = M.lm_loss_forward(self.h, self.table, self.targets, workspace=self.ws)
        pol = M.policy_loss_forward(nll, self.old, self.adv, self.offsets, ref_nll=self.ref,
                                    mask=self.mask, workspace=self.ws, **POLICY)
        pre = M.preference_loss_forward(nll, self.offsets, ref_nll=self.ref, mask=self.mask,
                                        workspace=self.ws, **PREFERENCE)
        M.policy_loss_backward(nll, self.old, self.adv, self.offsets, pol[2], self.a,
                               ref_nll=self.ref, mask=self.mask, dnll=self.dpol, **POLICY)
        M.preference_loss_backward(self.offsets, pre[1], pre[3], self.b, mask=self.mask,
                                   dnll=self.dpre, **PREFERENCE)
        M.lm_loss_backward(self.h, self.table, self.targets, lse, self.dpol + self.dpre,
                           dhidden=self.dh, dweight=self.dtable, workspace=self.ws)
        kl = M.distill_loss_forward(self.h, self.table, self.ids, self.teacher, T,
                                    workspace=self.ws)
        M.distill_loss_backward(self.h, self.table, self.ids, self.teacher, kl[1], kl[2], self.c, T,
                                dhidden=self.dh2, dweight=self.dtable, accumulate=True,
                                workspace=self.ws)
        master = None if self.master is None else self.master.view(-1)
        M.adamw_step(self.table.view(-1), master, self.dtable.view(-1), self.m, self.v,
                     W.AdamWHParams(), 1)
        self.out = [nll, *pol, *pre, *kl]

    def tensors(self):
        held = [self.dh, self.dh2, self.dtable, self.table, self.dpol, self.dpre, self.m, self.v]
        return held + ([self.master] if self.master is not None else []) + self.out


def _reference(s):
    """Losses and gradients by autograd in fp64 from the step's inputs."""
    h, table = s.h.double().requires_grad_(), s.table.double().requires_grad_()
    logits = h @ table.t()
    at = logits.gather(1, s.targets.clamp(min=0)[:, None])[:, 0]
    nll = torch.where(s.mask, torch.logsumexp(logits, 1) - at, torch.zeros_like(at))
    b = s.offsets.tolist()
    total = 0.0
    for q in range(S):
        use = s.mask[b[q]:b[q + 1]]
        x = nll[b[q]:b[q + 1]][use]
        if not x.numel():
            continue
        r = torch.exp(s.old[b[q]:b[q + 1]][use].double() - x)
        adv = s.adv[q].double()
        clip = r.clamp(1 - POLICY["clip_low"], 1 + POLICY["clip_high"])
        d = x - s.ref[b[q]:b[q + 1]][use].double()
        token = -torch.minimum(r * adv, clip * adv) + POLICY["kl_weight"] * (d.exp() - 1 - d)
        total = total + s.a[q].double() * token.mean()
    reward = [PREFERENCE["beta"] * (s.ref[b[q]:b[q + 1]].double() - nll[b[q]:b[q + 1]])
              [s.mask[b[q]:b[q + 1]]].sum() for q in range(S)]
    e = PREFERENCE["smoothing"]
    for i in range(S // 2):
        if s.mask[b[2 * i]:b[2 * i + 1]].any() and s.mask[b[2 * i + 1]:b[2 * i + 2]].any():
            x = reward[2 * i] - reward[2 * i + 1]
            sp = torch.nn.functional.softplus
            total = total + s.b[i].double() * ((1 - e) * sp(-x) + e * sp(x))
    h2 = s.h.double().requires_grad_()
    logp = torch.log_softmax(h2 @ table.t() / T, 1).gather(1, s.ids.clamp(min=0))
    there = s.ids >= 0
    lq = torch.log_softmax(torch.where(there, s.teacher.double() / T,
                                       torch.full_like(logp, -1e9)), 1)
    kl = torch.where(there, lq.exp() * (lq - logp), torch.zeros_like(logp)).sum(1)
    kl = torch.where(there.any(1), kl, torch.zeros_like(kl))
    total = total + (kl * s.c.double()).sum()
    total.backward()
    return h.grad, h2.grad, table.grad, kl.detach()


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_step_against_fp64_autograd(gpu, dt):
    s = Step(gpu, dt, 3)
    dh, dh2, dtable, kl = _reference(s)
    before = s.table.clone()
    s.step()
    torch.cuda.synchronize()
    tol = 1.3e-3 + (1.2e-2 if dt == "bf16" else 0.0)
    for got, want in ((s.dh, dh), (s.dh2, dh2), (s.dtable, dtable)):
        assert float(want.norm()) > 0
        assert float((got.double() - want).norm()) <= tol * float(want.norm())
    assert float((s.out[9].double() - kl).norm()) <= tol * float(kl.norm())
    # padding behind the sequences and rows without a target have no gradient
    assert not bool(s.dh[250:].any()) and not bool(s.dh[~s.mask].any())
    assert not torch.equal(s.table, before) and bool(s.table.float().isfinite().all())


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_captured_step_replays_bitwise(gpu, dt):
    eager = Step(gpu, dt, 4)
    ref = []
    for _ in range(3):
        eager.step()
        torch.cuda.synchronize()
        ref.append([t.clone() for t in eager.tensors()])
    cap = Step(gpu, dt, 4)
    cap.step()  # sizes of everything that a step leaves
    start = Step(gpu, dt, 4)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            cap.step()
    torch.cuda.synchronize()
    for name in ("table", "master", "m", "v"):
        if getattr(cap, name) is not None:
            getattr(cap, name).copy_(getattr(start, name))
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
    ref.step()
    steps = [Step(gpu, "bf16", 5), Step(gpu, "bf16", 5)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, st in zip(steps, streams):
        with torch.cuda.stream(st):
            s.step()
    torch.cuda.synchronize()
    for s in steps:
        for a, b in zip(s.tensors(), ref.tensors()):
            assert same_bits(a, b)


def test_a_stream_that_is_not_the_current_one(gpu):
    s = Step(gpu, "bf16", 6)
    nll, _ = M.lm_loss_forward(s.h, s.table, s.targets)
    how = dict(ref_nll=s.ref, mask=s.mask, **POLICY)
    want = M.policy_loss_forward(nll, s.old, s.adv, s.offsets, **how)
    dwant = M.policy_loss_backward(nll, s.old, s.adv, s.offsets, want[2], s.a, **how)
    pre = M.preference_loss_forward(nll, s.offsets, mask=s.mask)
    dpre = M.preference_loss_backward(s.offsets, pre[1], pre[3], s.b, mask=s.mask)
    kl = M.distill_loss_forward(s.h, s.table, s.ids, s.teacher, T)
    dkl = M.distill_loss_backward(s.h, s.table, s.ids, s.teacher, kl[1], kl[2], s.c, T)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = M.policy_loss_forward(nll, s.old, s.adv, s.offsets, stream=stream, **how)
        dgot = M.policy_loss_backward(nll, s.old, s.adv, s.offsets, got[2], s.a, stream=stream,
                                      **how)
        pre2 = M.preference_loss_forward(nll, s.offsets, mask=s.mask, stream=stream)
        dpre2 = M.preference_loss_backward(s.offsets, pre2[1], pre2[3], s.b, mask=s.mask,
                                           stream=stream)
        kl2 = M.distill_loss_forward(s.h, s.table, s.ids, s.teacher, T, stream=stream)
        dkl2 = M.distill_loss_backward(s.h, s.table, s.ids, s.teacher, kl2[1], kl2[2], s.c, T,
                                       stream=stream)
        side.synchronize()
        for a, b in zip((*want, dwant, *pre, dpre, *kl, *dkl),
                        (*got, dgot, *pre2, dpre2, *kl2, *dkl2)):
            assert same_bits(a, b)


def test_the_losses_are_not_recorded_by_autograd(gpu):
    s = Step(gpu, "fp32", 7)
    s.table.requires_grad_()
    kl = M.distill_loss_forward(s.h, s.table, s.ids, s.teacher)
    nll = torch.rand(N, device=gpu, requires_grad=True)
    pol = M.policy_loss_forward(nll, s.old, s.adv, s.offsets)
    pre = M.preference_loss_forward(nll, s.offsets)
    assert not any(t.requires_grad for t in (*kl, *pol, *pre))
