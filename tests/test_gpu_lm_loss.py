"""The vocabulary loss and its gradient against fp64.

Bounds, with STEP = 2^-23 (one step: matrix cores need not round to nearest)
and U = 2^-24.  Logits: d_t = (dim + 1) STEP max_v sum|h||w|.  Each term of
the sum of exponentials is off by E relative (argument and exp: 2^-19 with
the hardware's exp of the bf16 path, 2^-20 with the accurate one), the sum by
its longest chain of additions, (64 + vocab / 64) U; so lse is off by
r_t = d_t + E + (64 + vocab / 64) U + 2 STEP |lse|, the loss by r_t + d_t and
one rounding.  g is off by |dloss| (p (r_t + d_t + E) + U) plus, in bf16, half
a step of itself.  dhidden and dweight: those errors times |w| and |h|, the
additions of vocab + 16 or n terms, half a step of the result."""

import math

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import DT, HALF, assert_within, fill_normal, guarded, same_bits

pytestmark = pytest.mark.gpu

STEP, U = 2.0 ** -23, 2.0 ** -24


class Ref:
    def __init__(self, h, w, tgt, dloss, dt):
        h, w = h.double(), w.double()
        n, vocab, dim = h.shape[0], w.shape[0], w.shape[1]
        e = 2.0 ** -19 if dt == "bf16" else 2.0 ** -20
        logits = h @ w.t()
        d = (dim + 1) * STEP * (h.abs() @ w.abs().t()).max(1).values if n else h.new_zeros(0)
        self.ok = (tgt >= 0) & (tgt < vocab)
        self.lse = torch.logsumexp(logits, 1)
        at = logits.gather(1, tgt.clamp(0, vocab - 1).long()[:, None])[:, 0]
        self.loss = torch.where(self.ok, self.lse - at, torch.zeros_like(at))
        r = d + e + (64 + vocab / 64) * U + 2 * STEP * self.lse.abs()
        self.lse_bound = 1.01 * r
        self.loss_bound = 1.01 * torch.where(self.ok, r + d + U * self.loss.abs(),
                                             torch.zeros_like(r))
        if dloss is None:
            return
        dl = torch.where(self.ok, dloss.double(), torch.zeros_like(r))
        p = torch.exp(logits - self.lse[:, None])
        g = p.clone()
        rows = self.ok.nonzero()[:, 0]
        g[rows, tgt[rows].long()] -= 1.0
        g *= dl[:, None]
        err = dl.abs()[:, None] * (p * (r + d + e)[:, None] + U)
        if dt == "bf16":
            err = err + g.abs() * HALF[torch.bfloat16]
        self.dh = g @ w
        self.dh_err = err @ w.abs() + (vocab + 16) * STEP * (g.abs() @ w.abs())
        self.dw = g.t() @ h
        self.dw_err = err.t() @ h.abs() + (n + 1) * STEP * (g.abs().t() @ h.abs())


def _inputs(gpu, n, vocab, dim, dt, off, pad, t64, ignored=0.2):
    g = torch.Generator(device=gpu)
    g.manual_seed(n + vocab + dim)
    h, _ = guarded((n, dim), DT[dt], gpu, off, dim + pad)
    w, _ = guarded((vocab, dim), DT[dt], gpu, off)
    fill_normal(h, 1.0, g)
    fill_normal(w, 1.5 / math.sqrt(dim), g)
    tgt = torch.randint(0, vocab, (n,), generator=g, device=gpu)
    gone = torch.rand(n, generator=g, device=gpu) < ignored
    tgt[gone] = -100
    if n > 6:
        tgt[1], tgt[2], tgt[3], tgt[4] = vocab - 1, 0, vocab, -1
    tgt = tgt if t64 else tgt.int()
    dl = torch.rand(n, generator=g, device=gpu) + 0.5
    if n > 6:
        dl[3] = float("nan")  # of a row without a target: unused
        dl[5] = 0.0
    return h, w, tgt, dl


CASES = [
    # n, vocab, dim, dtype, dhidden, dweight, off, pad, t64, acc
    (1, 1, 1, "fp32", "fp32", "fp32", 0, 0, 1, 0),
    (1, 1000, 64, "bf16", "bf16", "bf16", 0, 0, 1, 0),
    (7, 5, 33, "bf16", "bf16", "bf16", 1, 3, 0, 0),
    (33, 257, 128, "bf16", "fp32", "fp32", 0, 8, 1, 1),
    (33, 4099, 256, "bf16", "bf16", "bf16", 0, 0, 1, 0),
    (128, 128, 32, "bf16", "bf16", "bf16", 0, 0, 0, 0),
    (129, 385, 100, "fp32", "fp32", "fp32", 3, 1, 1, 0),
    (129, 127, 257, "fp32", "bf16", "bf16", 0, 0, 0, 1),
    (300, 1000, 264, "bf16", "bf16", "fp32", 0, 0, 1, 1),
    (300, 777, 101, "bf16", "fp32", "bf16", 1, 0, 1, 1),
    (513, 1025, 512, "bf16", "bf16", "bf16", 0, 16, 1, 0),
    (257, 2048, 40, "bf16", "bf16", "bf16", 0, 0, 1, 0),
]


@pytest.mark.parametrize("n,vocab,dim,dt,hd,wd,off,pad,t64,acc", CASES)
def test_loss_and_gradients(gpu, n, vocab, dim, dt, hd, wd, off, pad, t64, acc):
    h, w, tgt, dl = _inputs(gpu, n, vocab, dim, dt, off, pad, t64)
    ref = Ref(h, w, tgt, dl, dt)
    ws = torch.full((M.lm_loss_workspace_size(n, vocab, dim, dt),), 255, dtype=torch.uint8,
                    device=gpu)
    loss, lse = M.lm_loss_forward(h, w, tgt, workspace=ws)
    assert_within(lse, ref.lse, ref.lse_bound)
    assert_within(loss, ref.loss, ref.loss_bound)
    assert not bool(loss[~ref.ok].any())

    dh, check_h = guarded((n, dim), DT[hd], gpu, off, dim + pad)
    dh.fill_(float("nan"))
    dw, check_w = guarded((vocab, dim), DT[wd], gpu, off)
    dw.fill_(float("nan"))
    old = None
    if acc:
        g = torch.Generator(device=gpu)
        g.manual_seed(1)
        fill_normal(dw, 1.0, g)
        old = dw.clone()
    out = M.lm_loss_backward(h, w, tgt, lse, dl, dhidden=dh, dweight=dw, accumulate=bool(acc),
                             workspace=ws)
    assert out[0] is dh and out[1] is dw
    torch.cuda.synchronize()
    check_h()
    check_w()
    assert_within(dh, ref.dh, 1.01 * (ref.dh_err + ref.dh.abs() * HALF[DT[hd]]))
    want, err = ref.dw, ref.dw_err
    if acc:
        want = want + old.double()
        err = err + (want.abs() + old.double().abs()) * STEP
    assert_within(dw, want, 1.01 * (err + want.abs() * HALF[DT[wd]]))
    assert not bool(dh[~ref.ok].any())

    # each gradient alone, in fresh outputs, gives the same bits; and again
    dh2, none = M.lm_loss_backward(h, w, tgt, lse, dl, dhidden=torch.empty_like(dh), dweight=False)
    assert none is None and same_bits(dh2, dh)
    dw2 = old.clone() if acc else torch.empty_like(dw)
    none, _ = M.lm_loss_backward(h, w, tgt, lse, dl, dhidden=False, dweight=dw2,
                                 accumulate=bool(acc))
    assert none is None and same_bits(dw2, dw)
    loss2, lse2 = M.lm_loss_forward(h, w, tgt)
    assert same_bits(loss2, loss) and same_bits(lse2, lse)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_several_pieces_of_the_vocabulary(gpu, dt):
    # n * vocab beyond one piece of the logits' gradient
    n, vocab, dim = 8200, 20011, 24
    h, w, tgt, dl = _inputs(gpu, n, vocab, dim, dt, 0, 0, 1)
    ref = Ref(h, w, tgt, dl, dt)
    loss, lse = M.lm_loss_forward(h, w, tgt)
    assert_within(loss, ref.loss, ref.loss_bound)
    dh, dw = M.lm_loss_backward(h, w, tgt, lse, dl)
    assert_within(dh, ref.dh, 1.01 * (ref.dh_err + ref.dh.abs() * HALF[DT[dt]]))
    assert_within(dw, ref.dw, 1.01 * (ref.dw_err + ref.dw.abs() * HALF[DT[dt]]))


def test_several_passes_over_the_rows(gpu):
    # more rows than one pass of the forward's tile statistics
    n, vocab, dim = 40000, 300, 16
    h, w, tgt, dl = _inputs(gpu, n, vocab, dim, "bf16", 0, 0, 1)
    ref = Ref(h, w, tgt, None, "bf16")
    loss, lse = M.lm_loss_forward(h, w, tgt)
    assert_within(loss, ref.loss, ref.loss_bound)
    assert_within(lse, ref.lse, ref.lse_bound)


def test_no_rows(gpu):
    h = torch.empty(0, 8, dtype=torch.bfloat16, device=gpu)
    w = torch.ones(5, 8, dtype=torch.bfloat16, device=gpu)
    tgt = torch.empty(0, dtype=torch.int64, device=gpu)
    loss, lse = M.lm_loss_forward(h, w, tgt)
    assert loss.numel() == 0 and lse.numel() == 0
    dh, dw = M.lm_loss_backward(h, w, tgt, lse, loss,
                                dweight=torch.full((5, 8), 3.0, device=gpu))
    assert dh.shape == (0, 8) and not bool(dw.any())
    dw = torch.full((5, 8), 3.0, device=gpu)
    M.lm_loss_backward(h, w, tgt, lse, loss, dweight=dw, accumulate=True)
    assert bool((dw == 3).all())


def test_no_labelled_rows(gpu):
    g = torch.Generator(device=gpu)
    g.manual_seed(2)
    h = torch.randn(70, 32, generator=g, device=gpu).to(torch.bfloat16)
    w = torch.randn(200, 32, generator=g, device=gpu).to(torch.bfloat16)
    tgt = torch.full((70,), -100, device=gpu)
    loss, lse = M.lm_loss_forward(h, w, tgt)
    assert not bool(loss.any()) and bool(lse.isfinite().all())
    dh, dw = M.lm_loss_backward(h, w, tgt, lse, torch.full((70,), float("nan"), device=gpu))
    assert not bool(dh.any()) and not bool(dw.any())


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_extreme_logits(gpu, dt):
    # logits of +-6e4 (exp overflows and underflows without the running
    # maximum), equal ones, a row of zeros, a NaN row, an infinite row
    dim, vocab = 8, 300
    w = torch.zeros(vocab, dim, dtype=DT[dt], device=gpu)
    w[:, 0] = torch.where(torch.arange(vocab, device=gpu) % 2 == 0, 1.0, -1.0).to(DT[dt])
    w[7, 0] = 2.0
    h = torch.zeros(6, dim, dtype=DT[dt], device=gpu)
    h[0, 0], h[1, 0], h[3, 0] = 30000.0, -30000.0, 0.5
    h[4, 1] = float("nan")
    h[5, 0] = float("inf")
    tgt = torch.tensor([7, 1, 5, 7, 3, 2], device=gpu)
    loss, lse = M.lm_loss_forward(h, w, tgt)
    big = float(h[0, 0])  # 30000 as the type holds it
    assert float(lse[0]) == 2 * big and float(loss[0]) == 0.0
    # the 149 odd rows but row 7 have logit 30000
    assert abs(float(lse[1]) - (big + math.log(149))) <= 0.01
    assert abs(float(loss[1]) - math.log(149)) <= 0.01
    assert abs(float(loss[2]) - math.log(300)) <= 1e-5
    assert bool(lse[4].isnan()) and bool(loss[4].isnan()) and not bool(lse[5].isfinite())
    dl = torch.ones(6, device=gpu)
    dh, dw = M.lm_loss_backward(h[:4], w, tgt[:4], lse[:4].contiguous(), dl[:4])
    assert bool(dh.isfinite().all()) and bool(dw.isfinite().all())
    assert not bool(dh[0].any())   # p is exactly the one-hot target
    # a row that is not finite keeps to its own dhidden
    dh6, _ = M.lm_loss_backward(h, w, tgt, lse, dl, dweight=False)
    assert same_bits(dh6[:4], dh) and bool(dh6[4].isnan().all())


def test_gradients_against_differences(gpu):
    # central differences of the fp32 loss along random directions: off by
    # R^3 eps^2 / 6 (the third cumulant along a direction whose logits span R
    # is at most R^3) and by the two losses' errors over 2 eps
    n, vocab, dim = 5, 61, 19
    h, w, tgt, dl = _inputs(gpu, n, vocab, dim, "fp32", 0, 0, 1, ignored=0.0)
    loss, lse = M.lm_loss_forward(h, w, tgt)
    dh, dw = M.lm_loss_backward(h, w, tgt, lse, dl)
    g = torch.Generator(device=gpu)
    g.manual_seed(9)
    eps = 2.0 ** -6
    for which in ("h", "w"):
        for _ in range(3):
            v = torch.randn(h.shape if which == "h" else w.shape, generator=g, device=gpu)
            vals = []
            for s in (1.0, -1.0):
                a = h + s * eps * v if which == "h" else h
                b = w + s * eps * v if which == "w" else w
                vals.append(float((M.lm_loss_forward(a, b, tgt)[0].double() * dl.double()).sum()))
            slope = (vals[0] - vals[1]) / (2 * eps)
            grad = dh if which == "h" else dw
            dirv = (v.double() @ w.double().t()) if which == "h" else (h.double() @ v.double().t())
            span = (dirv.max(1).values - dirv.min(1).values)
            ref = Ref(h, w, tgt, dl, "fp32")
            tol = float((dl.double() * (span ** 3 * eps ** 2 / 6 + 2 * ref.loss_bound / eps)).sum())
            # the evaluation points are rounded to fp32: 2^-24 of each value
            tol += float((dl.double() * span).sum()) * 2.0 ** -24 / eps * 8
            assert abs(slope - float((grad.double() * v.double()).sum())) <= tol
