"""The distillation loss and its gradient against fp64.

Bounds, with STEP = 2^-23, U = 2^-24 and everything about the products and the
sum of exponentials as in test_gpu_lm_loss.py: scaled logits are off by d_t =
(dim + 1) STEP max_v sum|h||w| / T and by 2 STEP of themselves (1 / T and the
product round), lse by r_t = d_t + E + (64 + vocab / 64) U + 2 STEP |lse|.
  logp: r_t + d_t, and the roundings of l - m, of log s and of their
  difference, 4 STEP (|logp| + log vocab).
  log q: its argument and the logarithm of the sum round, 4 STEP |log q|, and
  the sum of at most 16 terms a lane and 6 joins has exp's 2^-20 and 22 U; q has
  that and exp's own error, 2^-20, relative to itself.
  loss: the sum over the list of q times (log q - logp) with those errors, and
  22 additions.
  g: |dloss| / T times p's error, p (r_t + d_t + E) (listed: p (that of logp +
  2^-20)), and q's; four roundings of itself; in bf16 calls, whose g is two bf16
  values, 2^-16 of itself.
dhidden and dweight: those errors times |w| and |h|, the additions of vocab +
16 or n terms, half a step of the result."""

import math

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import DT, HALF, assert_within, fill_normal, guarded, same_bits

pytestmark = pytest.mark.gpu

STEP, U = 2.0 ** -23, 2.0 ** -24


class Ref:
    def __init__(self, h, w, ids, z, T, dloss, dt):
        h, w = h.double(), w.double()
        n, vocab, dim = h.shape[0], w.shape[0], w.shape[1]
        e = 2.0 ** -19 if dt == "bf16" else 2.0 ** -20
        logits = (h @ w.t()) / T
        big = logits.abs().max(1).values if n else h.new_zeros(0)
        d = ((dim + 1) * STEP * (h.abs() @ w.abs().t()).max(1).values / T if n
             else h.new_zeros(0)) + 2 * STEP * big
        self.lse = torch.logsumexp(logits, 1)
        r = d + e + (64 + vocab / 64) * U + 2 * STEP * self.lse.abs()
        self.lse_bound = 1.01 * r
        counts = (ids >= 0) & (ids < vocab) & ~(z == -math.inf)
        self.ok = counts.any(1)
        safe = torch.where(counts, ids.long(), torch.zeros_like(ids.long()))
        zz = torch.where(counts, z.double() / T, torch.full_like(z.double(), -math.inf))
        top = zz.max(1, keepdim=True).values
        total = torch.where(counts, (zz - top).exp(), torch.zeros_like(zz)).sum(1, keepdim=True)
        zero = torch.zeros_like(zz)
        lq = torch.where(counts, zz - top - total.log(), zero)
        q = torch.where(counts, lq.exp(), zero)
        lp = torch.where(counts, logits.gather(1, safe) - self.lse[:, None], zero)
        self.logp = lp
        lp_err = (r + d)[:, None] + 4 * STEP * (lp.abs() + math.log(vocab) + 1)
        self.logp_bound = 1.01 * torch.where(counts, lp_err, zero)
        q_err = 4 * STEP * lq.abs() + 2.0 ** -19 + 44 * U
        gap = torch.where(q > 0, lq - lp, zero)   # (0 log 0 = 0)
        self.loss = (q * gap).sum(1)
        q_fin = torch.where(q > 0, q_err, zero)
        self.loss_bound = 1.01 * ((q * (q_fin * (1 + gap.abs()) + lp_err)).sum(1)
                                  + 22 * STEP * (q * gap).abs().sum(1) + 2.0 ** -126)
        if dloss is None:
            return
        dl = torch.where(self.ok, dloss.double(), torch.zeros_like(r)) / T
        p = torch.exp(logits - self.lse[:, None])
        err = p * (r + d + e)[:, None]
        qs = torch.zeros_like(p).scatter_add_(1, safe, q)
        listed = torch.zeros_like(p).scatter_add_(1, safe, torch.where(counts, lp_err, zero))
        err = torch.where(listed > 0, p * (listed + 2.0 ** -19), err)
        err = err + torch.zeros_like(p).scatter_add_(1, safe, q * q_fin) + 4 * U * (p + qs)
        g = (p - qs) * dl[:, None]
        err = dl.abs()[:, None] * err + 8 * U * g.abs()
        if dt == "bf16":
            err = err + 2.0 ** -16 * g.abs()
        self.g = g
        self.dh = g @ w
        self.dh_err = err @ w.abs() + (vocab + 16) * STEP * (g.abs() @ w.abs())
        self.dw = g.t() @ h
        self.dw_err = err.t() @ h.abs() + (n + 1) * STEP * (g.abs().t() @ h.abs())


def _inputs(gpu, n, vocab, dim, top, dt, zt, off=0, pad=0, i64=1, kind="spread"):
    g = torch.Generator(device=gpu)
    g.manual_seed(n + vocab + dim + top)
    h, _ = guarded((n, dim), DT[dt], gpu, off, dim + pad)
    w, _ = guarded((vocab, dim), DT[dt], gpu, off)
    fill_normal(h, 1.0, g)
    fill_normal(w, 1.5 / math.sqrt(dim), g)
    z, _ = guarded((n, top), DT[zt], gpu, off, top + pad)
    fill_normal(z, 2.0, g)
    ids = torch.empty((n, top + pad), dtype=torch.int64 if i64 else torch.int32,
                      device=gpu)[:, :top]
    if kind == "near":  # lists in a few columns, most of them named more than once
        lo = int(torch.randint(0, vocab, (1,), generator=g, device=gpu))
        ids.copy_((torch.randint(0, max(1, min(vocab, 40)), (n, top), generator=g, device=gpu) + lo)
                  % vocab)
    else:
        ids.copy_(torch.randint(-max(1, vocab // 10), vocab + max(1, vocab // 20), (n, top),
                                generator=g, device=gpu))
    if n > 6:
        ids[1], ids[2] = -1, vocab              # lists with nothing in them
        ids[3, 0], ids[4, top - 1] = vocab - 1, 0
        z[5, :top // 2] = -math.inf
        z[6, :top // 2] = torch.finfo(DT[zt]).min
        if top > 1:
            ids[5, 1] = ids[5, 0]
    dl = torch.rand(n, generator=g, device=gpu) + 0.5
    if n > 6:
        dl[1] = float("nan")  # of a row without a list: unused
    return h, w, ids, z, dl


CASES = [
    # n, vocab, dim, top, dtype, teacher, T, dhidden, dweight, off, pad, i64, acc, kind
    (1, 1, 1, 1, "fp32", "fp32", 1.0, "fp32", "fp32", 0, 0, 1, 0, "near"),
    (1, 1000, 64, 3, "bf16", "fp32", 1.0, "bf16", "bf16", 0, 0, 1, 0, "spread"),
    (7, 5, 33, 9, "bf16", "bf16", 2.0, "bf16", "bf16", 1, 3, 0, 0, "near"),
    (33, 257, 128, 64, "bf16", "fp32", 0.7, "fp32", "fp32", 0, 8, 1, 1, "spread"),
    (33, 4099, 256, 65, "bf16", "bf16", 1.0, "bf16", "bf16", 0, 0, 1, 0, "near"),
    (128, 128, 32, 128, "bf16", "fp32", 3.0, "bf16", "bf16", 0, 0, 0, 0, "near"),
    (129, 385, 100, 17, "fp32", "fp32", 1.0, "fp32", "fp32", 3, 1, 1, 0, "spread"),
    (129, 127, 257, 200, "fp32", "bf16", 0.5, "bf16", "bf16", 0, 0, 0, 1, "spread"),
    (300, 1000, 264, 31, "bf16", "fp32", 1.0, "bf16", "fp32", 0, 0, 1, 1, "near"),
    (300, 777, 101, 300, "bf16", "bf16", 2.0, "fp32", "bf16", 1, 0, 1, 1, "spread"),
    (513, 1025, 512, 8, "bf16", "fp32", 1.0, "bf16", "bf16", 0, 16, 1, 0, "spread"),
    (257, 2048, 40, 1024, "bf16", "fp32", 1.0, "bf16", "bf16", 0, 0, 1, 0, "spread"),
    # rows off the grid that are laid out on it: backward, and both
    (95, 500, 205, 12, "bf16", "fp32", 1.0, "bf16", "bf16", 0, 0, 1, 0, "spread"),
    (96, 500, 205, 12, "bf16", "fp32", 1.0, "bf16", "fp32", 1, 5, 1, 1, "spread"),
    (511, 300, 1, 12, "bf16", "fp32", 1.0, "fp32", "bf16", 0, 0, 1, 0, "near"),
    (512, 1000, 1001, 7, "bf16", "bf16", 2.0, "bf16", "bf16", 3, 1, 0, 0, "spread"),
    (700, 900, 262, 40, "bf16", "fp32", 1.0, "fp32", "bf16", 0, 0, 1, 1, "near"),
]


@pytest.mark.parametrize("n,vocab,dim,top,dt,zt,T,hd,wd,off,pad,i64,acc,kind", CASES)
def test_loss_and_gradients(gpu, n, vocab, dim, top, dt, zt, T, hd, wd, off, pad, i64, acc, kind):
    h, w, ids, z, dl = _inputs(gpu, n, vocab, dim, top, dt, zt, off, pad, i64, kind)
    ref = Ref(h, w, ids, z, T, dl, dt)
    ws = torch.full((M.distill_loss_workspace_size(n, vocab, dim, top, dt),), 255,
                    dtype=torch.uint8, device=gpu)
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z, T, workspace=ws)
    assert_within(lse, ref.lse, ref.lse_bound)
    assert_within(logp, ref.logp, ref.logp_bound)
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
    out = M.distill_loss_backward(h, w, ids, z, lse, logp, dl, T, dhidden=dh, dweight=dw,
                                  accumulate=bool(acc), workspace=ws)
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
    dh2, none = M.distill_loss_backward(h, w, ids, z, lse, logp, dl, T,
                                        dhidden=torch.empty_like(dh), dweight=False)
    assert none is None and same_bits(dh2, dh)
    dw2 = old.clone() if acc else torch.empty_like(dw)
    none, _ = M.distill_loss_backward(h, w, ids, z, lse, logp, dl, T, dhidden=False, dweight=dw2,
                                      accumulate=bool(acc))
    assert none is None and same_bits(dw2, dw)
    again = M.distill_loss_forward(h, w, ids, z, T)
    assert same_bits(again[0], loss) and same_bits(again[1], lse) and same_bits(again[2], logp)


# one for each tile core of the statistics: Thin, Medium, Half, Large; any
# operands bf16 and fp32, 64 and 128 (test_tile_core_coverage.py's sizes)
@pytest.mark.parametrize("n,vocab,dim,top,dt,off", [
    (128, 2000, 1032, 64, "bf16", 0), (128, 20011, 264, 65, "bf16", 0),
    (129, 20011, 264, 64, "bf16", 0), (100, 8000, 1541, 33, "bf16", 1),
    (128, 8000, 1541, 64, "fp32", 0), (40, 300, 261, 50, "fp32", 0),
    (130, 2000, 1032, 20, "bf16", 0), (40, 20011, 264, 64, "bf16", 0),
    (600, 20011, 520, 70, "bf16", 0), (4000, 4000, 840, 33, "bf16", 0),
    (8200, 20011, 1032, 16, "bf16", 0), (130, 8000, 1544, 40, "bf16", 1),
    (2100, 2000, 264, 12, "bf16", 1), (130, 8000, 1541, 40, "bf16", 1),
    (2100, 2000, 261, 12, "bf16", 1), (8200, 20011, 133, 9, "bf16", 0), (130, 8000, 1541, 30, "fp32", 0),
    (2100, 2000, 261, 64, "fp32", 0)])
def test_tile_cores(gpu, n, vocab, dim, top, dt, off):
    h, w, ids, z, dl = _inputs(gpu, n, vocab, dim, top, dt, "fp32", off)
    ref = Ref(h, w, ids, z, 1.5, dl.nan_to_num(), dt)
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z, 1.5)
    assert_within(lse, ref.lse, ref.lse_bound)
    assert_within(logp, ref.logp, ref.logp_bound)
    assert_within(loss, ref.loss, ref.loss_bound)
    dh, dw = M.distill_loss_backward(h, w, ids, z, lse, logp, dl, 1.5)
    assert_within(dh, ref.dh, 1.01 * (ref.dh_err + ref.dh.abs() * HALF[DT[dt]]))
    assert_within(dw, ref.dw, 1.01 * (ref.dw_err + ref.dw.abs() * HALF[DT[dt]]))


def test_several_passes_over_the_rows(gpu):
    # more rows than one pass of the forward's tile statistics
    n, vocab, dim, top = 40000, 300, 16, 5
    h, w, ids, z, _ = _inputs(gpu, n, vocab, dim, top, "bf16", "bf16")
    ref = Ref(h, w, ids, z, 1.0, None, "bf16")
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z)
    assert_within(loss, ref.loss, ref.loss_bound)
    assert_within(lse, ref.lse, ref.lse_bound)
    assert_within(logp, ref.logp, ref.logp_bound)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_one_entry_is_cross_entropy(gpu, dt):
    # a teacher with one column a row: lm_loss, to the roundings of p - 1
    n, vocab, dim = 200, 500, 64
    h, w, ids, z, _ = _inputs(gpu, n, vocab, dim, 1, dt, "fp32")
    z.fill_(3.0)
    dl = torch.full((n,), 1.0 / n, device=gpu)
    tgt = torch.where((ids >= 0) & (ids < vocab), ids, torch.full_like(ids, -1))[:, 0]
    want, want_lse = M.lm_loss_forward(h, w, tgt.contiguous())
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z)
    assert same_bits(lse, want_lse)
    assert_within(loss, want.double(), 4 * STEP * (want.double().abs() + 10))
    dh, dw = M.distill_loss_backward(h, w, ids, z, lse, logp, dl,
                                     dhidden=torch.empty(n, dim, device=gpu),
                                     dweight=torch.empty(vocab, dim, device=gpu))
    dh2, dw2 = M.lm_loss_backward(h, w, tgt.contiguous(), lse, dl,
                                  dhidden=torch.empty(n, dim, device=gpu),
                                  dweight=torch.empty(vocab, dim, device=gpu))
    ref = Ref(h, w, ids, z, 1.0, dl, dt)
    assert_within(dh, dh2.double(), 2.02 * ref.dh_err)
    assert_within(dw, dw2.double(), 2.02 * ref.dw_err)


def test_gradient_is_small_where_the_student_is_the_teacher(gpu):
    # every column listed with the student's own logits: loss 0 and g 0, to the
    # errors of the two distributions
    n, vocab, dim = 40, 200, 48
    h, w, _, _, dl = _inputs(gpu, n, vocab, dim, 1, "fp32", "fp32")
    z = (h.double() @ w.double().t()).float()
    ids = torch.arange(vocab, device=gpu).flip(0).expand(n, vocab)
    z = z.flip(1).contiguous()
    dl = dl.nan_to_num(nan=1.0)
    ref = Ref(h, w, ids, z, 1.0, dl, "fp32")
    loss, lse, logp = M.distill_loss_forward(h, w, ids.contiguous(), z)
    assert_within(loss, ref.loss, ref.loss_bound)
    assert float(loss.abs().max()) < 1e-4
    dh, _ = M.distill_loss_backward(h, w, ids.contiguous(), z, lse, logp, dl, dweight=False)
    assert_within(dh, ref.dh, 1.01 * (ref.dh_err + ref.dh.abs() * HALF[torch.float32]))


@pytest.mark.parametrize("dt,n,vocab,dim", [("bf16", 70, 400, 64), ("bf16", 70, 400, 61),
                                            ("fp32", 70, 400, 61), ("bf16", 600, 2000, 1024)])
def test_rows_without_a_list_reach_no_gradient(gpu, dt, n, vocab, dim):
    h, w, ids, z, dl = _inputs(gpu, n, vocab, dim, 6, dt, "fp32")
    gone = torch.arange(n, device=gpu) % 5 == 1
    ids[gone] = -7
    z[gone.nonzero()[::2, 0]] = float("nan")   # of entries that do not count
    _, lse, logp = M.distill_loss_forward(h, w, ids, z)
    dl = torch.where(gone, dl, dl.nan_to_num(nan=1.0))
    dl[gone] = float("inf")
    ok = ((ids >= 0) & (ids < vocab) & ~(z == -math.inf)).any(1)
    dl[~ok] = float("inf")
    dh, dw = M.distill_loss_backward(h, w, ids, z, lse, logp, dl)
    assert bool(dw.isfinite().all()) and not bool(dh[gone].any())
    h[gone] = float("nan")
    loss2, lse2, logp2 = M.distill_loss_forward(h, w, ids, z)
    assert same_bits(lse2[~gone], lse[~gone]) and not bool(loss2[gone].any())
    dh2, dw2 = M.distill_loss_backward(h, w, ids, z, lse2, logp2, dl)
    assert same_bits(dw2, dw) and same_bits(dh2, dh)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_extreme_values(gpu, dt):
    # student logits of +-6e4, teacher values of the type's ends, NaN and +inf
    dim, vocab, top = 8, 300, 3
    w = torch.zeros(vocab, dim, dtype=DT[dt], device=gpu)
    w[:, 0] = torch.where(torch.arange(vocab, device=gpu) % 2 == 0, 1.0, -1.0).to(DT[dt])
    w[7, 0] = 2.0
    h = torch.zeros(6, dim, dtype=DT[dt], device=gpu)
    h[0, 0], h[3, 0] = 30000.0, 0.5
    ids = torch.tensor([[7, 0, 1], [5, 6, 7], [1, 2, 3], [4, 5, 6], [0, 1, 2], [3, 4, 5]],
                       device=gpu)
    big = torch.finfo(torch.float32).max
    z = torch.tensor([[0.0, -math.inf, -math.inf], [big, -big, -big], [-big, -big, -big],
                      [0.0, float("nan"), 0.0], [math.inf, 0.0, 0.0], [80.0, -80.0, 0.0]],
                     device=gpu)
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z)
    assert float(loss[0]) == 0.0 and float(logp[0, 0]) == 0.0
    assert float(lse[0]) == 2 * float(h[0, 0])
    assert abs(float(loss[1]) - math.log(300)) <= 1e-5
    assert abs(float(loss[2]) - (math.log(300) - math.log(3))) <= 1e-5
    assert bool(loss[3].isnan()) and bool(loss[4].isnan())
    assert abs(float(loss[5]) - math.log(300)) <= 1e-5
    keep = torch.tensor([0, 1, 2, 5], device=gpu)
    dl = torch.ones(6, device=gpu)
    args = [t[keep].contiguous() for t in (h, ids, z, lse, logp, dl)]
    dh, dw = M.distill_loss_backward(args[0], w, *args[1:])
    assert bool(dh.isfinite().all()) and bool(dw.isfinite().all())
    assert not bool(dh[0].any())
    # a teacher that is not finite keeps to its own row of dhidden
    dh6, _ = M.distill_loss_backward(h, w, ids, z, lse, logp, dl, dweight=False)
    assert same_bits(dh6[keep], dh)


def test_no_rows_and_no_lists(gpu):
    h = torch.empty(0, 8, dtype=torch.bfloat16, device=gpu)
    w = torch.ones(5, 8, dtype=torch.bfloat16, device=gpu)
    ids = torch.empty(0, 3, dtype=torch.int64, device=gpu)
    z = torch.empty(0, 3, device=gpu)
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z)
    assert loss.numel() == 0 and lse.numel() == 0 and logp.shape == (0, 3)
    dh, dw = M.distill_loss_backward(h, w, ids, z, lse, logp, loss,
                                     dweight=torch.full((5, 8), 3.0, device=gpu))
    assert dh.shape == (0, 8) and not bool(dw.any())
    h = torch.randn(9, 8, device=gpu).to(torch.bfloat16)
    ids = torch.full((9, 3), -1, device=gpu)
    z = torch.full((9, 3), float("nan"), device=gpu)
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z)
    assert not bool(loss.any()) and not bool(logp.any()) and bool(lse.isfinite().all())
    dh, dw = M.distill_loss_backward(h, w, ids, z, lse, logp, loss + float("nan"))
    assert not bool(dh.any()) and not bool(dw.any())


def test_gradients_against_differences(gpu):
    # central differences of the fp32 loss along random directions, as in
    # test_gpu_lm_loss.py: the third cumulant of the logits, over T, along a
    # direction of span R is at most R^3
    n, vocab, dim, top, T = 5, 61, 19, 7, 1.3
    h, w, ids, z, dl = _inputs(gpu, n, vocab, dim, top, "fp32", "fp32")
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z, T)
    dh, dw = M.distill_loss_backward(h, w, ids, z, lse, logp, dl, T)
    ref = Ref(h, w, ids, z, T, dl, "fp32")
    g = torch.Generator(device=gpu)
    g.manual_seed(9)
    eps = 2.0 ** -6
    for which in ("h", "w"):
        for _ in range(3):
            v = torch.randn(h.shape if which == "h" else w.shape, generator=g, device=gpu)
            vals = []
            for s in (1.0, -1.0):
                a = h + s * eps * v if which == "h" else h
                b = (w + s * eps * v).contiguous() if which == "w" else w
                out = M.distill_loss_forward(a, b, ids, z, T)[0]
                vals.append(float((out.double() * dl.double()).sum()))
            slope = (vals[0] - vals[1]) / (2 * eps)
            grad = dh if which == "h" else dw
            dirv = (v.double() @ w.double().t() if which == "h" else h.double() @ v.double().t()) / T
            span = dirv.max(1).values - dirv.min(1).values
            tol = float((dl.double() * (span ** 3 * eps ** 2 / 6 + 2 * ref.loss_bound / eps)).sum())
            tol += float((dl.double() * span).sum()) * 2.0 ** -24 / eps * 8
            assert abs(slope - float((grad.double() * v.double()).sum())) <= tol


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_the_largest_vocabulary(gpu, dt):
    n, vocab, dim, top = 5, 1 << 21, 8, 1024
    h, w, ids, z, _ = _inputs(gpu, n, vocab, dim, top, dt, "fp32")
    ids[0, 0], ids[1, 1], ids[2, 2], ids[3, 3] = vocab - 1, vocab, 0, -1
    dl = torch.rand(n, device=gpu) + 0.5
    ref = Ref(h, w, ids, z, 1.0, dl, dt)
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z)
    assert_within(loss, ref.loss, ref.loss_bound)
    assert_within(logp, ref.logp, ref.logp_bound)
    dh, dw = M.distill_loss_backward(h, w, ids, z, lse, logp, dl)
    assert_within(dh, ref.dh, 1.01 * (ref.dh_err + ref.dh.abs() * HALF[DT[dt]]))
    assert_within(dw, ref.dw, 1.01 * (ref.dw_err + ref.dw.abs() * HALF[DT[dt]]))
