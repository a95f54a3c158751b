"""Products grouped by expert against fp64, expert by expert.

Bound.  A sum of K products in fp32: products of bf16 are exact in fp32,
those of fp32 are off by 2^-24 each; every one of the K additions is off by
at most one step (2^-23) of a partial sum, which sum|x||w| bounds (matrix
cores need not round to nearest).  Then one rounding to the storage type.
accumulate: one addition more."""

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import DT, HALF, assert_within, fill_normal, guarded, same_bits

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23


def _offsets(kind, rows, experts, gen, dev):
    """Host list of experts + 1 offsets."""
    if kind == "even":
        return [e * rows // experts for e in range(experts + 1)]
    if kind == "one":      # every row to one expert
        k = experts // 2
        return [0] * (k + 1) + [rows] * (experts - k)
    if kind == "gaps":     # rows before the first and behind the last expert
        lo, hi = rows // 5, rows - rows // 4
        cut = torch.randint(lo, hi + 1, (experts - 1,), generator=gen).sort().values.tolist()
        return [lo] + cut + [hi]
    if kind == "none":
        return [0] * (experts + 1)
    cut = torch.randint(0, rows + 1, (experts - 1,), generator=gen).sort().values.tolist()
    return [0] + cut + [rows]


CASES = [
    # rows, experts, k, n, kind, dtype, out, off, pad
    (0, 3, 16, 16, "ragged", "bf16", "bf16", 0, 0),
    (1, 1, 1, 1, "even", "fp32", "fp32", 0, 0),
    (1, 4, 64, 128, "one", "bf16", "bf16", 0, 0),
    (8, 64, 256, 176, "ragged", "bf16", "bf16", 0, 0),
    (37, 5, 33, 65, "ragged", "bf16", "bf16", 1, 3),
    (200, 3, 100, 130, "ragged", "fp32", "fp32", 3, 1),
    (129, 2, 127, 129, "one", "fp32", "bf16", 0, 0),
    (300, 4, 256, 256, "even", "bf16", "fp32", 0, 8),
    (513, 3, 264, 520, "gaps", "bf16", "bf16", 0, 0),
    (700, 70, 64, 72, "ragged", "bf16", "bf16", 0, 0),
    (1000, 200, 40, 48, "ragged", "bf16", "bf16", 0, 16),
    (1500, 7, 1001, 703, "gaps", "bf16", "bf16", 1, 0),
    (1024, 4, 512, 768, "ragged", "bf16", "bf16", 0, 0),
    (2000, 3, 96, 264, "ragged", "bf16", "bf16", 0, 24),
    (50, 6, 8, 8, "none", "bf16", "bf16", 0, 0),
    (4096, 2, 160, 320, "one", "bf16", "fp32", 0, 0),
    (260, 4096, 16, 24, "ragged", "bf16", "bf16", 0, 0),
    (777, 4, 200, 136, "gaps", "fp32", "fp32", 0, 4),
]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("rows,experts,k,n,kind,dt,od,off,pad", CASES)
def test_matmul(gpu, rows, experts, k, n, kind, dt, od, off, pad, trans):
    g = torch.Generator(device=gpu)
    g.manual_seed(rows + k + n)
    host = torch.Generator()
    host.manual_seed(rows)
    offs = _offsets(kind, rows, experts, host, gpu)
    x, _ = guarded((rows, k), DT[dt], gpu, off, k + pad)
    fill_normal(x, 1.0, g)
    wf, _ = guarded((1, experts * k * n), DT[dt], gpu, off)
    fill_normal(wf, 0.05, g)
    w = wf.view((experts, n, k) if trans else (experts, k, n))
    y, check = guarded((rows, n), DT[od], gpu, off, n + pad)
    y.fill_(5.0)
    o = torch.tensor(offs, dtype=torch.int32, device=gpu)
    assert M.expert_matmul(x, w, o, trans=trans, out=y) is y
    torch.cuda.synchronize()
    check()
    want = torch.full((rows, n), 5.0, dtype=torch.float64, device=gpu)
    size = torch.zeros_like(want)
    for e in range(experts):
        lo, hi = offs[e], offs[e + 1]
        if lo < hi:
            we = w[e].double().t() if trans else w[e].double()
            want[lo:hi] = x[lo:hi].double() @ we
            size[lo:hi] = x[lo:hi].double().abs() @ we.abs()
    bound = 1.01 * (size * (k + 1) * STEP + want.abs() * HALF[DT[od]] * (size > 0))
    assert_within(y, want, bound)
    got = M.expert_matmul(x, w, o, trans=trans, out_dtype=od)
    lo, hi = offs[0], offs[-1]
    assert same_bits(got[lo:hi], y[lo:hi])
    assert not bool(got[:lo].any()) and not bool(got[hi:].any())


@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("rows,experts,k,n,kind,dt,od,off,pad", CASES)
def test_wgrad(gpu, rows, experts, k, n, kind, dt, od, off, pad, acc):
    g = torch.Generator(device=gpu)
    g.manual_seed(rows + k + n)
    host = torch.Generator()
    host.manual_seed(rows)
    offs = _offsets(kind, rows, experts, host, gpu)
    a, _ = guarded((rows, k), DT[dt], gpu, off, k + pad)
    b, _ = guarded((rows, n), DT[dt], gpu, off, n + pad)
    fill_normal(a, 1.0, g)
    fill_normal(b, 1.0, g)
    df, check = guarded((1, experts * k * n), DT[od], gpu, off)
    if acc:
        fill_normal(df, 1.0, g)
    else:
        df.fill_(float("nan"))
    dw = df.view(experts, k, n)
    old = dw.clone()
    o = torch.tensor(offs, dtype=torch.int32, device=gpu)
    assert M.expert_wgrad(a, b, o, dw, accumulate=acc) is dw
    torch.cuda.synchronize()
    check()
    for e in range(experts):
        lo, hi = offs[e], offs[e + 1]
        if lo >= hi:
            if e < 50 or e > experts - 50:
                assert same_bits(dw[e], old[e]) if acc else not bool(dw[e].any())
            continue
        want = a[lo:hi].double().t() @ b[lo:hi].double()
        size = a[lo:hi].double().abs().t() @ b[lo:hi].double().abs()
        bound = size * (hi - lo + 1) * STEP
        if acc:
            want = want + old[e].double()
            bound = bound + (size + old[e].double().abs()) * STEP
        assert_within(dw[e], want, 1.01 * (bound + want.abs() * HALF[DT[od]]))
    again = old.clone()
    M.expert_wgrad(a, b, o, again, accumulate=acc)
    assert same_bits(again, dw)


@pytest.mark.parametrize("acc", [False, True])
def test_wgrad_of_large_gradients(gpu, acc):
    # 134 MB, rows that are no whole lines
    test_wgrad(gpu, 400, 16, 2040, 2056, "gaps", "bf16", "bf16", 0, 0, acc)


def test_offsets_out_of_order_stay_in_bounds(gpu):
    # clamped to [0, rows]; a range that is not positive holds no rows
    x = torch.ones(40, 64, dtype=torch.bfloat16, device=gpu)
    w = torch.ones(5, 64, 32, dtype=torch.bfloat16, device=gpu)
    y = torch.full((40, 32), 3.0, dtype=torch.bfloat16, device=gpu)
    o = torch.tensor([-7, 10, 5, 20, 1000, 2], dtype=torch.int32, device=gpu)
    M.expert_matmul(x, w, o, out=y)          # rows 0-9, none, 5-19, 20-39, none
    assert bool((y == 64).all())
    dw = torch.empty(5, 64, 32, device=gpu)
    M.expert_wgrad(x, y, o, dw)
    assert [float(dw[e, 0, 0]) for e in range(5)] == [640.0, 0.0, 960.0, 1280.0, 0.0]


def test_non_finite_rows_stay_their_own(gpu):
    # a NaN row and an infinite weight reach their own results only
    x = torch.ones(300, 72, dtype=torch.bfloat16, device=gpu)
    x[130] = float("nan")
    w = torch.ones(3, 72, 40, dtype=torch.bfloat16, device=gpu)
    w[2, 5, 7] = float("inf")
    o = torch.tensor([0, 131, 131, 300], dtype=torch.int32, device=gpu)
    y = M.expert_matmul(x, w, o)
    assert bool(y[130].isnan().all()) and bool((y[:130] == 72).all())
    assert bool(y[131:, 7].isinf().all())
    y[:, 7] = 72
    assert bool((y[131:] == 72).all())
    # rows of another expert beside the range do not leak into a sum
    dw = torch.empty(3, 72, 72, device=gpu)
    o = torch.tensor([0, 130, 130, 130], dtype=torch.int32, device=gpu)
    M.expert_wgrad(x, x, o, dw)
    assert bool((dw[0] == 130).all()) and not bool(dw[1:].any())


def test_gradients_are_the_adjoints_of_the_product(gpu):
    # <y, dy> = <x, dx> = <w, dw>, and dw agrees with a difference of <y, dy>,
    # which is linear in w
    g = torch.Generator(device=gpu)
    g.manual_seed(3)
    x = torch.randn(90, 48, generator=g, device=gpu)
    w = torch.randn(4, 48, 36, generator=g, device=gpu)
    dy = torch.randn(90, 36, generator=g, device=gpu)
    o = torch.tensor([0, 20, 20, 70, 90], dtype=torch.int32, device=gpu)
    y = M.expert_matmul(x, w, o)
    dx = M.expert_matmul(dy, w, o, trans=True)
    dw = M.expert_wgrad(x, dy, o, torch.empty_like(w))
    a, b, c = ((p.double() * q.double()) for p, q in ((y, dy), (x, dx), (w, dw)))
    tol = 100 * STEP * float(a.abs().sum() + b.abs().sum() + c.abs().sum())
    assert abs(float(a.sum() - b.sum())) <= tol and abs(float(a.sum() - c.sum())) <= tol
    w2 = w.clone()
    w2[2, 5, 6] += 1.0
    y2 = M.expert_matmul(x, w2, o)
    diff = float(((y2.double() - y.double()) * dy.double()).sum())
    assert abs(diff - float(dw[2, 5, 6])) <= tol


@pytest.mark.parametrize("k", [40, 264])
def test_fp32_values_at_the_ends_of_the_range(gpu, k):
    # not finite; the largest fp32 (whose nearest bf16 is infinite); results
    # that overflow; operands near the smallest normal
    x = torch.ones(200, k, device=gpu)
    w = torch.ones(2, k, 70, device=gpu)
    big = float(torch.finfo(torch.float32).max)
    x[3] = float("nan")
    x[5, 1] = float("inf")
    x[7] = 0.0
    x[7, 2] = big
    x[9] = big
    x[150] = 2.0 ** -120
    w[1, :, 69] = 2.0 ** -60
    o = torch.tensor([0, 100, 200], dtype=torch.int32, device=gpu)
    y = M.expert_matmul(x, w, o)
    assert bool(y[3].isnan().all()) and bool((y[5] == float("inf")).all())
    assert bool((y[7] == big).all()) and bool((y[9] == float("inf")).all())
    rest = [r for r in range(100) if r not in (3, 5, 7, 9)]
    assert bool((y[rest] == k).all())
    assert bool((y[150, :69] == k * 2.0 ** -120).all())
    assert bool((y[151:, 69] == k * 2.0 ** -60).all())


def test_fp32_products_keep_fp32_accuracy(gpu):
    # operands whose bits reach from the first to the last place: a product
    # of two loses at most 2^-24, the sum of k as the bound at the top says,
    # and without cancellation (all positive) that is relative to the result
    g = torch.Generator(device=gpu)
    g.manual_seed(8)
    k = 300
    x = 1.0 + torch.rand(130, k, generator=g, device=gpu)
    w = 1.0 + torch.rand(1, k, 90, generator=g, device=gpu)
    o = torch.tensor([0, 130], dtype=torch.int32, device=gpu)
    want = x.double() @ w[0].double()
    y = M.expert_matmul(x, w, o)
    # sums of 256 restart; a random walk of their roundings stays far below
    # the worst case, 2^-24 sqrt(256) with a factor 4 for the largest of 11700
    assert float(((y.double() - want) / want).abs().max()) <= 4 * 16 * 2.0 ** -24
