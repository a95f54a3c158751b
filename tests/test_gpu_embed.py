"""Embedding lookup and its gradient against fp64.

Bounds.  Lookup: one fp32 product and one rounding to the storage type.
Gradient: a sum of m terms in fp32, in any order, is off by at most
(m - 1) 2^-24 sum|x| (first order); then one product by the scale, one
addition when accumulating, one rounding to the storage type.  Each bound
below counts those, with 1% for the higher orders."""

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import DT, HALF, assert_within, fill_normal, guarded, same_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _ids(kind, n, vocab, gen, dev, dtype):
    if kind == "same":
        ids = torch.full((n,), vocab // 2, device=dev)
    elif kind == "missing":
        ids = torch.full((n,), -1, device=dev)
    elif kind == "zipf":
        u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64)
        ids = ((vocab + 1.0) ** u).floor().long() - 1
        ids = ids.clamp(0, vocab - 1)
    else:  # outside the table on both sides too
        ids = torch.randint(-vocab // 4 - 1, vocab + vocab // 4 + 1, (n,), generator=gen, device=dev)
        if n > 3:
            ids[0], ids[1], ids[2] = vocab - 1, vocab, 0
            if dtype == torch.int64:
                ids[3] = 1 << 40
    return ids.to(dtype)


@pytest.mark.parametrize("n,vocab,dim,td,od,idt,off,pad", [
    (1, 1, 1, "fp32", "fp32", torch.int32, 0, 0),
    (0, 5, 8, "bf16", "bf16", torch.int64, 0, 0),
    (5, 100, 7, "bf16", "bf16", torch.int64, 1, 3),
    (33, 1000, 256, "bf16", "bf16", torch.int64, 0, 0),
    (257, 1000, 2048, "bf16", "fp32", torch.int32, 0, 8),
    (4, 300, 2051, "fp32", "bf16", torch.int64, 3, 1),
    (1025, 32000, 2048, "bf16", "bf16", torch.int32, 0, 0),
    (130, 500, 7168, "fp32", "fp32", torch.int64, 0, 0),
])
def test_lookup(gpu, n, vocab, dim, td, od, idt, off, pad):
    g = torch.Generator(device=gpu)
    g.manual_seed(n + dim)
    table, _ = guarded((vocab, dim), DT[td], gpu, off)
    fill_normal(table, 1.0, g)
    ids = _ids("uniform", n, vocab, g, gpu, idt)
    out, check = guarded((n, dim), DT[od], gpu, off, dim + pad)
    scale = 45.254834
    assert M.embed_forward(table, ids, scale, out=out) is out
    torch.cuda.synchronize()
    check()
    ok = (ids >= 0) & (ids < vocab)
    want = torch.zeros(n, dim, dtype=torch.float64, device=gpu)
    want[ok] = table[ids[ok].long()].double() * float(torch.tensor(scale, dtype=torch.float32))
    assert_within(out, want, want.abs() * 1.01 * (U + HALF[DT[od]] * (od == "bf16")))
    assert bool((out[~ok] == 0).all())
    again = M.embed_forward(table, ids.view(-1, 1) if n else ids, scale, out_dtype=od)
    assert again.dtype == DT[od] and again.shape[-1] == dim
    assert same_bits(again.reshape(n, dim), out)


def test_lookup_of_non_finite_rows_and_offsets_past_32_bits(gpu):
    # a table of 2^31 + 2^25 elements: the last rows lie past 2^31 elements
    dim = 8192
    vocab = (1 << 31) // dim + 4096
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device=gpu)
    table[vocab - 1] = 3.0
    table[vocab - 2] = float("nan")
    table[0] = float("inf")
    ids = torch.tensor([vocab - 1, vocab - 2, 0, -1, vocab], device=gpu)
    out = M.embed_forward(table, ids, 0.5)
    assert bool((out[0] == 1.5).all()) and bool(out[1].isnan().all())
    assert bool(out[2].isinf().all()) and bool((out[3:] == 0).all())
    # its gradient: rows there are written, and the rest is zeroed
    table.fill_(7.0)
    dout = torch.ones(5, dim, dtype=torch.bfloat16, device=gpu)
    M.embed_backward(dout, ids, table, 0.5)
    assert bool((table[vocab - 1] == 0.5).all()) and bool((table[0] == 0.5).all())
    assert float(table[1:vocab - 2].float().abs().max()) == 0.0


@pytest.mark.parametrize("pad", [0, 64, 8])
@pytest.mark.parametrize("od", ["bf16", "fp32"])
def test_lookup_of_a_large_output(gpu, od, pad):
    # 360 MB and more, in whole lines (pad 8: not, for bf16)
    g = torch.Generator(device=gpu)
    g.manual_seed(pad)
    n, vocab, dim = 24611 if od == "bf16" else 12307, 211, 7360
    table, _ = guarded((vocab, dim), torch.bfloat16, gpu)
    fill_normal(table, 1.0, g)
    ids = _ids("uniform", n, vocab, g, gpu, torch.int64)
    out, check = guarded((n, dim), DT[od], gpu, 0, dim + pad)
    M.embed_forward(table, ids, 0.5, out=out)
    torch.cuda.synchronize()
    check()
    row = torch.where((ids >= 0) & (ids < vocab), ids, torch.full_like(ids, vocab))
    want = torch.cat([table * 0.5, torch.zeros_like(table[:1])])[row].to(DT[od])  # exact
    assert torch.equal(out, want)


def test_lookup_of_the_most_positions(gpu):
    # 2^26 - 1 positions: more than one launch holds
    n, vocab = (1 << 26) - 1, 97
    table = torch.arange(vocab, device=gpu, dtype=torch.bfloat16).view(vocab, 1)
    ids = torch.arange(n, device=gpu, dtype=torch.int32).remainder_(vocab + 1)  # vocab: no row
    out = M.embed_forward(table, ids)
    want = torch.where(ids < vocab, ids, torch.zeros_like(ids)).to(torch.bfloat16)
    assert torch.equal(out.view(n), want)


@pytest.mark.parametrize("n,vocab,dim,dd,gd,idt,kind,acc,off,pad", [
    (0, 40, 9, "bf16", "bf16", torch.int64, "uniform", False, 1, 0),
    (0, 40, 9, "bf16", "bf16", torch.int64, "uniform", True, 1, 0),
    (1, 1, 1, "fp32", "fp32", torch.int32, "same", False, 0, 0),
    (1, 700, 2048, "bf16", "bf16", torch.int64, "same", False, 0, 0),
    (31, 50, 8, "bf16", "fp32", torch.int64, "uniform", False, 0, 0),
    (32, 50, 16, "bf16", "bf16", torch.int32, "same", True, 0, 0),
    (33, 50, 16, "fp32", "fp32", torch.int32, "same", False, 2, 5),
    (64, 3, 40, "bf16", "bf16", torch.int64, "uniform", False, 3, 1),
    (500, 1000, 333, "bf16", "bf16", torch.int64, "missing", False, 1, 0),
    (1000, 77, 2051, "fp32", "bf16", torch.int64, "uniform", True, 1, 7),
    (4096, 32000, 256, "bf16", "bf16", torch.int32, "zipf", False, 0, 0),
    (8192, 33001, 101, "bf16", "fp32", torch.int64, "zipf", False, 0, 0),
    (8193, 33001, 101, "fp32", "fp32", torch.int64, "zipf", True, 0, 3),
    (20000, 512, 64, "bf16", "bf16", torch.int32, "uniform", False, 0, 0),
    (12289, 511, 40, "bf16", "bf16", torch.int64, "uniform", False, 5, 0),
    (30000, 300000, 24, "bf16", "fp32", torch.int64, "uniform", False, 0, 0),
    (1500, 300000, 24, "bf16", "fp32", torch.int64, "uniform", False, 1, 0),
    (2048, 40, 1032, "bf16", "bf16", torch.int32, "zipf", False, 0, 0),
    (2049, 700, 520, "bf16", "bf16", torch.int32, "zipf", True, 0, 0),
    (16384, 32000, 72, "bf16", "bf16", torch.int64, "zipf", False, 0, 0),
    (16385, 163840, 8, "fp32", "bf16", torch.int64, "uniform", False, 0, 0),
    (70000, 1000003, 16, "bf16", "bf16", torch.int64, "zipf", False, 0, 0),
    (9000, 5, 2056, "bf16", "bf16", torch.int64, "same", False, 0, 8),
])
def test_gradient(gpu, n, vocab, dim, dd, gd, idt, kind, acc, off, pad):
    g = torch.Generator(device=gpu)
    g.manual_seed(n + vocab + dim)
    dout, _ = guarded((n, dim), DT[dd], gpu, off, dim + pad)
    fill_normal(dout, 1.0, g)
    ids = _ids(kind, n, vocab, g, gpu, idt)
    grad, check = guarded((vocab, dim), DT[gd], gpu, off)
    if acc:
        fill_normal(grad, 0.5, g)
    else:
        grad.fill_(float("nan"))  # every row is written
    old = grad.clone()
    scale = 3.25
    ws = torch.full((max(1, M.embed_backward_workspace_size(n, vocab, dim)),), 255,
                    dtype=torch.uint8, device=gpu)
    assert M.embed_backward(dout, ids, grad, scale, accumulate=acc, workspace=ws) is grad
    torch.cuda.synchronize()
    check()
    ok = (ids >= 0) & (ids < vocab)
    at = ids[ok].long()
    want = torch.zeros(vocab, dim, dtype=torch.float64, device=gpu)
    size = torch.zeros_like(want)
    count = torch.zeros(vocab, dtype=torch.float64, device=gpu)
    want.index_add_(0, at, dout[ok].double())
    size.index_add_(0, at, dout[ok].double().abs())
    count.index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    bound = scale * U * (size * count[:, None].clamp(min=1) + want.abs())
    want = want * scale + (old.double() if acc else 0.0)
    bound = 1.01 * (bound + want.abs() * (U if acc else 0.0) + want.abs() * HALF[DT[gd]])
    if acc:
        assert same_bits(grad[count == 0], old[count == 0])
    else:
        assert bool((grad[count == 0] == 0).all())
    assert_within(grad, want, bound)
    # the same bits again, in a workspace of its own
    grad2 = old.clone()
    M.embed_backward(dout, ids, grad2, scale, accumulate=acc)
    assert same_bits(grad2, grad.contiguous())


def test_gradient_sums_in_the_order_of_the_positions(gpu):
    # 2^24 + 1 + 1 - 2^24 in fp32 is 0 in this order only (each 1 is lost)
    dim = 8
    vals = [2.0 ** 24, 1.0, 1.0, -2.0 ** 24]
    ids = torch.tensor([3, 1, 3, 3, 1, 3], device=gpu)
    dout = torch.zeros(6, dim, device=gpu)
    for k, t in enumerate([0, 2, 3, 5]):
        dout[t] = vals[k]
    grad = torch.empty(5, dim, device=gpu)
    M.embed_backward(dout, ids, grad)
    assert bool((grad == 0).all())


def test_gradient_is_the_adjoint_of_the_lookup(gpu):
    # <lookup(E), D> = <E, gradient(D)>, both sides summed in fp64
    g = torch.Generator(device=gpu)
    g.manual_seed(5)
    table = torch.randn(300, 96, generator=g, device=gpu)
    ids = torch.randint(-20, 300, (40, 25), generator=g, device=gpu)
    dout = torch.randn(1000, 96, generator=g, device=gpu)
    out = M.embed_forward(table, ids, 2.0)
    assert out.shape == (40, 25, 96)
    grad = torch.empty_like(table)
    M.embed_backward(dout, ids, grad, 2.0)
    a = (out.view(1000, 96).double() * dout.double())
    b = (table.double() * grad.double())
    # every gradient element is off by at most its sum's bound: 1000 terms
    tol = 1000 * U * float(a.abs().sum())
    assert abs(float(a.sum() - b.sum())) <= tol


def test_another_stream(gpu):
    s = torch.cuda.Stream()
    ids = torch.arange(5000, device=gpu) % 37
    dout = torch.ones(5000, 64, device=gpu)
    torch.cuda.synchronize()
    grad = torch.empty(40, 64, device=gpu)
    for how in (s, s.cuda_stream):
        grad.fill_(9.0)
        torch.cuda.synchronize()
        M.embed_backward(dout, ids, grad, stream=how)
        s.synchronize()
        assert float(grad[0, 0]) == 136.0 and float(grad[36, 5]) == 135.0
        assert float(grad[37:].abs().max()) == 0.0
    out = M.embed_forward(grad, ids[:7], stream=s)
    s.synchronize()
    assert torch.equal(out, grad[:7])
