"""fp32 products whose operands are too small for three bf16 values to hold:
below 2^-107 the parts of a split fall under bf16's smallest value, 2^-133.

Bound as in test_gpu_experts.py, and k steps of fp32's smallest value, 2^-149,
for products below the normal range.  All operands have full mantissas."""

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import assert_within, same_bits

pytestmark = pytest.mark.gpu

STEP, HALF32, TINY = 2.0 ** -23, 2.0 ** -24, 2.0 ** -149

# 64 x 64 tiles, and enough of them for 128 x 128
SIZES = [(200, 2, 40, 70), (130, 1, 300, 90), (4096, 1, 200, 2048)]


def _full(shape, g, dev):
    sign = torch.randint(0, 2, shape, generator=g, device=dev) * 2 - 1
    return (1.0 + torch.rand(shape, generator=g, device=dev)) * sign


def _small_rows(t, every, exponent):
    t[::every] = torch.ldexp(t[::every], torch.tensor(exponent, device=t.device))


@pytest.mark.parametrize("exponent", [-108, -112, -120, -126, -132])
@pytest.mark.parametrize("rows,experts,k,n", SIZES)
@pytest.mark.parametrize("trans", [False, True])
def test_products_of_small_rows(gpu, rows, experts, k, n, exponent, trans):
    g = torch.Generator(device=gpu)
    g.manual_seed(rows + k - exponent)
    x, w = _full((rows, k), g, gpu), _full((experts, k, n), g, gpu)
    offs = [e * rows // experts for e in range(experts + 1)]
    o = torch.tensor(offs, dtype=torch.int32, device=gpu)
    wt = w.transpose(1, 2).contiguous() if trans else w
    before = M.expert_matmul(x, wt, o, trans=trans)
    _small_rows(x, 7, exponent)      # whole rows
    x[3, k // 2] *= 2.0 ** -120      # one small value in a row of others
    y = M.expert_matmul(x, wt, o, trans=trans)
    for e in range(experts):
        a, b = x[offs[e]:offs[e + 1]].double(), w[e].double()
        want, size = a @ b, a.abs() @ b.abs()
        assert_within(y[offs[e]:offs[e + 1]], want,
                      1.01 * (size * (k + 1) * STEP + want.abs() * HALF32) + k * TINY)
    # the rows beside them keep their bits
    rest = [r for r in range(rows) if r % 7 and r != 3]
    assert same_bits(y[rest], before[rest])


@pytest.mark.parametrize("exponent", [-112, -120, -126])
@pytest.mark.parametrize("rows,experts,k,n", SIZES)
def test_products_of_small_weights(gpu, rows, experts, k, n, exponent):
    g = torch.Generator(device=gpu)
    g.manual_seed(rows + n - exponent)
    x, w = _full((rows, k), g, gpu), _full((experts, k, n), g, gpu)
    o = torch.tensor([e * rows // experts for e in range(experts + 1)], dtype=torch.int32,
                     device=gpu)
    wt = w.transpose(1, 2)
    wt[:, ::5] = torch.ldexp(wt[:, ::5], torch.tensor(exponent, device=gpu))
    y = M.expert_matmul(x, w, o)
    y2 = M.expert_matmul(x, wt.contiguous(), o, trans=True)
    for e in range(experts):
        a, b = x[int(o[e]):int(o[e + 1])].double(), w[e].double()
        want, size = a @ b, a.abs() @ b.abs()
        bound = 1.01 * (size * (k + 1) * STEP + want.abs() * HALF32) + k * TINY
        assert_within(y[int(o[e]):int(o[e + 1])], want, bound)
        assert_within(y2[int(o[e]):int(o[e + 1])], want, bound)


@pytest.mark.parametrize("exponent", [-112, -120, -126])
@pytest.mark.parametrize("rows,m,n", [(40, 70, 200), (300, 130, 90), (200, 4096, 2048)])
def test_weight_gradients_of_small_columns(gpu, rows, m, n, exponent):
    g = torch.Generator(device=gpu)
    g.manual_seed(rows + n - exponent)
    a, b = _full((rows, m), g, gpu), _full((rows, n), g, gpu)
    _small_rows(a.t(), 9, exponent)
    _small_rows(b.t(), 11, exponent + 60)   # not small: exact parts, results that are
    o = torch.tensor([0, rows], dtype=torch.int32, device=gpu)
    dw = M.expert_wgrad(a, b, o, torch.empty(1, m, n, device=gpu))
    want, size = a.double().t() @ b.double(), a.double().abs().t() @ b.double().abs()
    assert_within(dw[0], want,
                  1.01 * (size * (rows + 1) * STEP + want.abs() * HALF32) + rows * TINY)


def test_loss_gradients_of_unlikely_words(gpu):
    # a word that is e^-75 = 2^-108 to e^-85 = 2^-123 likely in every row: its row of
    # dweight is as accurate as the others'.  g is off by p (r + d + e), the
    # logits' and exp's errors (as in test_gpu_lm_loss.py).
    n, vocab, dim = 60, 200, 40
    g = torch.Generator(device=gpu)
    g.manual_seed(6)
    h = _full((n, dim), g, gpu) * 0.1
    w = _full((vocab, dim), g, gpu) * 0.1
    h[:, 0] = 1.0
    w[17, 0], w[99, 0] = -72.0, -80.0
    tgt = torch.randint(0, 17, (n,), generator=g, device=gpu)
    dl = torch.rand(n, generator=g, device=gpu) + 0.5
    _, lse = M.lm_loss_forward(h, w, tgt)
    _, dw = M.lm_loss_backward(h, w, tgt, lse, dl, dhidden=False)
    logits = h.double() @ w.double().t()
    p = torch.exp(logits - torch.logsumexp(logits, 1)[:, None])
    rows = [17, 99]
    assert float(p[:, rows].max()) < 2.0 ** -107
    size = h.double().abs() @ w.double().abs().t()
    d = (dim + 1) * STEP * size
    # r: the row's lse is off by its largest d among the words that count, and roundings
    r = (dim + 1) * STEP * size[:, [v for v in range(vocab) if v not in rows]].max(1).values
    err = p * (d + (r + 2.0 ** -19)[:, None]) * dl.double()[:, None]
    gr = (p * dl.double()[:, None])[:, rows]
    want = gr.t() @ h.double()
    bound = (err[:, rows].t() @ h.double().abs()
             + (n + 1) * STEP * (gr.abs().t() @ h.double().abs()) + want.abs() * HALF32)
    assert_within(dw[rows], want, 1.01 * bound + n * TINY)
