"""The vocabulary loss's gradients: what bf16 calls keep of g.

Bounds as in test_gpu_lm_loss.py, but for g's own rounding in bf16 calls: g
is the sum of two bf16 values, of which the first is off by half a step, 2^-8
of g, and the second by as much of what is left, so 2^-16 of g."""

import pytest
import torch

import muon_newton_schulz_amd as M
from test_gpu_lm_loss import Ref, _inputs
from train_ops_util import DT, HALF, assert_within

pytestmark = pytest.mark.gpu


def _tight(ref, h, w, tgt, dl):
    """Takes the bound of one bf16 value of g out of ref, for that of two."""
    h, w = h.double(), w.double()
    g = torch.exp(h @ w.t() - ref.lse[:, None])
    rows = ref.ok.nonzero()[:, 0]
    g[rows, tgt[rows].long()] -= 1.0
    g = g.abs() * torch.where(ref.ok, dl.double(), torch.zeros_like(ref.lse)).abs()[:, None]
    less = HALF[torch.bfloat16] - 2.0 ** -16
    ref.dh_err = ref.dh_err - less * (g @ w.abs())
    ref.dw_err = ref.dw_err - less * (g.t() @ h.abs())
    return ref


def _dloss(kind, n, g, dev):
    if kind == "common":
        return torch.full((n,), 1.0 / n, device=dev)
    if kind == "random":
        return torch.rand(n, generator=g, device=dev) + 0.5
    dl = torch.full((n,), 0.502, device=dev)  # two values, one of them in a single row
    dl[n // 2] = 1.0
    return dl


@pytest.mark.parametrize("dim", [64, 61])
@pytest.mark.parametrize("od", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["common", "random", "two"])
def test_bf16_gradients_keep_more_of_g_than_bf16(gpu, kind, od, dim):
    # (one bf16 value alone fails in every kind: the other terms of the bound
    # come to less than 2^-11 of a row's largest gradient)
    n, vocab = 300, 500
    h, w, tgt, _ = _inputs(gpu, n, vocab, dim, "bf16", 0, 0, 1)
    g = torch.Generator(device=gpu)
    g.manual_seed(4)
    dl = _dloss(kind, n, g, gpu)
    ref = _tight(Ref(h, w, tgt, dl, "bf16"), h, w, tgt, dl)
    _, lse = M.lm_loss_forward(h, w, tgt)
    dh, dw = M.lm_loss_backward(h, w, tgt, lse, dl,
                                dhidden=torch.empty(n, dim, dtype=DT[od], device=gpu),
                                dweight=torch.empty(vocab, dim, dtype=DT[od], device=gpu))
    assert_within(dh, ref.dh, 1.01 * (ref.dh_err + ref.dh.abs() * HALF[DT[od]]))
    assert_within(dw, ref.dw, 1.01 * (ref.dw_err + ref.dw.abs() * HALF[DT[od]]))
