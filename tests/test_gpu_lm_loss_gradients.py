"""The vocabulary loss's gradients: what bf16 calls keep of g, and rows
without a target.

Bounds as in test_gpu_lm_loss.py, but for g's own rounding in bf16 calls: g
is the sum of two bf16 values, of which the first is off by half a step, 2^-8
of g, and the second by as much of what is left, so 2^-16 of g."""

import pytest
import torch

import muon_newton_schulz_amd as M
from test_gpu_lm_loss import Ref, _inputs
from train_ops_util import DT, HALF, assert_within, same_bits

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


@pytest.mark.parametrize("dt,n,vocab,dim", [("bf16", 70, 400, 64), ("bf16", 70, 400, 61),
                                            ("fp32", 70, 400, 61), ("bf16", 600, 2000, 1024),
                                            ("fp32", 600, 2000, 1024)])
def test_what_ignored_rows_hold_reaches_no_gradient(gpu, dt, n, vocab, dim):
    h, w, tgt, dl = _inputs(gpu, n, vocab, dim, dt, 0, 3, 1)
    gone = ~((tgt >= 0) & (tgt < vocab))
    assert 3 < int(gone.sum()) < n
    _, lse = M.lm_loss_forward(h, w, tgt)
    dh, dw = M.lm_loss_backward(h, w, tgt, lse, dl)
    assert bool(dw.isfinite().all()) and not bool(dh[gone].any())
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device=gpu)
    at = gone.nonzero()[:, 0]
    held = h[at]
    h[at] = bad[torch.arange(at.numel(), device=gpu) % 3].to(h.dtype)[:, None].expand(-1, dim)
    loss2, lse2 = M.lm_loss_forward(h, w, tgt)
    assert same_bits(lse2[~gone], lse[~gone]) and not bool(loss2[gone].any())
    dh2, dw2 = M.lm_loss_backward(h, w, tgt, lse2, dl)
    assert same_bits(dw2, dw) and same_bits(dh2, dh)
    h[at] = held
    # a weight that is not finite: no gradient for those rows still
    w[vocab // 2, dim // 2] = float("inf")
    w[vocab - 1] = float("nan")
    _, lse3 = M.lm_loss_forward(h, w, tgt)
    dh3, _ = M.lm_loss_backward(h, w, tgt, lse3, dl, dweight=False)
    assert not bool(dh3[gone].any())
