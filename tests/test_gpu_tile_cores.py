"""Every tile core of the loss and of the expert products in its steady state,
against fp64 (the bounds of test_gpu_experts.py and test_gpu_lm_loss*.py).

bf16 gradients of the loss are also compared by norm, where sums of many terms
leave the bound of single elements wide: an element is off by half a step, 2^-8,
and by what the fp32 sums lose, a random walk of sqrt(20011) steps of 2^-23 times
the at most tenfold size of their terms, below 2^-10."""

import pytest
import torch

import muon_newton_schulz_amd as M
from test_gpu_experts import test_matmul as check_matmul
from test_gpu_experts import test_wgrad as check_wgrad
from test_gpu_lm_loss import Ref, _inputs
from test_gpu_lm_loss_gradients import _tight
from tile_core_cases import EXPERTS, LOSS
from train_ops_util import DT, HALF, assert_within, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout,rows,experts,k,n,kind,dt,off", EXPERTS)
def test_expert_products(gpu, layout, rows, experts, k, n, kind, dt, off):
    if layout == "TN":
        check_wgrad(gpu, rows, experts, k, n, kind, dt, dt, off, 0, False)
    else:
        check_matmul(gpu, rows, experts, k, n, kind, dt, dt, off, 0, layout == "NT")


@pytest.mark.parametrize("n,vocab,dim,dt,off", LOSS)
def test_loss(gpu, n, vocab, dim, dt, off):
    h, w, tgt, dl = _inputs(gpu, n, vocab, dim, dt, off, 0, 1)
    ref = Ref(h, w, tgt, dl, dt)
    if dt == "bf16":
        _tight(ref, h, w, tgt, dl.nan_to_num())
    loss, lse = M.lm_loss_forward(h, w, tgt)
    assert_within(lse, ref.lse, ref.lse_bound)
    assert_within(loss, ref.loss, ref.loss_bound)
    dh, dw = M.lm_loss_backward(h, w, tgt, lse, dl)
    assert_within(dh, ref.dh, 1.01 * (ref.dh_err + ref.dh.abs() * HALF[DT[dt]]))
    assert_within(dw, ref.dw, 1.01 * (ref.dw_err + ref.dw.abs() * HALF[DT[dt]]))
    if dt == "bf16":
        for got, want in ((dh, ref.dh), (dw, ref.dw)):
            assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -8 + 2.0 ** -10
    again = M.lm_loss_backward(h, w, tgt, lse, dl)
    assert same_bits(again[0], dh) and same_bits(again[1], dw)
