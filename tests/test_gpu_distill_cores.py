"""The distillation loss and its gradients on the tile cores of
distill_core_cases.py, against fp64 with the bounds of test_gpu_distill.py."""

import pytest
import torch

import muon_newton_schulz_amd as M
from distill_core_cases import CORES
from test_gpu_distill import HALF, Ref, _inputs
from train_ops_util import DT, assert_within, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,vocab,dim,top,dt,off,wide", CORES)
def test_tile_cores(gpu, n, vocab, dim, top, dt, off, wide):
    h, w, ids, z, dl = _inputs(gpu, n, vocab, dim, top, dt, "fp32", off)
    ref = Ref(h, w, ids, z, 1.5, dl.nan_to_num(), dt)
    loss, lse, logp = M.distill_loss_forward(h, w, ids, z, 1.5)
    assert_within(lse, ref.lse, ref.lse_bound)
    assert_within(logp, ref.logp, ref.logp_bound)
    assert_within(loss, ref.loss, ref.loss_bound)
    t = torch.float32 if wide else DT[dt]
    dh = torch.empty(n, dim, dtype=t, device=gpu)
    dw = torch.empty(vocab, dim, dtype=t, device=gpu)
    M.distill_loss_backward(h, w, ids, z, lse, logp, dl, 1.5, dhidden=dh, dweight=dw)
    assert_within(dh, ref.dh, 1.01 * (ref.dh_err + ref.dh.abs() * HALF[t]))
    assert_within(dw, ref.dw, 1.01 * (ref.dw_err + ref.dw.abs() * HALF[t]))
    again, _ = M.distill_loss_backward(h, w, ids, z, lse, logp, dl, 1.5,
                                       dhidden=torch.empty_like(dh), dweight=False)
    assert same_bits(again, dh)
