"""The loss of targets that are nearly certain, against fp64.

The logits are exact here (one product of powers of two and small integers
each), so the loss (m - l_y) + log sum exp(l - m) is off by the sum's and the
logarithm's roundings only: each term by 2^-19 (exp), the sum by its additions,
64 + vocab / 64 halves of a step of 2^-23, relative to a sum that is 1 at
least, and the logarithm and the last addition by two steps of the loss."""

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import DT, assert_within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("top", [0.0, 16.0, 1024.0, 8192.0])
@pytest.mark.parametrize("n", [5, 700])
def test_small_losses_of_large_logits(gpu, dt, top, n):
    vocab, dim = 300, 16
    h = torch.zeros(n, dim, dtype=DT[dt], device=gpu)
    w = torch.zeros(vocab, dim, dtype=DT[dt], device=gpu)
    h[:, 0] = 1.0
    h[:, 1] = (torch.arange(n, device=gpu) % 5 + 4).to(DT[dt])     # gap of 4 to 8, in ...
    w[:, 0] = top
    w[:, 1] = -2.0                                                  # ... logits 2 apart
    tgt = torch.arange(n, device=gpu) % vocab
    tgt[::2] = 7
    w[7, 1] = 0.0
    loss, lse = M.lm_loss_forward(h, w, tgt)
    logits = h.double() @ w.double().t()
    m = logits.max(1).values
    terms = torch.exp(logits - m[:, None]).sum(1)
    want = (m - logits.gather(1, tgt[:, None])[:, 0]) + torch.log(terms)
    assert float(want.min()) < 0.11
    bound = (2.0 ** -19 * (terms - 1) + (64 + vocab / 64) * U * terms) / terms + 4 * U * want
    assert_within(loss, want, 1.01 * bound)
