"""Values of the losses over packed sequences where a shortcut shows: a NaN
beside an advantage of 0, sums that cancel, slopes far from and next to a
border.

U = 2^-24, half a step of fp32; bounds stand at the tests."""

import math

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import assert_within, same_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _offsets(gpu, *values):
    return torch.tensor(values, dtype=torch.int32, device=gpu)


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("which", ["nll", "old"])
def test_nan_beside_an_advantage_of_zero(gpu, which, per_token):
    # r A is NaN where r is, whatever A; an infinite ratio counts nothing at A = 0
    n, off = 1300, _offsets(gpu, 0, 300, 700, 1300)
    t = {"nll": torch.rand(n, device=gpu), "old": torch.rand(n, device=gpu)}
    t[which][310] = math.nan
    t["old"][900] = math.inf
    adv = torch.zeros(n if per_token else 3, device=gpu)
    loss, _, count, _ = M.policy_loss_forward(t["nll"], t["old"], adv, off, per_token=per_token)
    assert loss.isnan().tolist() == [False, True, False]
    assert float(loss[0]) == 0.0 and float(loss[2]) == 0.0
    dn = M.policy_loss_backward(t["nll"], t["old"], adv, off, count, torch.ones(3, device=gpu),
                                per_token=per_token)
    assert dn.isnan().nonzero()[:, 0].tolist() == [310]
    dn[310] = 0.0
    assert not bool(dn.any())
    # a masked NaN is not used
    mask = torch.ones(n, dtype=torch.bool, device=gpu)
    mask[310] = False
    loss, _, count, _ = M.policy_loss_forward(t["nll"], t["old"], adv, off, mask=mask,
                                              per_token=per_token)
    assert not bool(loss.any())
    dn = M.policy_loss_backward(t["nll"], t["old"], adv, off, count, torch.ones(3, device=gpu),
                                mask=mask, per_token=per_token)
    assert not bool(dn.any())


@pytest.mark.parametrize("cuts", [(0, 3000), (0, 5, 6, 517, 1029, 1030, 1040, 2900, 3000),
                                  (0, 0, 3, 3, 2000, 2000, 20000), (1, 9, 300000)])
def test_sums_of_terms_that_cancel(gpu, cuts):
    # A ratio of 1 and advantages of 2^24, 1, -2^24 and 1 in turns: a term is
    # -A, and any fp32 sum of the first two loses the second.  All sums are
    # whole numbers below 2^53, so the results are exact, rounded once.
    off = _offsets(gpu, *cuts)
    n = cuts[-1] + 3
    nll = torch.rand(n, device=gpu)
    adv = torch.tensor([2.0 ** 24, 1.0, -2.0 ** 24, 1.0], device=gpu).repeat(n // 4 + 1)[:n]
    ends = torch.cat([adv.new_zeros(1).double(), adv.double().cumsum(0)])[off.long()]
    want = -(ends[1:] - ends[:-1]).float()
    loss, _, _, _ = M.policy_loss_forward(nll, nll, adv, off, per_token=True, mean=False)
    assert torch.equal(loss, want)


@pytest.mark.parametrize("smoothing", [0.0, 1.0, 0.25, 0.5])
def test_logistic_slopes_far_from_zero(gpu, smoothing):
    # f'(x) = e s(x) - (1 - e) s(-x), s(x) = 1 / (1 + exp(-x)), at margins given
    # to the backward as they are.  Each s is off by exp's 2^-22 and 4 roundings
    # of itself, each product by one more, the sum by U; then two factors of 1
    # and their roundings, 2 U.
    x = torch.cat([torch.linspace(-80, 80, 1601), torch.tensor([-17.0, -1e30, 1e30, 0.0])])
    x = x.float().to(gpu)
    pairs = x.numel()
    off = torch.arange(2 * pairs + 1, dtype=torch.int32, device=gpu)
    count = torch.ones(2 * pairs, dtype=torch.int32, device=gpu)
    dn = M.preference_loss_backward(off, x, count, torch.ones(pairs, device=gpu), n=2 * pairs,
                                    beta=1.0, smoothing=smoothing)
    up, down = smoothing * torch.sigmoid(x.double()), (1 - smoothing) * torch.sigmoid(-x.double())
    want = up - down
    err = 1.01 * ((2.0 ** -22 + 6 * U) * (up + down) + 3 * U * want.abs()) + 2.0 ** -140
    assert_within(dn[0::2], -want, err)
    assert_within(dn[1::2], want, err)


def test_hinge_next_to_its_border(gpu):
    # x = 1 - 2^-k and 1 + 2^-k, exact in fp64: a pair with a loss has a slope
    ks = [22, 23, 24, 25, 26, 30, 40, 50]
    gaps = [2.0 ** -k for k in ks] + [0.0] + [-2.0 ** -k for k in ks]
    pairs = len(gaps)
    ref = torch.tensor([v for g in gaps for v in (1.0, g)], device=gpu)
    nll = torch.zeros(2 * pairs, device=gpu)
    off = torch.arange(2 * pairs + 1, dtype=torch.int32, device=gpu)
    want = 1.0 - torch.tensor(gaps, dtype=torch.float64, device=gpu)
    for kind in ("hinge", "squared", "logistic"):
        loss, x, _, count = M.preference_loss_forward(nll, off, ref_nll=ref, beta=1.0, kind=kind)
        if kind != "hinge":
            assert torch.equal(x, want.float())
            continue
        # the margin moves by less than a step
        assert torch.equal(x < 1, want < 1) and bool(((x.double() - want).abs() < 2.0 ** -23).all())
        assert torch.equal(loss, (1 - want).clamp(min=0).float())
        dn = M.preference_loss_backward(off, x, count, torch.ones(pairs, device=gpu), kind=kind,
                                        n=2 * pairs, beta=1.0)
        slope = (want < 1).float()
        assert torch.equal(dn[0::2], slope) and torch.equal(dn[1::2], -slope)
