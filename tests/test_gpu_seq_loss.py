"""The losses over packed sequences and their gradients against fp64.

Bounds, with U = 2^-24 (half a step of fp32).  A term's ratio r = exp(d) is off
by d's rounding, U |d|, and exp's 2^-22, relative to itself, and two roundings
of r A; k = e^x - 1 - x and e^x - 1 by x's rounding, U |x| e^x, 8 U of
themselves below |x| = 1/2, and 2^-22 e^x + 2 U of themselves above.  The
policy loss's terms round twice more and are added in fp32 by eights, in at most
seven additions (each off by U of what it adds up), and those in fp64, so a
sequence's value is off by its terms' errors, 9 U of the sum of their sizes
and one rounding of the result; the preference loss's terms are exact but for fp64's
roundings, and its results are rounded once (x before f' in the backward, where
it is off by U |x|, f' by 2^-21 and 4 roundings)."""

import math

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import assert_within, same_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _lengths(kind, seqs, total, rng):
    """Lengths that sum to total."""
    if kind == "even":
        n = [total // seqs] * seqs
        n[-1] += total - sum(n)
        return n
    if kind == "ones":
        assert total == seqs
        return [1] * seqs
    if kind == "gaps":  # a third empty, runs of them, the first and last too
        w = torch.rand(seqs, generator=rng)
        w[torch.rand(seqs, generator=rng) < 0.33] = 0.0
        w[0] = w[-1] = 0.0
        w[seqs // 2] = 1.0
    elif kind == "one":  # all in one sequence, the others empty
        w = torch.zeros(seqs)
        w[seqs // 3] = 1.0
    else:
        w = torch.exp(torch.randn(seqs, generator=rng))
    n = (w / w.sum() * total).long()
    n[int(w.argmax())] += total - int(n.sum())
    return n.tolist()


def _pack(gpu, kind, seqs, inside, lead, tail, seed, masked):
    rng = torch.Generator()
    rng.manual_seed(seed)
    n = lead + inside + tail
    off = [lead]
    for c in _lengths(kind, seqs, inside, rng):
        off.append(off[-1] + c)
    offsets = torch.tensor(off, dtype=torch.int32, device=gpu)
    g = torch.Generator(device=gpu)
    g.manual_seed(seed)
    r = lambda std=1.0: torch.randn(n, generator=g, device=gpu) * std  # noqa: E731
    nll = torch.rand(n, generator=g, device=gpu).clamp(min=1e-6).log().square()
    old, ref = (nll + r(0.3)).clamp(min=0), (nll + r(0.4)).clamp(min=0)
    mask = None
    if masked:
        mask = torch.rand(n, generator=g, device=gpu) < 0.6
        if seqs > 3:
            mask[off[2]:off[3]] = False          # a sequence in which nothing counts
        bad = torch.tensor([math.nan, math.inf, -math.inf], device=gpu)
        for t in (nll, old, ref):
            at = (~mask).nonzero()[:, 0]
            t[at] = bad[torch.arange(at.numel(), device=gpu) % 3]
    for t in (nll, old, ref):                    # tokens of no sequence
        t[:lead] = math.nan
        t[off[-1]:] = math.inf
    return n, off, offsets, nll, old, ref, mask, g


def _seq(off, n, mask, dev):
    o = torch.tensor(off, device=dev)
    s = torch.searchsorted(o, torch.arange(n, device=dev), right=True) - 1
    inside = (s >= 0) & (s < len(off) - 1)
    counts = inside if mask is None else inside & mask
    return s.clamp(0, len(off) - 2), inside, counts


def _by(values, s, count):
    return torch.zeros(count, dtype=torch.float64, device=values.device).index_add_(0, s, values)


CASES = [
    # kind, sequences, tokens in them, before, behind
    ("even", 1, 1, 0, 0),
    ("ones", 1000, 1000, 3, 5),
    ("even", 7, 511, 0, 1),
    ("even", 2, 512, 0, 0),
    ("even", 4, 2048, 512, 512),
    ("ragged", 13, 1537, 9, 0),
    ("gaps", 300, 5000, 1, 700),
    ("ragged", 30, 8192, 0, 0),         # the most tokens of one workgroup, and one more
    ("ragged", 30, 8192, 1, 0),
    ("gaps", 1024, 7000, 0, 5),         # the most sequences, and one more
    ("gaps", 1025, 7000, 0, 5),
    ("one", 900, 40001, 0, 3),
    ("ragged", 5000, 70000, 0, 0),
    ("gaps", 5000, 3000, 2, 2),
    ("ragged", 40, 5000011, 513, 77),   # spans of several tiles
    ("ragged", 30000, 4400000, 0, 9),
]


def _policy_ref(off, n, nll, old, ref, mask, adv, per_token, lo, hi, w, mean, dloss):
    s, inside, counts = _seq(off, n, mask, nll.device)
    seqs = len(off) - 1
    z = torch.zeros(n, dtype=torch.float64, device=nll.device)
    pick = lambda t: torch.where(counts, t.double(), z)  # noqa: E731
    nll64, old64, ref64 = pick(nll), pick(old), pick(ref) if ref is not None else None
    a = pick(adv if per_token else adv[s])
    d = old64 - nll64
    r = d.exp()
    cut = counts & (((a > 0) & (r > 1 + hi)) | ((a < 0) & (r < 1 - lo)))
    edge = torch.where(a > 0, torch.full_like(a, 1 + hi), torch.full_like(a, 1 - lo))
    token, slope = -torch.where(cut, edge, r) * a, torch.where(cut, z, r * a)
    err = torch.where(cut, edge * a.abs() * 2 * U, r * a.abs() * (U * d.abs() + 2.0 ** -22 + 4 * U))
    g_err = torch.where(cut, z, err)
    k, k_err = z, z
    if ref is not None:
        x = nll64 - ref64
        k, em1 = torch.expm1(x) - x, torch.expm1(x)
        near = x.abs() < 0.5
        # k' = e^x - 1: x's rounding moves k by U |x| |e^x - 1|
        e1 = torch.where(near, 8 * U * em1.abs(), 2.0 ** -22 * x.exp() + 2 * U * em1.abs())
        k_err = torch.where(near, 8 * U * k, e1 + 2 * U * k) + U * x.abs() * em1.abs()
        e1 = e1 + U * x.abs() * x.exp()
        token, slope = token + w * k, slope + w * em1
        err = err + abs(w) * (k_err + 2 * U * k)
        g_err = g_err + abs(w) * (e1 + 2 * U * em1.abs())
    count = _by(counts.double(), s, seqs)
    part = 1.0 / count.clamp(min=1) if mean else torch.ones_like(count)
    c64 = counts.double()
    loss, kl = _by(token * c64, s, seqs) * part, _by(k * c64, s, seqs) * part
    loss_err = _by((err + 9 * U * (token.abs() + abs(w) * k)) * c64, s, seqs) * part + U * loss.abs()
    kl_err = _by((k_err + 7 * U * k) * c64, s, seqs) * part + U * kl
    clipped = _by(cut.double(), s, seqs)
    out = dict(loss=loss, loss_err=1.01 * loss_err + 1e-37, kl=kl, kl_err=1.01 * kl_err + 1e-37,
               count=count.int(), clipped=clipped.int(), inside=inside)
    if dloss is not None:
        each = (dloss.double() * part)[s]
        out["dnll"] = torch.where(counts, slope * each, z)
        out["dnll_err"] = 1.01 * torch.where(
            counts, each.abs() * (g_err + 6 * U * slope.abs()), z) + 1e-37
    return out


@pytest.mark.parametrize("kind,seqs,inside,lead,tail", CASES)
@pytest.mark.parametrize("ref,masked,per_token,mean", [(1, 1, 0, 1), (1, 0, 1, 0), (0, 1, 1, 1),
                                                       (0, 0, 0, 0)])
def test_policy(gpu, kind, seqs, inside, lead, tail, ref, masked, per_token, mean):
    n, off, offsets, nll, old, rf, mask, g = _pack(gpu, kind, seqs, inside, lead, tail,
                                                   seqs + inside, masked)
    rf = rf if ref else None
    adv = torch.randn(n if per_token else seqs, generator=g, device=gpu)
    adv[::7] = 0.0
    if per_token and masked:
        adv[~mask] = math.nan
    dloss = torch.randn(seqs, generator=g, device=gpu)
    lo, hi, w = 0.2, 0.28, 0.05 if ref else 0.0
    want = _policy_ref(off, n, nll, old, rf, mask, adv, per_token, lo, hi, w, mean, dloss)
    how = dict(ref_nll=rf, mask=mask, clip_low=lo, clip_high=hi, kl_weight=w, mean=bool(mean),
               per_token=bool(per_token))
    ws = torch.full((M.sequence_loss_workspace_size(n, seqs),), 255, dtype=torch.uint8, device=gpu)
    loss, kl, count, clipped = M.policy_loss_forward(nll, old, adv, offsets, workspace=ws, **how)
    assert torch.equal(count, want["count"]) and torch.equal(clipped, want["clipped"])
    assert_within(loss, want["loss"], want["loss_err"])
    assert_within(kl, want["kl"], want["kl_err"])
    # a buffer with guards on both sides; tokens of no sequence stay as they were
    buf = torch.full((n + 32,), 7.0, device=gpu)
    dnll = buf[16:16 + n]
    out = M.policy_loss_backward(nll, old, adv, offsets, count, dloss, dnll=dnll, **how)
    assert out is dnll
    assert_within(dnll[want["inside"]], want["dnll"][want["inside"]],
                  want["dnll_err"][want["inside"]])
    assert bool((dnll[~want["inside"]] == 7).all())
    assert bool((buf[:16] == 7).all()) and bool((buf[16 + n:] == 7).all())
    # again, and allocated
    again = M.policy_loss_forward(nll, old, adv, offsets, **how)
    assert all(same_bits(a, b) for a, b in zip(again, (loss, kl, count, clipped)))
    fresh = M.policy_loss_backward(nll, old, adv, offsets, count, dloss, **how)
    assert same_bits(fresh[want["inside"]], dnll[want["inside"]])
    assert not bool(fresh[~want["inside"]].any())


def _preference_ref(off, n, nll, ref, mask, beta, kind, margin, eps, mean, dloss):
    s, inside, counts = _seq(off, n, mask, nll.device)
    seqs = len(off) - 1
    z = torch.zeros(n, dtype=torch.float64, device=nll.device)
    term = -nll.double() if ref is None else ref.double() - nll.double()
    count = _by(counts.double(), s, seqs)
    scale = torch.full_like(count, beta)
    if mean:
        scale = scale / count.clamp(min=1)
    term = torch.where(counts, term, z)
    reward = _by(term, s, seqs) * scale
    x = reward[0::2] - reward[1::2] - margin
    sp = torch.nn.functional.softplus
    if kind == "logistic":
        loss = (1 - eps) * sp(-x, threshold=100) + eps * sp(x, threshold=100)
        slope = eps - torch.sigmoid(-x)
        turn = torch.sigmoid(x) * torch.sigmoid(-x)
    elif kind == "hinge":
        loss, slope, turn = (1 - x).clamp(min=0), -(x < 1).double(), torch.zeros_like(x)
    else:
        loss, slope, turn = (1 - x) ** 2, 2 * (x - 1), torch.full_like(x, 2.0)
    both = (count[0::2] > 0) & (count[1::2] > 0)
    slope = torch.where(both, slope, torch.zeros_like(x))
    # beta and margin come as fp32, fp64 sums of n terms
    r_err = (U + n * 2.0 ** -50) * (_by(term.abs(), s, seqs) * scale.abs())
    x_err = r_err[0::2] + r_err[1::2] + U * abs(margin)
    out = dict(loss=torch.where(both, loss, torch.zeros_like(x)), x=x, reward=reward,
               count=count.int(), inside=inside,
               reward_err=1.01 * (r_err + U * reward.abs()) + 1e-37,
               x_err=1.01 * (x_err + U * x.abs()) + 1e-37,
               loss_err=1.01 * ((slope.abs() + turn * x_err) * x_err + U * (1 + x.abs()) * (eps > 0)
                                + 2 * U * loss) + 1e-37)
    g = slope * dloss.double()
    g_err = dloss.double().abs() * (turn * 2 * (x_err + U * x.abs())
                                    + (2.0 ** -21 + 8 * U) * slope.abs() + (eps > 0) * 4 * U)
    each = torch.stack([-g, g], 1).reshape(-1) * scale
    each_err = torch.stack([g_err, g_err], 1).reshape(-1) * scale.abs()
    out["dnll"] = torch.where(counts, each[s], z)
    out["dnll_err"] = 1.01 * torch.where(counts, each_err[s], z) + 1e-37
    return out


@pytest.mark.parametrize("kind,seqs,inside,lead,tail", [
    ("even", 2, 2, 0, 0), ("ones", 1000, 1000, 3, 5), ("even", 8, 511, 0, 1),
    ("even", 2, 1024, 0, 0), ("ragged", 14, 1537, 9, 0), ("gaps", 300, 5000, 1, 700),
    ("one", 900, 40001, 0, 3), ("ragged", 5000, 70000, 0, 0), ("ragged", 40, 5000011, 513, 77)])
@pytest.mark.parametrize("loss,ref,masked,mean,eps", [
    ("logistic", 1, 1, 0, 0.0), ("logistic", 0, 0, 1, 0.1), ("hinge", 1, 0, 0, 0.0),
    ("squared", 1, 1, 1, 0.0)])
def test_preference(gpu, kind, seqs, inside, lead, tail, loss, ref, masked, mean, eps):
    n, off, offsets, nll, _, rf, mask, g = _pack(gpu, kind, seqs, inside, lead, tail,
                                                 seqs + inside, masked)
    rf = rf if ref else None
    dloss = torch.randn(seqs // 2, generator=g, device=gpu)
    beta, margin = (2.0, 0.3) if mean else (0.1, 0.0)
    want = _preference_ref(off, n, nll, rf, mask, beta, loss, margin, eps, mean, dloss)
    how = dict(mask=mask, beta=beta, kind=loss, smoothing=eps, mean=bool(mean))
    ws = torch.full((M.sequence_loss_workspace_size(n, seqs),), 255, dtype=torch.uint8, device=gpu)
    got = M.preference_loss_forward(nll, offsets, ref_nll=rf, margin=margin, workspace=ws, **how)
    assert torch.equal(got[3], want["count"])
    assert_within(got[2], want["reward"], want["reward_err"])
    assert_within(got[1], want["x"], want["x_err"])
    assert_within(got[0], want["loss"], want["loss_err"])
    # the border of the hinge is a step of its slope
    sure = torch.ones(n, dtype=torch.bool, device=gpu)
    if loss == "hinge":
        s, _, _ = _seq(off, n, mask, gpu)
        sure = ((want["x"] - 1).abs() > want["x_err"])[s // 2]
    buf = torch.full((n + 32,), 7.0, device=gpu)
    dnll = buf[16:16 + n]
    out = M.preference_loss_backward(offsets, got[1], got[3], dloss, dnll=dnll, **how)
    assert out is dnll
    at = want["inside"] & sure
    assert_within(dnll[at], want["dnll"][at], want["dnll_err"][at])
    assert bool((dnll[~want["inside"]] == 7).all())
    assert bool((buf[:16] == 7).all()) and bool((buf[16 + n:] == 7).all())
    again = M.preference_loss_forward(nll, offsets, ref_nll=rf, margin=margin, **how)
    assert all(same_bits(a, b) for a, b in zip(again, got))
    fresh = M.preference_loss_backward(offsets, got[1], got[3], dloss, n=n, **how)
    assert same_bits(fresh[want["inside"]], dnll[want["inside"]])
    assert not bool(fresh[~want["inside"]].any())


def test_ratios_at_the_border_are_not_held(gpu):
    # d a step to each side of log(1.28) and log(0.8), and ratios of 1
    hi, lo = 0.28, 0.2
    up, down = torch.tensor(math.log1p(hi)), torch.tensor(math.log1p(-lo))
    step = lambda v, to: torch.nextafter(v, torch.tensor(to))  # noqa: E731
    d = torch.stack([step(up, 9.0), step(up, 0.0), up, step(down, -9.0), step(down, 0.0), down,
                     torch.tensor(0.0)]).to(gpu)
    nll = torch.zeros(7, device=gpu)
    off = torch.tensor([0, 7], dtype=torch.int32, device=gpu)
    for a in (1.0, -1.0):
        adv = torch.full((7,), a, device=gpu)
        r = d.double().exp()
        cut = (r > 1 + hi) if a > 0 else (r < 1 - lo)
        _, _, count, clipped = M.policy_loss_forward(nll, d, adv, off, clip_low=lo, clip_high=hi,
                                                     per_token=True)
        assert int(clipped[0]) == int(cut.sum()) and int(count[0]) == 7
        dn = M.policy_loss_backward(nll, d, adv, off, count, torch.ones(1, device=gpu),
                                    clip_low=lo, clip_high=hi, per_token=True, mean=False)
        assert torch.equal(dn == 0, cut)
    # clip_low 1 holds no low ratio, clip_high 0 every one above 1
    _, _, _, c = M.policy_loss_forward(nll, d - 200, -torch.ones(7, device=gpu), off, clip_low=1.0,
                                       clip_high=0.0, per_token=True)
    assert int(c[0]) == 0
    _, _, _, c = M.policy_loss_forward(nll, d.abs(), torch.ones(7, device=gpu), off, clip_low=1.0,
                                       clip_high=0.0, per_token=True)
    assert int(c[0]) == 6


def test_values_that_are_not_finite_stay_in_their_sequence(gpu):
    n, off, offsets, nll, old, ref, _, g = _pack(gpu, "ragged", 9, 3000, 0, 0, 5, 0)
    adv, dl = torch.randn(9, generator=g, device=gpu), torch.randn(9, generator=g, device=gpu)
    adv[6] = 0.0
    how = dict(ref_nll=ref, kl_weight=0.1)
    base = M.policy_loss_forward(nll, old, adv, offsets, **how)
    grad = M.policy_loss_backward(nll, old, adv, offsets, base[2], dl, **how)
    mid = (off[3] + off[4]) // 2
    held = nll[mid].clone()
    nll[mid] = math.nan
    old[off[6]] = math.inf       # a ratio of infinity with an advantage of 0
    got = M.policy_loss_forward(nll, old, adv, offsets, **how)
    others = torch.arange(9, device=gpu) != 3
    assert bool(got[0][3].isnan()) and bool(got[0][others].isfinite().all())
    same = others & (torch.arange(9, device=gpu) != 6)
    assert same_bits(got[0][same], base[0][same])
    dn = M.policy_loss_backward(nll, old, adv, offsets, got[2], dl, **how)
    assert bool(dn[mid].isnan())
    dn[mid] = grad[mid]
    dn[off[6]] = grad[off[6]]
    assert same_bits(dn, grad)
    nll[mid] = held
    pairs = torch.tensor(off[:9], dtype=torch.int32, device=gpu)
    nll[mid] = math.inf
    loss, x, reward, _ = M.preference_loss_forward(nll, pairs, ref_nll=ref)
    assert float(reward[3]) == -math.inf and float(x[1]) == math.inf and float(loss[1]) == 0.0
    assert bool(loss.isfinite().all())
    d = M.preference_loss_backward(pairs, x, _, torch.ones(4, device=gpu), n=n)
    assert bool(d.isfinite().all()) and not bool(d[off[2]:off[4]].any())


def test_nothing_to_do(gpu):
    e, off = torch.empty(0, device=gpu), torch.zeros(1, dtype=torch.int32, device=gpu)
    assert M.policy_loss_forward(e, e, e, off)[0].numel() == 0
    dn = M.policy_loss_backward(e, e, e, off, off[:0], e)
    assert dn.numel() == 0
    # sequences without tokens, tokens without sequences
    off = torch.zeros(5, dtype=torch.int32, device=gpu)
    four = torch.ones(4, device=gpu)
    loss, kl, count, clipped = M.policy_loss_forward(e, e, four, off)
    assert not bool(loss.any()) and not bool(kl.any()) and not bool(count.any())
    t = torch.full((600,), math.nan, device=gpu)
    for off in (torch.zeros(5, dtype=torch.int32, device=gpu),
                torch.full((5,), 600, dtype=torch.int32, device=gpu)):
        loss, kl, count, clipped = M.policy_loss_forward(t, t, four, off)
        assert not bool(loss.any()) and not bool(count.any()) and not bool(clipped.any())
        dn = M.policy_loss_backward(t, t, four, off, count, four, dnll=t.clone())
        assert bool(dn.isnan().all())
        loss, x, reward, count = M.preference_loss_forward(t, off, margin=0.25)
        assert not bool(loss.any()) and not bool(reward.any()) and bool((x == -0.25).all())
        assert not bool(M.preference_loss_backward(off, x, count, four[:2], n=600).any())
    # a batch in which nothing counts
    off = torch.tensor([0, 100, 200, 500, 600], dtype=torch.int32, device=gpu)
    mask = torch.zeros(600, dtype=torch.uint8, device=gpu)
    loss, kl, count, clipped = M.policy_loss_forward(t, t, four, off, mask=mask)
    assert not bool(loss.any()) and not bool(count.any())
    dn = M.policy_loss_backward(t, t, four, off, count, four * math.nan, mask=mask)
    assert not bool(dn.any())


def test_offsets_beyond_the_tokens_are_clamped(gpu):
    nll = torch.rand(700, device=gpu)
    adv = torch.ones(3, device=gpu)
    off = torch.tensor([-5, 300, 650, 2 ** 31 - 1], dtype=torch.int32, device=gpu)
    want = torch.tensor([0, 300, 650, 700], dtype=torch.int32, device=gpu)
    a = M.policy_loss_forward(nll, nll, adv, off)
    b = M.policy_loss_forward(nll, nll, adv, want)
    assert all(same_bits(x, y) for x, y in zip(a, b)) and a[2].tolist() == [300, 350, 50]


def test_gradients_against_differences(gpu):
    # central differences of the fp64 sums: f's third derivative over 6 times
    # eps^2, and the results' roundings over eps
    n, off, offsets, nll, old, ref, mask, g = _pack(gpu, "ragged", 6, 400, 0, 0, 8, 0)
    adv, dl = torch.randn(6, generator=g, device=gpu), torch.rand(6, generator=g, device=gpu)
    eps = 2.0 ** -9
    how = dict(ref_nll=ref, kl_weight=0.2, mean=False)
    base = M.policy_loss_forward(nll, old, adv, offsets, **how)
    grad = M.policy_loss_backward(nll, old, adv, offsets, base[2], dl, **how)
    d = (old - nll).double()
    # a token whose border lies within the step is left out
    near = ((d - math.log1p(0.2)).abs() < 2 * eps) | ((d - math.log1p(-0.2)).abs() < 2 * eps)
    v = torch.where(near, torch.zeros(n, device=gpu), torch.randn(n, generator=g, device=gpu).sign())
    f = lambda t: float((M.policy_loss_forward(t, old, adv, offsets, **how)[0].double()  # noqa: E731
                         * dl.double()).sum())
    slope = (f(nll + eps * v) - f(nll - eps * v)) / (2 * eps)
    size = float((dl.double() * base[0].double().abs()).sum())
    s, _, _ = _seq(off, n, None, gpu)
    third = (d.exp() * adv[s].double().abs() + 0.2 * (nll - ref).double().exp()) * 1.02
    tol = float((dl[s].double() * third).sum()) * eps ** 2 / 6
    terms = float((dl[s].double() * (third + 1)).sum())
    tol += (size * U + terms * 2.0 ** -21) / eps
    assert abs(slope - float((grad.double() * v.double()).sum())) <= tol

    dp = torch.rand(3, generator=g, device=gpu)
    for kind, sm in (("logistic", 0.1), ("squared", 0.0)):
        pk = dict(kind=kind, smoothing=sm, beta=0.05)
        loss, x, reward, count = M.preference_loss_forward(nll, offsets, ref_nll=ref, **pk)
        grad = M.preference_loss_backward(offsets, x, count, dp, n=n, **pk)
        v = torch.randn(n, generator=g, device=gpu).sign()
        f = lambda t: float((M.preference_loss_forward(t, offsets, ref_nll=ref, **pk)[0]  # noqa: E731
                             .double() * dp.double()).sum())
        slope = (f(nll + eps * v) - f(nll - eps * v)) / (2 * eps)
        span = 0.05 * n * eps     # x moves by no more; |f'''| <= 1/4, quadratics have none
        tol = float(dp.sum()) * (span ** 3 / 24 / eps + 4 * U * float(loss.max() + 1) / eps)
        # the points are rounded: 2^-24 of each token
        tol += float(dp.max()) * 0.05 * float((nll.abs() + 1).sum()) * U / eps * 4
        tol += 2.0 ** -20 * float((grad.abs()).sum())
        assert abs(slope - float((grad.double() * v.double()).sum())) <= tol


@pytest.mark.parametrize("seqs,tail", [(3, 0), (1 << 24, 1000)])
def test_most_tokens_and_most_sequences(gpu, seqs, tail):
    # values that every sum holds exactly: small integers over 8
    n = (1 << 26) - 1
    g = torch.Generator(device=gpu)
    g.manual_seed(seqs)
    cuts = torch.randint(0, n - tail + 1, (seqs - 1,), generator=g, device=gpu).sort().values
    off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), n - tail)]).int()
    nll = torch.randint(0, 8, (n,), generator=g, device=gpu).float() / 8
    mask = torch.randint(0, 2, (n,), generator=g, device=gpu, dtype=torch.uint8)
    adv = torch.ones(seqs, device=gpu)
    loss, kl, count, clipped = M.policy_loss_forward(nll, nll, adv, off, mask=mask, mean=False)
    ends = torch.cat([off.new_zeros(1).long(), mask.long().cumsum(0)])[off.long()]
    want = ends[1:] - ends[:-1]
    assert torch.equal(count.long(), want) and not bool(clipped.any()) and not bool(kl.any())
    assert torch.equal(loss, -want.float())          # a ratio of 1 for every token
    dn = M.policy_loss_backward(nll, nll, adv, off, count, adv, mask=mask, mean=False,
                                dnll=torch.full((n,), 7.0, device=gpu))
    assert torch.equal(dn[:n - tail], mask[:n - tail].float())
    assert bool((dn[n - tail:] == 7).all())
    if seqs % 2 == 0:
        loss, x, reward, count = M.preference_loss_forward(nll, off, mask=mask, beta=1.0)
        ends = torch.cat([nll.new_zeros(1).double(), (nll * mask).double().cumsum(0)])[off.long()]
        assert torch.equal(reward, -(ends[1:] - ends[:-1]).float())
        assert torch.equal(count.long(), want)
