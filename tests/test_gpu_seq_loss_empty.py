"""Offsets with long runs of empty sequences, as a batch of fixed capacity has
whose unused slots all hold the same offset."""

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import same_bits

pytestmark = pytest.mark.gpu

# the sequences that hold tokens, by their ends; n is no multiple of 512
LIVE = [1, 2, 70, 511, 512, 513, 1500, 1501, 1600, 9000, 9001, 9777]


def _runs(gpu, at, run):
    """Offsets of LIVE with `run` empty sequences, an even number, before each
    of the live ones named by `at` (len(LIVE): behind the last), and the
    indexes of the live ones."""
    off, live, last = [0], [], 0
    for k, end in enumerate([*LIVE, None]):
        if k in at:
            off += [last] * run
        if end is not None:
            live.append(len(off) - 1)
            off.append(end)
            last = end
    return (torch.tensor(off, dtype=torch.int32, device=gpu), torch.tensor(live, device=gpu))


@pytest.mark.parametrize("run", [62, 64, 126, 128, 130, 190, 192, 4098, 70002])
@pytest.mark.parametrize("at", [(0,), (3,), (5, 6), (12,), (0, 2, 3, 7, 9, 12)])
@pytest.mark.parametrize("tail", [0, 5, 700])
def test_runs_of_empty_sequences(gpu, at, run, tail):
    n = LIVE[-1] + tail
    g = torch.Generator(device=gpu)
    g.manual_seed(run)
    r = lambda m: torch.rand(m, generator=g, device=gpu)  # noqa: E731
    nll, old, ref, adv, dl = r(n), r(n), r(n), r(len(LIVE)) - 0.5, r(len(LIVE))
    mask = r(n) < 0.7
    base = torch.tensor([0, *LIVE], dtype=torch.int32, device=gpu)
    off, live = _runs(gpu, at, run)
    seqs = off.numel() - 1
    how = dict(ref_nll=ref, mask=mask, kl_weight=0.1)
    want = M.policy_loss_forward(nll, old, adv, base, **how)
    dwant = M.policy_loss_backward(nll, old, adv, base, want[2], dl, **how)
    wide = torch.full((2, seqs), float("nan"), device=gpu)
    wide[0, live], wide[1, live] = adv, dl
    got = M.policy_loss_forward(nll, old, wide[0], off, **how)
    empty = torch.ones(seqs, dtype=torch.bool, device=gpu)
    empty[live] = False
    for a, b in zip(got, want):
        assert torch.equal(a[live], b) and not bool(a[empty].any())
    assert same_bits(M.policy_loss_backward(nll, old, wide[0], off, got[2], wide[1], **how), dwant)
    # preference: pairs stay pairs, as every run is even
    how = dict(mask=mask, mean=True)
    want = M.preference_loss_forward(nll, base, ref_nll=ref, **how)
    dwant = M.preference_loss_backward(base, want[1], want[3], dl[:6], n=n, **how)
    pairs = live[0::2] // 2
    if bool((live[0::2] % 2 == 0).all()) and bool((live[1::2] == live[0::2] + 1).all()):
        got = M.preference_loss_forward(nll, off, ref_nll=ref, **how)
        assert torch.equal(got[2][live], want[2]) and torch.equal(got[0][pairs], want[0])
        dp = torch.full((seqs // 2,), float("nan"), device=gpu)
        dp[pairs] = dl[:6]
        assert same_bits(M.preference_loss_backward(off, got[1], got[3], dp, n=n, **how), dwant)


def test_runs_of_all_lengths_in_one_tile(gpu):
    # every token of two tiles starts a sequence, with 0 to 200 empty ones before
    # it; and the offsets' clamped ends
    n = 1023
    lengths = (torch.arange(n) * 37) % 201
    off = torch.repeat_interleave(torch.arange(n), lengths + 1)
    live = (lengths + 1).cumsum(0) - 1
    off = torch.cat([off, torch.full((300,), n + 9)]).int().to(gpu)
    seqs = off.numel() - 1
    adv = torch.full((seqs,), float("nan"), device=gpu)
    adv[live.to(gpu)] = torch.arange(n, device=gpu).float() + 1
    nll = torch.rand(n, device=gpu)
    loss, _, count, _ = M.policy_loss_forward(nll, nll, adv, off)
    want = torch.zeros(seqs, device=gpu)
    want[live.to(gpu)] = -(torch.arange(n, device=gpu).float() + 1)
    assert torch.equal(loss, want) and int(count.sum()) == n
    dn = M.policy_loss_backward(nll, nll, adv, off, count, adv.nan_to_num() * 0 + 1)
    assert torch.equal(dn, torch.arange(n, device=gpu).float() + 1)


def test_unused_slots_take_no_time(gpu):
    # 2^20 slots, 100 of them used: no longer than 2^20 spread over the tokens
    # (0.6 ms); going through the slots 64 at a time, each load waiting for the
    # one before, took 22 ms
    n, used, slots = 50001, 100, 1 << 20
    nll = torch.rand(n, device=gpu)
    adv = torch.ones(slots, device=gpu)
    lived = torch.linspace(0, n, used + 1, device=gpu).int()
    spread = (torch.arange(slots + 1, device=gpu) * n // slots).int()
    padded = torch.cat([lived, lived.new_full((slots - used,), n)])
    times = {}
    for name, off in (("spread", spread), ("padded", padded)):
        ws = torch.empty(M.sequence_loss_workspace_size(n, slots), dtype=torch.uint8, device=gpu)
        dn = torch.empty(n, device=gpu)
        best = float("inf")
        for _ in range(4):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            out = M.policy_loss_forward(nll, nll, adv, off, workspace=ws)
            M.policy_loss_backward(nll, nll, adv, off, out[2], adv, dnll=dn)
            e[1].record()
            e[1].synchronize()
            best = min(best, e[0].elapsed_time(e[1]))
        times[name] = best
    assert times["padded"] <= 3 * times["spread"] + 1.0, times
