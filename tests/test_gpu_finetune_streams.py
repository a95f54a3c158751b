"""The stream that the losses of fine-tuning run on.  The stream asked for first
has some 30 ms of work, then copies of the inputs into buffers that hold other
values; the calls are made without waiting for it.  On any other stream they
would read those other values."""

import pytest
import torch

import muon_newton_schulz_amd as M
from train_ops_util import same_bits

pytestmark = pytest.mark.gpu

N, V, D, K, S = 3000, 700, 96, 9, 12


def _inputs(gpu, seed):
    g = torch.Generator(device=gpu)
    g.manual_seed(seed)
    r = lambda *s: torch.rand(*s, generator=g, device=gpu)  # noqa: E731
    cuts = torch.randint(0, N + 1, (S - 1,), generator=g, device=gpu).sort().values
    t = dict(nll=r(N), old=r(N), ref=r(N), mask=r(N) < 0.7, adv=r(S) - 0.5, a=r(S), b=r(S // 2),
             offsets=torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), N)]).int(),
             h=(r(N, D) - 0.5).bfloat16(), w=(r(V, D) - 0.5).bfloat16(),
             ids=torch.randint(-20, V, (N, K), generator=g, device=gpu), z=r(N, K) * 4,
             dloss=r(N))
    how = dict(ref_nll=t["ref"], mask=t["mask"])
    # what the backward calls take from the forward ones
    t["count"] = M.policy_loss_forward(t["nll"], t["old"], t["adv"], t["offsets"], **how)[2]
    _, t["x"], _, _ = M.preference_loss_forward(t["nll"], t["offsets"], **how)
    _, t["lse"], t["logp"] = M.distill_loss_forward(t["h"], t["w"], t["ids"], t["z"])
    return t


CALLS = {
    "policy_loss_forward": lambda t, **k: M.policy_loss_forward(
        t["nll"], t["old"], t["adv"], t["offsets"], ref_nll=t["ref"], mask=t["mask"],
        kl_weight=0.1, **k),
    "policy_loss_backward": lambda t, **k: (M.policy_loss_backward(
        t["nll"], t["old"], t["adv"], t["offsets"], t["count"], t["a"], ref_nll=t["ref"],
        mask=t["mask"], kl_weight=0.1, **k),),
    "preference_loss_forward": lambda t, **k: M.preference_loss_forward(
        t["nll"], t["offsets"], ref_nll=t["ref"], mask=t["mask"], **k),
    "preference_loss_backward": lambda t, **k: (M.preference_loss_backward(
        t["offsets"], t["x"], t["count"], t["b"], mask=t["mask"], **k),),
    "distill_loss_forward": lambda t, **k: M.distill_loss_forward(
        t["h"], t["w"], t["ids"], t["z"], **k),
    "distill_loss_backward": lambda t, **k: M.distill_loss_backward(
        t["h"], t["w"], t["ids"], t["z"], t["lse"], t["logp"], t["dloss"], **k),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("how", ["stream", "handle", "current", "default", "zero"])
def test_calls_follow_their_stream(gpu, name, how):
    real, held = _inputs(gpu, 1), _inputs(gpu, 2)
    want, other = CALLS[name](real), CALLS[name](held)
    assert not any(torch.equal(a, b) for a, b in zip(want, other))
    side = torch.cuda.Stream()
    first = torch.cuda.default_stream() if how in ("default", "zero") else side
    given = {"stream": side, "handle": side.cuda_stream, "current": None,
             "default": first, "zero": 0}[how]
    a = torch.full((8192, 8192), 2.0 ** -13, dtype=torch.bfloat16, device=gpu)
    c = torch.empty_like(a)
    torch.mm(a, a, out=c)
    torch.cuda.synchronize()
    with torch.cuda.stream(first):
        torch.mm(a, a, out=c)  # (the stream's first, with what it allocates)
        torch.cuda.synchronize()
        for _ in range(40):
            torch.mm(a, a, out=c)
        for k, t in held.items():
            t.copy_(real[k])
    # the calls' own current stream: the one asked for, or another
    with torch.cuda.stream(first if how == "current" else torch.cuda.Stream()):
        got = CALLS[name](held, **({} if given is None else {"stream": given}))
    busy = not first.query()
    torch.cuda.synchronize()
    assert busy, "the work before the call ended too early to show anything"
    for x, y in zip(got, want):
        assert same_bits(x, y)


@pytest.mark.parametrize("name", list(CALLS))
def test_the_handle_that_reaches_the_library(gpu, name, monkeypatch):
    t = _inputs(gpu, 3)
    side, seen, real = torch.cuda.Stream(), [], M.lib()

    class Spy:
        def __getattr__(self, attr):
            call = getattr(real, attr)
            if attr != name:
                return call

            def spy(*args):
                seen.append(args[-1] or 0)
                return call(*args)
            return spy

    torch.cuda.synchronize()
    monkeypatch.setattr(M, "lib", Spy)
    CALLS[name](t)
    CALLS[name](t, stream=side)
    CALLS[name](t, stream=side.cuda_stream)
    with torch.cuda.stream(side):
        CALLS[name](t)
        CALLS[name](t, stream=torch.cuda.default_stream())
        CALLS[name](t, stream=0)
    torch.cuda.synchronize()
    h = side.cuda_stream
    assert h and seen == [0, h, h, h, 0, 0]
