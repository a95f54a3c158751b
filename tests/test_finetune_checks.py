"""Refusals of the distillation, policy and preference losses, without a GPU:
the binding's checks on stand-in tensors, outputs and workspaces that share
memory with other tensors, and the C entry points' own checks, which come
before any HIP call."""

import ctypes
import math

import pytest
import torch

import muon_newton_schulz_amd as M
from test_train_ops_checks import DTYPE, I64, INVALID, SHAPE, WS, Placed, _err, _rc

F32, I32, U8, BOOL = torch.float32, torch.int32, torch.uint8, torch.bool
AT = 1 << 24
p = ctypes.c_void_p(256)  # never dereferenced: the calls it goes to are refused


class T(Placed):
    """A stand-in in a part of memory of its own unless it is told where."""
    made = 0

    def __init__(self, shape, dtype=F32, stride=None, dev="cuda:0", at=None):
        T.made += 1
        super().__init__(AT * T.made if at is None else at, shape, dtype, stride)
        self.device = torch.device(dev)
        self.is_cuda = self.device.type == "cuda"

    def get_device(self):
        return self.device.index if self.is_cuda else -1


def _over(t, shape, dtype=F32):
    """Stand-ins that share memory with contiguous t: its start, its last
    element, and from before it into its first."""
    one = torch.empty(0, dtype=dtype).element_size()
    for d in (0, t.numel() * t.element_size() - one, 1 - torch.Size(shape).numel() * one):
        yield T(shape, dtype, at=t.data_ptr() + d)


# ------------------------------------------------------------ distillation

def _lists():
    return dict(hidden=T((6, 16), torch.bfloat16), weight=T((100, 16), torch.bfloat16),
                ids=T((6, 5), I64), teacher=T((6, 5)))


def test_distill_binding_checks():
    bf = torch.bfloat16

    def fwd(status, temperature=1.0, loss=None, lse=None, logp=None, workspace=None, **new):
        a = {**_lists(), **new}
        _err(status, M.distill_loss_forward, a["hidden"], a["weight"], a["ids"], a["teacher"],
             temperature, loss, lse, logp, workspace)

    fwd(INVALID, hidden=T((6, 16), bf, dev="cpu"))
    fwd(INVALID, weight=T((100, 16), bf, stride=(1, 100)))
    fwd(INVALID, weight=None)
    fwd(INVALID, teacher=None)
    fwd(INVALID, hidden=None)
    fwd(SHAPE, ids=None)
    fwd(SHAPE, weight=T((1600,), bf))
    fwd(SHAPE, ids=T((30,), I64))
    fwd(SHAPE, teacher=T((6, 4)))
    fwd(SHAPE, hidden=T((5, 16), bf))
    fwd(SHAPE, hidden=T((6, 17), bf))
    fwd(DTYPE, hidden=T((6, 16)))
    fwd(DTYPE, ids=T((6, 5), torch.int16))
    fwd(DTYPE, ids=T((6, 5)))
    fwd(DTYPE, teacher=T((6, 5), torch.float16))
    fwd(INVALID, ids=T((6, 5), I64, stride=(4, 1)))
    fwd(INVALID, ids=T((6, 5), I64, stride=(1, 6)))
    fwd(INVALID, teacher=T((6, 5), stride=(10, 2)))
    fwd(SHAPE, loss=T((5,)))
    fwd(DTYPE, lse=T((6,), bf))
    fwd(SHAPE, logp=T((5, 6)))
    fwd(INVALID, logp=T((6, 5), stride=(8, 1)))
    fwd(INVALID, teacher=T((6, 5), dev="cuda:1"))
    fwd(INVALID, workspace=T((10,), U8, dev="cuda:1"))

    def bwd(status, lse=None, logp=None, dloss=None, **k):
        a = _lists()
        _err(status, M.distill_loss_backward, a["hidden"], a["weight"], a["ids"], a["teacher"],
             T((6,)) if lse is None else lse, T((6, 5)) if logp is None else logp,
             T((6,)) if dloss is None else dloss, **k)

    bwd(SHAPE, lse=T((7,)))
    bwd(DTYPE, logp=T((6, 5), bf))
    bwd(SHAPE, logp=T((6, 4)))
    bwd(SHAPE, dloss=T((1,)))
    bwd(SHAPE, dhidden=T((6, 15), bf))
    bwd(SHAPE, dweight=T((16, 100), bf))
    bwd(DTYPE, dweight=T((100, 16), torch.float16))
    bwd(INVALID, dweight=T((100, 16), stride=(32, 1)))
    bwd(INVALID, accumulate=True)
    bwd(INVALID, dweight=False, accumulate=True)


def test_distill_outputs_share_no_memory():
    a = _lists()
    args = [a[k] for k in ("hidden", "weight", "ids", "teacher")]
    for x in args:
        for out in _over(x, (6,)):
            _err(INVALID, M.distill_loss_forward, *args, loss=out)
            _err(INVALID, M.distill_loss_forward, *args, lse=out)
        for out in _over(x, (6, 5)):
            _err(INVALID, M.distill_loss_forward, *args, logp=out)
        for ws in _over(x, (512,), U8):
            _err(INVALID, M.distill_loss_forward, *args, workspace=ws)
    one = T((6,))
    _err(INVALID, M.distill_loss_forward, *args, loss=one, lse=one)
    lse, logp, dl, dw = T((6,)), T((6, 5)), T((6,)), T((100, 16))
    for x in (*args, lse, logp, dl):
        for out in _over(x, (6, 16)):
            _err(INVALID, M.distill_loss_backward, *args, lse, logp, dl, dhidden=out,
                 dweight=False)
        for out in _over(x, (100, 16)):
            _err(INVALID, M.distill_loss_backward, *args, lse, logp, dl, dhidden=False,
                 dweight=out)
    for out in _over(dw, (6, 16)):
        _err(INVALID, M.distill_loss_backward, *args, lse, logp, dl, dhidden=out, dweight=dw)
    for ws in (*_over(logp, (512,), U8), *_over(dw, (512,), U8)):
        _err(INVALID, M.distill_loss_backward, *args, lse, logp, dl, dhidden=False, dweight=dw,
             workspace=ws)
    # ids beside the teacher's values in one buffer, rows of 8 and 5 elements
    ids = T((6, 5), I32, stride=(16, 1), at=AT)
    z = T((6, 5), stride=(16, 1), at=AT + 20)
    logp = T((6, 5), at=AT + 4096)
    assert M._distill_args(a["hidden"], a["weight"], ids, z)[0] == (6, 100, 16, 5)
    M._outputs_apart({"logp": M._vector(logp)}, {"ids": (ids, 6, 5, 16), "z": (z, 6, 5, 16)}, None)


def test_distill_entry_points_refuse():
    size = M.distill_loss_workspace_size
    need_f, need_b = size(4, 10, 8, 3, "bf16", False), size(4, 10, 8, 3, "bf16")
    assert 0 < need_f <= need_b
    assert size(0, 10, 8, 3, "bf16") == 0 and size(4, 10, 8, 0, "bf16") == 0
    assert size(4, 10, 8, 1025, "bf16") == 0 and size(4, 10, 8, 1024, "bf16") > 0
    assert size(4, 2 ** 21 + 1, 8, 3, "bf16") == 0 and size((1 << 24) + 1, 10, 8, 3, "bf16") == 0

    def fwd(h=p, ld=8, w=p, dt=1, ids=p, i64=1, ldi=3, z=p, zd=0, ldz=3, n=4, vocab=10, dim=8,
            top=3, T=1.0, loss=p, lse=p, logp=p, ws=p, nb=need_f):
        return _rc("distill_loss_forward", h, ld, w, dt, ids, i64, ldi, z, zd, ldz, n, vocab, dim,
                   top, T, loss, lse, logp, ws, nb, None)

    assert fwd(dt=2) == DTYPE and fwd(zd=2) == DTYPE and fwd(n=-1) == SHAPE
    assert fwd(vocab=0) == SHAPE and fwd(dim=0, ld=0) == SHAPE and fwd(ld=7) == SHAPE
    assert fwd(ldi=2) == SHAPE and fwd(ldz=2) == SHAPE
    assert fwd(top=0) == SHAPE and fwd(top=1025, ldi=1025, ldz=1025) == SHAPE
    for t in (0.0, -1.0, math.nan, math.inf, 1e-7, 1e7):
        assert fwd(T=t) == INVALID
    assert fwd(vocab=2 ** 21 + 1) == M.MUON_ERR_UNSUPPORTED
    for k in ("h", "w", "ids", "z", "loss", "lse", "logp"):
        assert fwd(**{k: None}) == INVALID
    assert fwd(ws=None) == WS and fwd(nb=need_f - 1) == WS and fwd(ws=ctypes.c_void_p(8)) == WS
    assert fwd(n=0, h=None, ids=None, ws=None, nb=0) == M.MUON_OK

    def bwd(h=p, ld=8, w=p, dt=1, ids=p, i64=1, ldi=3, z=p, zd=0, ldz=3, n=4, vocab=10, dim=8,
            top=3, T=1.0, lse=p, logp=p, dl=p, dh=p, dhd=1, ldh=8, dw=p, dwd=0, acc=0, ws=p,
            nb=need_b):
        return _rc("distill_loss_backward", h, ld, w, dt, ids, i64, ldi, z, zd, ldz, n, vocab, dim,
                   top, T, lse, logp, dl, dh, dhd, ldh, dw, dwd, acc, ws, nb, None)

    assert bwd(dt=2) == DTYPE and bwd(dhd=2) == DTYPE and bwd(dwd=-1) == DTYPE
    assert bwd(zd=-1) == DTYPE and bwd(T=0.0) == INVALID and bwd(top=0) == SHAPE
    assert bwd(ldh=7) == SHAPE and bwd(ld=7) == SHAPE and bwd(ldi=1) == SHAPE
    for k in ("h", "w", "ids", "z", "lse", "logp", "dl"):
        assert bwd(**{k: None}) == INVALID
    assert bwd(ws=None) == WS and bwd(nb=need_b - 1) == WS and bwd(ws=ctypes.c_void_p(8)) == WS
    assert bwd(dh=None, dw=None, ws=None, nb=0) == M.MUON_OK
    assert bwd(n=0, dw=None) == M.MUON_OK and bwd(n=0, acc=1) == M.MUON_OK


# --------------------------------------------------------- packed sequences

N, S = 40, 6


def _policy():
    return dict(nll=T((N,)), old_nll=T((N,)), advantages=T((S,)), offsets=T((S + 1,), I32))


def _bad(n, dtype=F32):
    """Stand-ins that are not n contiguous elements of dtype on the GPU."""
    other = torch.float64 if dtype is F32 else I64
    yield DTYPE, T((n,), other)
    yield SHAPE, T((n + 1,), dtype)
    yield SHAPE, T((n - 1,), dtype)
    yield INVALID, T((n,), dtype, stride=(2,))
    yield INVALID, T((n,), dtype, dev="cpu")
    yield INVALID, T((n,), dtype, dev="cuda:1")


def test_policy_binding_checks():
    def fwd(status, **k):
        _err(status, M.policy_loss_forward, **{**_policy(), **k})

    def bwd(status, **k):
        _err(status, M.policy_loss_backward,
             **{**_policy(), "count": T((S,), I32), "dloss": T((S,)), **k})

    for f in (fwd, bwd):
        f(INVALID, nll=None)
        f(INVALID, nll=T((N,), dev="cpu"))
        f(DTYPE, nll=T((N,), torch.bfloat16))
        f(INVALID, nll=T((N,), stride=(2,)))
        f(INVALID, old_nll=None)
        f(INVALID, advantages=None)
        f(INVALID, offsets=None)
        f(SHAPE, offsets=T((0,), I32))
        f(INVALID, kl_weight=0.1)
        f(SHAPE, per_token=True)
        f(SHAPE, advantages=T((N,)))
        f(DTYPE, offsets=T((S + 1,), I64))
        for status, t in _bad(N):
            f(status, old_nll=t)
            f(status, ref_nll=t)
            f(status, advantages=t, per_token=True)
        for status, t in _bad(S):
            f(status, advantages=t)
        f(DTYPE, mask=T((N,)))
        f(DTYPE, mask=T((N,), I32))
        f(SHAPE, mask=T((N + 1,), BOOL))
        f(INVALID, mask=T((N,), U8, stride=(2,)))
        f(INVALID, mask=T((N,), BOOL, dev="cuda:1"))
    for status, t in _bad(S):
        fwd(status, loss=t)
        fwd(status, kl=t)
        bwd(status, dloss=t)
    for status, t in _bad(S, I32):
        fwd(status, count=t)
        fwd(status, clipped=t)
        bwd(status, count=t)
    for status, t in _bad(N):
        bwd(status, dnll=t)
    fwd(INVALID, workspace=T((100,), U8, dev="cuda:1"))
    fwd(INVALID, workspace=T((100,), U8, stride=(2,)))
    bwd(INVALID, count=None)
    bwd(INVALID, dloss=None)


def test_preference_binding_checks():
    def fwd(status, **k):
        _err(status, M.preference_loss_forward,
             **{"nll": T((N,)), "offsets": T((S + 1,), I32), **k})

    def bwd(status, **k):
        _err(status, M.preference_loss_backward,
             **{"offsets": T((S + 1,), I32), "margins": T((S // 2,)), "count": T((S,), I32),
                "dloss": T((S // 2,)), "n": N, **k})

    fwd(INVALID, nll=None)
    for status, t in _bad(N):
        fwd(status, ref_nll=t)
        bwd(status, dnll=t)
    for f in (fwd, bwd):
        f(INVALID, offsets=None)
        f(SHAPE, offsets=T((6,), I32))       # five sequences
        f(DTYPE, offsets=T((S + 1,)))
        f(INVALID, kind="ranked")
        f(DTYPE, mask=T((N,)))
        f(SHAPE, mask=T((N - 1,), BOOL))
    for status, t in _bad(S // 2):
        fwd(status, loss=t)
        fwd(status, margins=t)
        bwd(status, margins=t)
        bwd(status, dloss=t)
    for status, t in _bad(S):
        fwd(status, reward=t)
    for status, t in _bad(S, I32):
        fwd(status, count=t)
        bwd(status, count=t)
    bwd(INVALID, n=None)
    bwd(INVALID, margins=None)
    bwd(INVALID, count=None)
    bwd(INVALID, dloss=None)
    bwd(INVALID, offsets=T((S + 1,), I32, dev="cpu"))


def test_sequence_outputs_share_no_memory():
    a = {**_policy(), "ref_nll": T((N,)), "mask": T((N,), BOOL)}
    for x in a.values():
        for name, dt in (("loss", F32), ("kl", F32), ("count", I32), ("clipped", I32)):
            for out in _over(x, (S,), dt):
                _err(INVALID, M.policy_loss_forward, **a, **{name: out})
        for ws in _over(x, (512,), U8):
            _err(INVALID, M.policy_loss_forward, **a, workspace=ws)
    b = {**a, "count": T((S,), I32), "dloss": T((S,))}
    for x in b.values():
        for out in _over(x, (N,)):
            _err(INVALID, M.policy_loss_backward, **b, dnll=out)
    one = T((S,))
    _err(INVALID, M.policy_loss_forward, **a, loss=one, kl=one)
    _err(INVALID, M.policy_loss_forward, **a, loss=one, workspace=T((64,), U8, at=one.data_ptr()))
    a = dict(nll=T((N,)), offsets=T((S + 1,), I32), ref_nll=T((N,)), mask=T((N,), U8))
    for x in a.values():
        for name, m, dt in (("loss", S // 2, F32), ("margins", S // 2, F32), ("reward", S, F32),
                            ("count", S, I32)):
            for out in _over(x, (m,), dt):
                _err(INVALID, M.preference_loss_forward, **a, **{name: out})
        for ws in _over(x, (512,), U8):
            _err(INVALID, M.preference_loss_forward, **a, workspace=ws)
    b = dict(offsets=a["offsets"], margins=T((S // 2,)), count=T((S,), I32), dloss=T((S // 2,)),
             mask=a["mask"])
    for x in b.values():
        for out in _over(x, (N,)):
            _err(INVALID, M.preference_loss_backward, **b, dnll=out)


def test_apart_calls_reach_the_library(monkeypatch):
    # tensors beside each other, and inputs that are the same tensor
    class Reached(Exception):
        pass

    def lib():
        raise Reached

    monkeypatch.setattr(M, "_on", lambda device, stream: M._HERE)
    monkeypatch.setattr(M, "_Launch", lambda dev, stream: (_ for _ in ()).throw(Reached()))
    monkeypatch.setattr(M, "lib", lib)
    nll = T((N,), at=AT)
    dnll = T((N,), at=AT + 4 * N)
    mask = T((N,), BOOL, at=AT + 8 * N)
    count, dloss = T((S,), I32), T((S,))
    a = dict(nll=nll, old_nll=nll, advantages=dloss, offsets=T((S + 1,), I32), ref_nll=nll,
             mask=mask)
    ws = T((512,), U8, at=AT + 9 * N)
    with pytest.raises(Reached):
        M.policy_loss_forward(**a, loss=T((S,)), kl=T((S,)), count=count, clipped=T((S,), I32),
                              workspace=ws)
    with pytest.raises(Reached):
        M.policy_loss_backward(**a, count=count, dloss=dloss, dnll=dnll)
    with pytest.raises(Reached):
        M.preference_loss_backward(a["offsets"], T((S // 2,)), count, T((S // 2,)), mask=mask,
                                   dnll=dnll)
    h = _lists()
    with pytest.raises(Reached):
        M.distill_loss_forward(h["hidden"], h["weight"], h["ids"], h["teacher"], loss=T((6,)),
                               lse=T((6,)), logp=T((6, 5)), workspace=ws)


def test_policy_entry_points_refuse():
    size = M.sequence_loss_workspace_size
    need = size(N, S)
    assert need > 0 and size(0, S) > 0 and size(N, 0) == 0 and size(-1, S) == 0
    assert size(1 << 26, S) == 0 and size(N, -1) == 0 and size(N, (1 << 24) + 1) == 0
    assert size((1 << 26) - 1, 1 << 24) > 0

    def fwd(nll=p, old=p, ref=p, mask=None, adv=p, per=0, off=p, s=S, n=N, lo=0.2, hi=0.2, w=0.1,
            mean=1, loss=p, kl=p, count=p, clipped=p, ws=p, nb=need):
        return _rc("policy_loss_forward", nll, old, ref, mask, adv, per, off, s, n, lo, hi, w, mean,
                   loss, kl, count, clipped, ws, nb, None)

    def bwd(nll=p, old=p, ref=p, mask=None, adv=p, per=0, off=p, s=S, n=N, lo=0.2, hi=0.2, w=0.1,
            mean=1, count=p, dloss=p, dnll=p):
        return _rc("policy_loss_backward", nll, old, ref, mask, adv, per, off, s, n, lo, hi, w,
                   mean, count, dloss, dnll, None)

    for f in (fwd, bwd):
        assert f(n=-1) == SHAPE and f(n=1 << 26) == SHAPE
        assert f(s=-1) == SHAPE and f(s=(1 << 24) + 1) == SHAPE
        for lo in (-0.1, 1.5, math.nan, math.inf):
            assert f(lo=lo) == INVALID
        for hi in (-0.1, math.nan, math.inf):
            assert f(hi=hi) == INVALID
        assert f(w=math.nan) == INVALID and f(w=math.inf) == INVALID
        for k in ("nll", "old", "adv", "off", "ref"):
            assert f(**{k: None}) == INVALID
        assert f(s=0, nll=None, off=None) == M.MUON_OK
    for k in ("loss", "kl", "count", "clipped"):
        assert fwd(**{k: None}) == INVALID
    for k in ("count", "dloss", "dnll"):
        assert bwd(**{k: None}) == INVALID
    assert fwd(ws=None) == WS and fwd(nb=need - 1) == WS and fwd(ws=ctypes.c_void_p(8)) == WS
    assert bwd(n=0, nll=None, old=None, ref=None, dnll=None) == M.MUON_OK


def test_preference_entry_points_refuse():
    need = M.sequence_loss_workspace_size(N, S)

    def fwd(nll=p, ref=None, mask=None, off=p, s=S, n=N, kind=0, beta=0.1, margin=0.0, sm=0.0,
            mean=0, loss=p, x=p, reward=p, count=p, ws=p, nb=need):
        return _rc("preference_loss_forward", nll, ref, mask, off, s, n, kind, beta, margin, sm,
                   mean, loss, x, reward, count, ws, nb, None)

    def bwd(mask=None, off=p, s=S, n=N, kind=0, beta=0.1, sm=0.0, mean=0, x=p, count=p, dloss=p,
            dnll=p):
        return _rc("preference_loss_backward", mask, off, s, n, kind, beta, sm, mean, x, count,
                   dloss, dnll, None)

    for f in (fwd, bwd):
        assert f(n=-1) == SHAPE and f(n=1 << 26) == SHAPE and f(s=5) == SHAPE and f(s=-2) == SHAPE
        assert f(kind=3) == INVALID and f(kind=-1) == INVALID
        assert f(beta=math.nan) == INVALID and f(beta=math.inf) == INVALID
        for sm in (-0.1, 1.1, math.nan):
            assert f(sm=sm) == INVALID
        assert f(sm=0.1, kind=1) == INVALID and f(sm=0.1, kind=2) == INVALID
        assert f(off=None) == INVALID
        assert f(s=0, off=None) == M.MUON_OK
    assert fwd(margin=math.inf) == INVALID and fwd(nll=None) == INVALID
    for k in ("loss", "x", "reward", "count"):
        assert fwd(**{k: None}) == INVALID
    for k in ("x", "count", "dloss", "dnll"):
        assert bwd(**{k: None}) == INVALID
    assert fwd(ws=None) == WS and fwd(nb=need - 1) == WS and fwd(ws=ctypes.c_void_p(8)) == WS
    assert bwd(n=0, dnll=None, x=None) == M.MUON_OK
