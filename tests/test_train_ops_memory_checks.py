"""Outputs and workspaces of the operators that write gradients share no
memory with index vectors, statistics, matrices or each other: the binding
refuses such calls before any library call (CPU, stand-in tensors).  Nor may a
result have more tiles than a launch holds."""

import ctypes

import pytest
import torch

import muon_newton_schulz_amd as M
from test_train_ops_checks import I64, INVALID, Placed, _err

F32, I32, U8 = torch.float32, torch.int32, torch.uint8
AT = 1 << 20


def _at(k, shape, dtype=torch.bfloat16, stride=None):
    """A tensor in the k-th MiB."""
    return Placed(AT * (k + 1), shape, dtype, stride)


def _over(t, shape, dtype):
    """Tensors that share memory with contiguous t: its start, its last
    element, and from before it into its first."""
    last = t.numel() * t.element_size() - torch.empty(0, dtype=dtype).element_size()
    n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
    for d in (0, last, 1 - n):
        yield Placed(t.data_ptr() + d, shape, dtype)


def _workspaces(*tensors):
    for t in tensors:
        yield from _over(t, (512,), U8)


def test_embed():
    table, ids = _at(0, (100, 16)), _at(1, (60,), I64)
    for out in _over(ids, (60, 16), torch.bfloat16):
        _err(INVALID, M.embed_forward, table, ids, out=out)
    dout, dtable = _at(2, (60, 16)), _at(3, (100, 16))
    for g in _over(ids, (100, 16), torch.bfloat16):
        _err(INVALID, M.embed_backward, dout, ids, g)
    for ws in _workspaces(dout, ids, dtable):
        _err(INVALID, M.embed_backward, dout, ids, dtable, workspace=ws)


def test_loss():
    h, w, t = _at(0, (60, 16)), _at(1, (100, 16)), _at(2, (60,), I64)
    lse, dl = _at(3, (60,), F32), _at(4, (60,), F32)
    dh, dw = _at(5, (60, 16)), _at(6, (100, 16))
    f, b = M.lm_loss_forward, M.lm_loss_backward
    for x in (h, w, t):
        for out in _over(x, (60,), F32):
            _err(INVALID, f, h, w, t, loss=out)
            _err(INVALID, f, h, w, t, lse=out, loss=dl)
    for ws in _workspaces(h, w, t, lse, dl):
        _err(INVALID, f, h, w, t, loss=dl, lse=lse, workspace=ws)
    for x in (t, lse, dl):
        for out in _over(x, (60, 16), torch.bfloat16):
            _err(INVALID, b, h, w, t, lse, dl, dhidden=out, dweight=False)
        for out in _over(x, (100, 16), torch.bfloat16):
            _err(INVALID, b, h, w, t, lse, dl, dhidden=False, dweight=out)
    for ws in _workspaces(h, w, t, lse, dl, dh, dw):
        _err(INVALID, b, h, w, t, lse, dl, dhidden=dh, dweight=dw, workspace=ws)


def test_experts():
    x, w, o = _at(0, (40, 16)), _at(1, (5, 16, 24)), _at(2, (6,), I32)
    for out in _over(o, (40, 24), torch.bfloat16):
        _err(INVALID, M.expert_matmul, x, w, o, out=out)
    for dw in _over(o, (5, 16, 24), F32):
        _err(INVALID, M.expert_wgrad, x, _at(3, (40, 24)), o, dw)


def test_a_vector_between_rows_is_apart():
    # 6 rows of 32 bytes, 96 bytes apart
    rows = Placed(AT, (6, 16), torch.bfloat16, (48, 1))
    block = {"a": (rows, 6, 16, 48)}
    for d, n, fine in ((32, 16, True), (64, 8, True), (96 * 3 + 40, 14, True), (30, 4, False),
                       (32, 17, False), (64, 9, False), (-32, 8, True), (-32, 9, False),
                       (96 * 5 + 32, 300, True), (96 * 5 + 28, 8, False), (0, 400, False)):
        v = Placed(AT + d, (n,), F32)
        for call in (lambda: M._apart("out", v, 1, n, n, **block),
                     lambda: M._apart("out", rows, 6, 16, 48, v=M._vector(v))):
            if fine:
                call()
            else:
                with pytest.raises(M.MuonError):
                    call()


def test_apart_calls_reach_the_library(monkeypatch):
    # tensors beside each other: the checks let them through
    class Reached(Exception):
        pass

    def lib():
        raise Reached

    monkeypatch.setattr(M, "_Launch", lambda dev, stream: (_ for _ in ()).throw(Reached()))
    monkeypatch.setattr(M, "lib", lib)
    table, ids = _at(0, (100, 16)), Placed(AT + 3200, (60,), I64)
    out = Placed(AT + 3200 + 480, (60, 16))
    ws = Placed(AT + 3200 + 480 + 1920, (512,), U8)
    with pytest.raises(Reached):
        M.embed_forward(table, ids, out=out)
    with pytest.raises(Reached):
        M.embed_backward(out, ids, table, workspace=ws)
    lse, dl = _at(3, (60,), F32), Placed(AT * 4 + 240, (60,), F32)
    with pytest.raises(Reached):
        M.lm_loss_forward(out, table, ids, loss=dl, lse=lse, workspace=ws)
    with pytest.raises(Reached):
        M.lm_loss_backward(out, table, ids, lse, dl, dhidden=_at(5, (60, 16)),
                           dweight=_at(6, (100, 16)), workspace=ws)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("trans", [0, 1])
def test_more_tiles_than_a_launch_holds_are_refused(dtype, trans):
    # 4096 experts with a side of 2^22: 4096 x 16384 tiles even of 256 columns
    p, side = ctypes.c_void_p(256), 1 << 22  # never dereferenced
    L = M.lib()
    assert L.expert_matmul(p, 8, p, dtype, p, 4096, 4096, 8, side, trans, p, dtype, side,
                           None) == M.MUON_ERR_UNSUPPORTED
    for m, n in ((8, side), (side, 8)):
        assert L.expert_wgrad(p, m, p, n, dtype, p, 4096, 40, m, n, p, dtype, 0,
                              None) == M.MUON_ERR_UNSUPPORTED
