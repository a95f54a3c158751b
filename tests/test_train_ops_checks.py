"""Refusals of the operators that write gradients, without a GPU: the
binding's checks on stand-in tensors, and the C entry points' own checks,
which come before any HIP call."""

import ctypes

import pytest
import torch

import muon_newton_schulz_amd as M


class Fake:
    """Answers what the binding asks of a GPU tensor, and has no address."""

    def __init__(self, shape, dtype=torch.bfloat16, stride=None, cuda=True, dev="cuda:0"):
        t = torch.empty(0, dtype=dtype)
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, cuda
        self.device = torch.device(dev)
        st, s = [], 1
        for d in reversed(shape):
            st.insert(0, s)
            s *= d
        self._contig = stride is None or list(stride) == st
        self._stride = tuple(st) if stride is None else stride
        self._esize = t.element_size()

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def stride(self, d):
        return self._stride[d]

    def is_contiguous(self):
        return self._contig

    def element_size(self):
        return self._esize

    def data_ptr(self):
        raise AssertionError("the address must not be taken before the checks pass")


def _err(status, fn, *a, **k):
    with pytest.raises(M.MuonError) as e:
        fn(*a, **k)
    assert e.value.status == status, e.value


I64 = torch.int64
INVALID, SHAPE, DTYPE = M.MUON_ERR_INVALID_ARG, M.MUON_ERR_BAD_SHAPE, M.MUON_ERR_BAD_DTYPE
WS = M.MUON_ERR_WORKSPACE_TOO_SMALL


def test_embed_binding_checks():
    table, ids = Fake((100, 16)), Fake((6,), I64)
    f = M.embed_forward
    _err(INVALID, f, Fake((100, 16), cuda=False), ids)
    _err(INVALID, f, Fake((100, 16), stride=(32, 1)), ids)
    _err(SHAPE, f, Fake((1600,)), ids)
    _err(DTYPE, f, Fake((100, 16), torch.float16), ids)
    _err(DTYPE, f, table, Fake((6,), torch.int16))
    _err(INVALID, f, table, Fake((6, 2), I64, stride=(1, 6)))
    _err(SHAPE, f, table, ids, out=Fake((5, 16)))
    _err(SHAPE, f, table, ids, out=Fake((6, 15)))
    _err(INVALID, f, table, ids, out=Fake((6, 16), stride=(15, 1)))
    _err(INVALID, f, table, ids, out=Fake((6, 16), stride=(0, 1)))
    _err(INVALID, f, table, ids, out=Fake((6, 16), stride=(32, 2)))
    _err(DTYPE, f, table, ids, out=Fake((6, 16), torch.float16))
    _err(DTYPE, f, table, ids, out=Fake((6, 16)), out_dtype="fp32")
    _err(DTYPE, f, table, ids, out_dtype="fp16")
    _err(INVALID, f, table, Fake((6,), I64, dev="cuda:1"))
    b, dout = M.embed_backward, Fake((6, 16))
    _err(INVALID, b, None, ids, table)
    _err(INVALID, b, dout, ids, None)
    _err(SHAPE, b, Fake((7, 16)), ids, table)
    _err(SHAPE, b, dout, ids, Fake((100, 17)))
    _err(SHAPE, b, dout, ids, Fake((100 * 16,)))
    _err(INVALID, b, dout, ids, Fake((100, 16), stride=(1, 100)))
    _err(INVALID, b, dout, ids, table, workspace=Fake((10,), torch.uint8, dev="cuda:1"))


def _rc(name, *a):
    return getattr(M.lib(), name)(*a)


def test_embed_entry_points_refuse():
    p = ctypes.c_void_p(256)  # never dereferenced: every call below is refused

    def fwd(table=p, td=1, vocab=10, dim=8, ids=p, i64=1, n=4, scale=1.0, out=p, od=1, ld=8):
        return _rc("embed_forward", table, td, vocab, dim, ids, i64, n, scale, out, od, ld, None)

    assert fwd(td=2) == DTYPE and fwd(od=-1) == DTYPE
    assert fwd(n=-1) == SHAPE and fwd(n=1 << 26) == SHAPE
    assert fwd(vocab=0) == SHAPE and fwd(vocab=2 ** 31 - 1) == SHAPE
    assert fwd(dim=0, ld=0) == SHAPE and fwd(dim=(1 << 24) + 1, ld=1 << 25) == SHAPE
    assert fwd(ld=7) == SHAPE
    assert fwd(scale=float("nan")) == INVALID and fwd(scale=float("inf")) == INVALID
    assert fwd(table=None) == INVALID and fwd(ids=None) == INVALID and fwd(out=None) == INVALID
    assert fwd(n=0, table=None, ids=None, out=None) == M.MUON_OK

    need = M.embed_backward_workspace_size(4, 10, 8)
    assert need > 0 and M.embed_backward_workspace_size(0, 10, 8) == 0
    assert M.embed_backward_workspace_size(-1, 10, 8) == 0
    assert M.embed_backward_workspace_size(4, 0, 8) == 0

    def bwd(dout=p, dd=1, ld=8, ids=p, i64=0, n=4, scale=1.0, g=p, gd=0, vocab=10, dim=8, acc=0,
            ws=p, nb=need):
        return _rc("embed_backward", dout, dd, ld, ids, i64, n, scale, g, gd, vocab, dim, acc, ws,
                   nb, None)

    assert bwd(dd=2) == DTYPE and bwd(gd=3) == DTYPE
    assert bwd(n=1 << 26) == SHAPE and bwd(vocab=0) == SHAPE and bwd(ld=7) == SHAPE
    assert bwd(dout=None) == INVALID and bwd(ids=None) == INVALID and bwd(g=None) == INVALID
    assert bwd(scale=float("inf")) == INVALID
    assert bwd(ws=None) == WS and bwd(nb=need - 1) == WS and bwd(ws=ctypes.c_void_p(128)) == WS
    assert bwd(n=0, acc=1, dout=None, ids=None, ws=None, nb=0) == M.MUON_OK
    assert "n" in M.muon_last_error() or M.muon_last_error()
