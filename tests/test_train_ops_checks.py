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


def test_loss_binding_checks():
    h, w, t = Fake((6, 16)), Fake((100, 16)), Fake((6,), I64)
    f32 = torch.float32
    f = M.lm_loss_forward
    _err(INVALID, f, Fake((6, 16), cuda=False), w, t)
    _err(INVALID, f, h, Fake((100, 16), stride=(1, 100)), t)
    _err(SHAPE, f, h, Fake((1600,)), t)
    _err(SHAPE, f, Fake((6, 17)), w, t)
    _err(SHAPE, f, Fake((5, 16)), w, t)
    _err(DTYPE, f, Fake((6, 16), f32), w, t)
    _err(DTYPE, f, Fake((6, 16), torch.float16), Fake((100, 16), torch.float16), t)
    _err(DTYPE, f, h, w, Fake((6,), f32))
    _err(INVALID, f, h, w, Fake((6,), I64, stride=(2,)))
    _err(INVALID, f, Fake((6, 16), stride=(8, 1)), w, t)
    _err(SHAPE, f, h, w, t, loss=Fake((5,), f32))
    _err(DTYPE, f, h, w, t, lse=Fake((6,)))
    _err(INVALID, f, h, Fake((100, 16), dev="cuda:1"), t)
    b, lse, dl = M.lm_loss_backward, Fake((6,), f32), Fake((6,), f32)
    _err(DTYPE, b, h, w, t, Fake((6,)), dl)
    _err(SHAPE, b, h, w, t, lse, Fake((7,), f32))
    _err(INVALID, b, h, w, t, lse, None)
    _err(SHAPE, b, h, w, t, lse, dl, dhidden=Fake((6, 15)))
    _err(SHAPE, b, h, w, t, lse, dl, dweight=Fake((16, 100)))
    _err(INVALID, b, h, w, t, lse, dl, dweight=Fake((100, 16), stride=(32, 1)))
    _err(DTYPE, b, h, w, t, lse, dl, dweight=Fake((100, 16), torch.float16))
    _err(INVALID, b, h, w, t, lse, dl, accumulate=True)
    _err(INVALID, b, h, w, t, lse, dl, dweight=False, accumulate=True)


def test_loss_entry_points_refuse():
    p = ctypes.c_void_p(256)
    size = M.lm_loss_workspace_size
    need_f, need_b = size(4, 10, 8, "bf16", False), size(4, 10, 8, "bf16")
    assert 0 < need_f <= need_b
    assert size(0, 10, 8, "bf16") == 0 and size(4, 0, 8, "bf16") == 0
    assert size(4, 2 ** 21 + 1, 8, "bf16") == 0
    # the gradient of the logits of one piece, not of all, is held
    assert size(8192, 163840, 7168, "bf16") < 8192 * 163840 * 2 // 2

    def fwd(h=p, ld=8, w=p, dt=1, t=p, t64=1, n=4, vocab=10, dim=8, loss=p, lse=p, ws=p,
            nb=need_f):
        return _rc("lm_loss_forward", h, ld, w, dt, t, t64, n, vocab, dim, loss, lse, ws, nb, None)

    assert fwd(dt=2) == DTYPE and fwd(n=-1) == SHAPE and fwd(vocab=0) == SHAPE
    assert fwd(dim=0, ld=0) == SHAPE and fwd(ld=7) == SHAPE
    assert fwd(vocab=2 ** 21 + 1) == M.MUON_ERR_UNSUPPORTED
    for k in ("h", "w", "t", "loss", "lse"):
        assert fwd(**{k: None}) == INVALID
    assert fwd(ws=None) == WS and fwd(nb=need_f - 1) == WS and fwd(ws=ctypes.c_void_p(8)) == WS
    assert fwd(n=0, h=None, ws=None, nb=0) == M.MUON_OK

    def bwd(h=p, ld=8, w=p, dt=1, t=p, t64=1, n=4, vocab=10, dim=8, lse=p, dl=p, dh=p, dhd=1,
            ldh=8, dw=p, dwd=0, acc=0, ws=p, nb=need_b):
        return _rc("lm_loss_backward", h, ld, w, dt, t, t64, n, vocab, dim, lse, dl, dh, dhd, ldh,
                   dw, dwd, acc, ws, nb, None)

    assert bwd(dt=2) == DTYPE and bwd(dhd=2) == DTYPE and bwd(dwd=-1) == DTYPE
    assert bwd(ldh=7) == SHAPE and bwd(ld=7) == SHAPE and bwd(n=1 << 26) == SHAPE
    for k in ("h", "w", "t", "lse", "dl"):
        assert bwd(**{k: None}) == INVALID
    assert bwd(ws=None) == WS and bwd(nb=need_b - 1) == WS and bwd(ws=ctypes.c_void_p(8)) == WS
    assert bwd(dh=None, dw=None, ws=None, nb=0) == M.MUON_OK
    assert bwd(n=0, dw=None) == M.MUON_OK and bwd(n=0, acc=1) == M.MUON_OK


def test_loss_refuses_more_rows_than_a_launch_holds():
    p = ctypes.c_void_p(256)
    n = (1 << 24) + 1
    assert M.lm_loss_workspace_size(n, 10, 8, "bf16") == 0
    assert M.lm_loss_workspace_size(n - 1, 10, 8, "bf16") > 0
    assert _rc("lm_loss_forward", p, 8, p, 1, p, 1, n, 10, 8, p, p, p, 1 << 40, None) == \
        M.MUON_ERR_UNSUPPORTED
    assert _rc("lm_loss_backward", p, 8, p, 1, p, 1, n, 10, 8, p, p, p, 1, 8, p, 1, 0, p, 1 << 40,
               None) == M.MUON_ERR_UNSUPPORTED


def test_expert_binding_checks():
    x, w, o = Fake((40, 16)), Fake((5, 16, 24)), Fake((6,), torch.int32)
    f = M.expert_matmul
    _err(SHAPE, f, x, Fake((80, 24)), o)
    _err(INVALID, f, x, Fake((5, 16, 24), stride=(400, 24, 1)), o)
    _err(SHAPE, f, Fake((40, 24)), w, o)
    _err(SHAPE, f, x, w, o, trans=True)
    _err(SHAPE, f, Fake((640,)), w, o)
    _err(SHAPE, f, None, w, o)
    _err(DTYPE, f, Fake((40, 16), torch.float32), w, o)
    _err(DTYPE, f, x, w, Fake((6,), I64))
    _err(SHAPE, f, x, w, Fake((5,), torch.int32))
    _err(INVALID, f, x, w, torch.zeros(6, dtype=torch.int32))
    _err(SHAPE, f, x, w, o, out=Fake((40, 16)))
    _err(INVALID, f, x, w, o, out=Fake((40, 24), stride=(1, 40)))
    _err(DTYPE, f, x, w, o, out=Fake((40, 24)), out_dtype="fp32")
    _err(INVALID, f, Fake((40, 16), dev="cuda:1"), w, o)
    g, dw = M.expert_wgrad, Fake((5, 16, 24), torch.float32)
    b = Fake((40, 24))
    _err(SHAPE, g, x, Fake((39, 24)), o, dw)
    _err(SHAPE, g, b, x, o, dw)
    _err(DTYPE, g, x, Fake((40, 24), torch.float32), o, dw)
    _err(DTYPE, g, x, b, o, Fake((5, 16, 24), torch.float16))
    _err(SHAPE, g, x, b, o, Fake((80, 24)))
    _err(SHAPE, g, x, b, Fake((5,), torch.int32), dw)
    _err(INVALID, g, x, b, o, None)
    _err(SHAPE, g, None, b, o, dw)


def test_expert_entry_points_refuse():
    p = ctypes.c_void_p(256)

    def mm(x=p, ldx=16, w=p, dt=1, off=p, e=5, rows=40, k=16, n=24, tr=0, y=p, yd=1, ldy=24):
        return _rc("expert_matmul", x, ldx, w, dt, off, e, rows, k, n, tr, y, yd, ldy, None)

    assert mm(dt=2) == DTYPE and mm(yd=5) == DTYPE
    assert mm(e=0) == SHAPE and mm(e=4097) == SHAPE and mm(rows=-1) == SHAPE
    assert mm(rows=1 << 26) == SHAPE and mm(k=0) == SHAPE and mm(n=0) == SHAPE
    assert mm(k=(1 << 22) + 1, ldx=1 << 23) == SHAPE and mm(ldx=15) == SHAPE and mm(ldy=23) == SHAPE
    for k in ("x", "w", "off", "y"):
        assert mm(**{k: None}) == INVALID
    assert mm(rows=0, x=None, y=None) == M.MUON_OK

    def wg(a=p, lda=16, b=p, ldb=24, dt=1, off=p, e=5, rows=40, m=16, n=24, dw=p, dwd=0, acc=0):
        return _rc("expert_wgrad", a, lda, b, ldb, dt, off, e, rows, m, n, dw, dwd, acc, None)

    assert wg(dt=2) == DTYPE and wg(dwd=2) == DTYPE and wg(lda=15) == SHAPE and wg(ldb=23) == SHAPE
    assert wg(e=0) == SHAPE and wg(rows=1 << 26) == SHAPE and wg(m=0) == SHAPE
    for k in ("a", "b", "off", "dw"):
        assert wg(**{k: None}) == INVALID
    assert wg(rows=0, a=None, b=None, acc=1) == M.MUON_OK


class Placed(Fake):
    """A stand-in at an address of its own."""

    def __init__(self, at, shape, dtype=torch.bfloat16, stride=None):
        super().__init__(shape, dtype, stride)
        self._at = at

    def data_ptr(self):
        return self._at


def test_outputs_that_share_memory_with_inputs_are_refused():
    f32, ids = torch.float32, Fake((6,), I64)
    at = 1 << 20
    table = Placed(at, (100, 16))  # 3200 bytes
    _err(INVALID, M.embed_forward, table, ids, out=Placed(at, (6, 16)))
    _err(INVALID, M.embed_forward, table, ids, out=Placed(at + 3198, (6, 16)))
    _err(INVALID, M.embed_forward, table, ids, out=Placed(at - 190, (6, 16)))
    _err(INVALID, M.embed_forward, table, ids, out=Placed(at - 190, (6, 16), stride=(17, 1)))
    _err(INVALID, M.embed_backward, Placed(at + 64, (6, 16)), ids, table)
    h, t = Placed(at, (6, 16), stride=(48, 1)), ids
    w = Placed(at + 4096, (100, 16))
    lse, dl = Fake((6,), f32), Fake((6,), f32)
    loss = Placed(at, (6,), f32)
    _err(INVALID, M.lm_loss_forward, h, w, t, loss=loss, lse=loss)
    b = M.lm_loss_backward
    _err(INVALID, b, h, w, t, lse, dl, dhidden=h)
    # columns [8, 24) of the buffer whose columns [0, 16) are hidden
    _err(INVALID, b, h, w, t, lse, dl, dhidden=Placed(at + 16, (6, 16), stride=(48, 1)))
    # columns [40, 56): the last ones are the next row's first
    _err(INVALID, b, h, w, t, lse, dl, dhidden=Placed(at + 80, (6, 16), stride=(48, 1)))
    _err(INVALID, b, h, w, t, lse, dl, dhidden=Placed(at + 32, (6, 16), stride=(47, 1)))
    _err(INVALID, b, h, w, t, lse, dl, dweight=w)
    _err(INVALID, b, h, w, t, lse, dl, dhidden=False, dweight=Placed(at + 100, (100, 16)))
    far = 1 << 30
    _err(INVALID, b, h, w, t, lse, dl, dhidden=Placed(far, (6, 16)),
         dweight=Placed(far - 3198, (100, 16)))
    x, o = Placed(at, (40, 24)), Fake((6,), torch.int32)
    w3 = Placed(far, (5, 24, 24))
    _err(INVALID, M.expert_matmul, x, w3, o, out=x)
    _err(INVALID, M.expert_matmul, x, w3, o, trans=True, out=Placed(far + 5758, (40, 24)))
    _err(INVALID, M.expert_wgrad, x, Placed(far, (40, 24)), o, Placed(at - 2, (5, 24, 24), f32))
    _err(INVALID, M.expert_wgrad, x, Placed(far, (40, 24)), o, Placed(far + 1918, (5, 24, 24), f32))


def test_memory_beside_an_input_is_no_overlap():
    at = 1 << 20
    a = Placed(at, (6, 16), stride=(48, 1))

    def apart(p, stride=48, cols=16, rows=6):
        M._apart("out", Placed(p, (rows, cols)), rows, cols, stride, a=(a, 6, 16, 48))

    apart(at + 32)
    apart(at + 64)
    apart(at - 32)
    apart(at - 6 * 96 + 96 - 32)      # before the buffer's first row
    apart(at + 6 * 96 - 64, 16)       # from the byte after the last row
    apart(at, rows=0)
    with pytest.raises(M.MuonError):
        apart(at + 30)
    with pytest.raises(M.MuonError):
        apart(at + 66)
    with pytest.raises(M.MuonError):
        apart(at + 6 * 96 - 66, 16)
