"""MI355X-native Muon (Newton-Schulz) and AdamW optimizer step.

Thin ctypes binding over ``libmuon.so`` (C ABI in ``include/muon.h``).  The
functions keep the C names; they only marshal arguments (tensor ->
device pointer, dtype -> code, current torch stream -> hipStream_t) and
turn status codes into ``MuonError``.  Every step of the optimizer runs in
the library's HIP kernels; there is no Python or CPU fallback: if the
library is missing, every call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmuon.so")

MUON_OK = 0
MUON_ERR_INVALID_ARG = -1
MUON_ERR_BAD_SHAPE = -2
MUON_ERR_OVERLAP = -3
MUON_ERR_WORKSPACE_TOO_SMALL = -4
MUON_ERR_BAD_DTYPE = -5
MUON_ERR_HIP = -6
MUON_ERR_UNSUPPORTED = -7

MUON_DTYPE_FP32 = 0
MUON_DTYPE_BF16 = 1
MUON_DTYPE_FP16 = 2

EXPORTED = [
    "muon_workspace_size", "muon_plan_create", "muon_plan_create_ex", "muon_plan_destroy",
    "muon_plan_get_info", "muon_plan_table_bytes", "muon_plan_upload",
    "muon_step", "muon_step_noalloc", "muon_stage_momentum", "muon_stage_ns_phase",
    "muon_stage_apply",
    "muon_stage_ns_apply",
    "muon_stage_export_x", "muon_stage_export_norms", "adamw_step", "adamw_step_ex",
    "muon_status_string",
    "muon_last_error", "grad_norm_clip_workspace_size", "grad_norm_clip",
    "state_stats_workspace_size", "state_stats",
    "muon_clip_plan_create", "muon_clip_plan_destroy", "muon_clip_plan_table_bytes",
    "muon_clip_plan_upload", "muon_clip",
    "embed_forward", "embed_backward", "embed_backward_workspace_size",
    "lm_loss_workspace_size", "lm_loss_forward", "lm_loss_backward",
    "expert_matmul", "expert_wgrad",
]

MUON_CLIP_FROBENIUS = 0
MUON_CLIP_MAX_LOGIT = 1
# size of the library's static device workspace (muon_step_noalloc)
MUON_NOALLOC_WORKSPACE_BYTES = 256 << 20


class MuonError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[{status}] {message}")
        self.status = status


class MuonMatrix(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_int64), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32)]


class MuonHParamsC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("momentum", ctypes.c_float), ("nesterov", ctypes.c_int32),
                ("ns_a", ctypes.c_float), ("ns_b", ctypes.c_float), ("ns_c", ctypes.c_float),
                ("ns_steps", ctypes.c_int32), ("eps", ctypes.c_float),
                ("scale_mode", ctypes.c_int32), ("rms_target", ctypes.c_float),
                ("clip", ctypes.c_void_p)]


class AdamWHParamsC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("clip", ctypes.c_void_p)]


class MuonClipState(ctypes.Structure):
    """Host view of muon_clip_state_t (the device copy lives in a 16-byte tensor)."""
    _fields_ = [("norm", ctypes.c_float), ("scale", ctypes.c_float), ("skip", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MuonGradBuffer(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MuonStateStats(ctypes.Structure):
    """Host view of muon_state_stats_t."""
    _fields_ = [("mean", ctypes.c_double), ("var", ctypes.c_double), ("min", ctypes.c_double),
                ("max", ctypes.c_double), ("absmax", ctypes.c_double),
                ("count", ctypes.c_int64), ("nonfinite", ctypes.c_int64)]


class MuonClipTarget(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_int64), ("ld", ctypes.c_int64), ("rows", ctypes.c_int32),
                ("cols", ctypes.c_int32), ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MuonPlanInfo(ctypes.Structure):
    _fields_ = [("n_mats", ctypes.c_int32), ("n_waves", ctypes.c_int32),
                ("tile", ctypes.c_int32), ("ns_dtype", ctypes.c_int32),
                ("k1_tiles", ctypes.c_int64), ("syrk_tiles", ctypes.c_int64),
                ("bx_tiles", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t),
                ("ns_flops_per_iter_alg", ctypes.c_double), ("small_mats", ctypes.c_int32),
                ("split_tile_mats", ctypes.c_int32), ("fused_apply_mats", ctypes.c_int32),
                ("round_sync_phases", ctypes.c_int32)]


_lib_handle = None


def lib() -> ctypes.CDLL:
    """Load libmuon.so (raises if it has not been built)."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m muon_newton_schulz_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    mats_p = ctypes.POINTER(MuonMatrix)
    L.muon_workspace_size.argtypes = [mats_p, I32, I64, I32, I32, I32, SZ, ctypes.POINTER(SZ)]
    L.muon_plan_create.argtypes = [mats_p, I32, I64, I32, I32, I32, SZ, ctypes.POINTER(P),
                                   ctypes.POINTER(SZ)]
    L.muon_plan_create_ex.argtypes = [mats_p, I32, I64, I32, I32, I32, SZ, ctypes.c_uint32,
                                      ctypes.POINTER(P), ctypes.POINTER(SZ)]
    L.muon_plan_destroy.argtypes = [P]
    L.muon_plan_destroy.restype = None
    L.muon_plan_get_info.argtypes = [P, ctypes.POINTER(MuonPlanInfo)]
    L.muon_plan_table_bytes.argtypes = [P]
    L.muon_plan_table_bytes.restype = SZ
    L.muon_plan_upload.argtypes = [P, P, SZ, P]
    hp_p = ctypes.POINTER(MuonHParamsC)
    L.muon_step.argtypes = [P, P, P, P, P, SZ, hp_p, P, P]
    L.muon_step_noalloc.argtypes = [P, P, P, P, hp_p, P, P]
    L.muon_stage_momentum.argtypes = [P, I32, P, P, P, SZ, hp_p, P]
    L.muon_stage_ns_phase.argtypes = [P, I32, P, SZ, hp_p, I32, I32, P]
    L.muon_stage_apply.argtypes = [P, I32, P, P, SZ, hp_p, P, P]
    L.muon_stage_ns_apply.argtypes = [P, I32, P, P, SZ, hp_p, P]
    L.muon_stage_export_x.argtypes = [P, I32, P, SZ, I32, P, P]
    L.muon_stage_export_norms.argtypes = [P, I32, P, SZ, P, P]
    L.adamw_step.argtypes = [P, I32, P, P, I32, P, P, I64, ctypes.POINTER(AdamWHParamsC), I64, P]
    L.adamw_step_ex.argtypes = [P, I32, P, P, I32, P, I32, P, I32, I64,
                                ctypes.POINTER(AdamWHParamsC), I64, P]
    L.grad_norm_clip_workspace_size.argtypes = [I32]
    L.grad_norm_clip_workspace_size.restype = SZ
    L.grad_norm_clip.argtypes = [ctypes.POINTER(MuonGradBuffer), I32, ctypes.c_float,
                                 ctypes.c_float, P, SZ, P, P]
    L.state_stats_workspace_size.argtypes = []
    L.state_stats_workspace_size.restype = SZ
    L.state_stats.argtypes = [P, I64, P, SZ, P, P]
    L.muon_clip_plan_create.argtypes = [ctypes.POINTER(MuonClipTarget), I32, I64, I32, I32,
                                        ctypes.POINTER(P), ctypes.POINTER(SZ)]
    L.muon_clip_plan_destroy.argtypes = [P]
    L.muon_clip_plan_destroy.restype = None
    L.muon_clip_plan_table_bytes.argtypes = [P]
    L.muon_clip_plan_table_bytes.restype = SZ
    L.muon_clip_plan_upload.argtypes = [P, P, SZ, P]
    L.muon_clip.argtypes = [P, P, I32, ctypes.c_float, P, P, SZ, P, P, P]
    F = ctypes.c_float
    L.embed_forward.argtypes = [P, I32, I64, I64, P, I32, I64, F, P, I32, I64, P]
    L.embed_backward_workspace_size.argtypes = [I64, I64, I64]
    L.embed_backward_workspace_size.restype = SZ
    L.embed_backward.argtypes = [P, I32, I64, P, I32, I64, F, P, I32, I64, I64, I32, P, SZ, P]
    L.lm_loss_workspace_size.argtypes = [I64, I64, I64, I32, I32]
    L.lm_loss_workspace_size.restype = SZ
    L.lm_loss_forward.argtypes = [P, I64, P, I32, P, I32, I64, I64, I64, P, P, P, SZ, P]
    L.lm_loss_backward.argtypes = [P, I64, P, I32, P, I32, I64, I64, I64, P, P, P, I32, I64, P,
                                   I32, I32, P, SZ, P]
    L.expert_matmul.argtypes = [P, I64, P, I32, P, I32, I64, I64, I64, I32, P, I32, I64, P]
    L.expert_wgrad.argtypes = [P, I64, P, I64, I32, P, I32, I64, I64, I64, P, I32, I32, P]
    L.muon_status_string.argtypes = [I32]
    L.muon_status_string.restype = ctypes.c_char_p
    L.muon_last_error.argtypes = []
    L.muon_last_error.restype = ctypes.c_char_p
    for name in EXPORTED:
        if name not in ("muon_plan_destroy", "muon_clip_plan_destroy", "muon_status_string",
                        "muon_last_error", "muon_plan_table_bytes", "muon_clip_plan_table_bytes",
                        "grad_norm_clip_workspace_size", "state_stats_workspace_size",
                        "embed_backward_workspace_size", "lm_loss_workspace_size"):
            getattr(L, name).restype = ctypes.c_int
    _lib_handle = L
    return L


def _check(rc: int) -> None:
    if rc != MUON_OK:
        msg = lib().muon_last_error().decode(errors="replace")
        raise MuonError(rc, msg or muon_status_string(rc))


def muon_status_string(status: int) -> str:
    return lib().muon_status_string(status).decode()


def muon_last_error() -> str:
    return lib().muon_last_error().decode(errors="replace")


# ---------------------------------------------------------------- marshalling

_dtype_codes = {"fp32": MUON_DTYPE_FP32, "bf16": MUON_DTYPE_BF16, "fp16": MUON_DTYPE_FP16}


def dtype_code(dt) -> int:
    code = _dtype_codes.get(dt)
    if code is None:
        import torch
        _dtype_codes.update({torch.float32: MUON_DTYPE_FP32, torch.bfloat16: MUON_DTYPE_BF16,
                             torch.float16: MUON_DTYPE_FP16})
        code = _dtype_codes.get(dt)
        if code is None:
            raise MuonError(MUON_ERR_BAD_DTYPE, f"unsupported dtype {dt}")
    return code


def _mats_array(mats: Sequence[Tuple[int, int, int]]):
    arr = (MuonMatrix * max(1, len(mats)))()
    for k, (o, r, c) in enumerate(mats):
        arr[k] = MuonMatrix(int(o), int(r), int(c))
    return arr


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def _buf(t, name: str, min_numel: int = 0, dtypes=None, optional: bool = False):
    """Checks a tensor before its address crosses the C ABI, which cannot
    see sizes: a GPU tensor, contiguous, with at least ``min_numel``
    elements of an allowed dtype.  Returns it."""
    if t is None:
        if optional:
            return None
        raise MuonError(MUON_ERR_INVALID_ARG, f"{name} is None")
    if not getattr(t, "is_cuda", False):
        raise MuonError(MUON_ERR_INVALID_ARG, f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise MuonError(MUON_ERR_INVALID_ARG, f"{name} must be contiguous")
    if t.numel() < min_numel:
        raise MuonError(MUON_ERR_INVALID_ARG,
                        f"{name} has {t.numel()} elements, needs at least {min_numel}")
    if dtypes is not None and dtype_code(t.dtype) not in dtypes:
        raise MuonError(MUON_ERR_BAD_DTYPE, f"{name} has dtype {t.dtype}")
    return t


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _hp(hp, clip=None) -> MuonHParamsC:
    if isinstance(hp, MuonHParamsC):
        h = MuonHParamsC.from_buffer_copy(hp)
    else:
        h = MuonHParamsC(float(hp.lr), float(hp.weight_decay), float(hp.momentum),
                         int(bool(hp.nesterov)), float(hp.ns_a), float(hp.ns_b),
                         float(hp.ns_c), int(hp.ns_steps), float(hp.eps), int(hp.scale_mode),
                         float(hp.rms_target))
    if clip is not None:
        h.clip = _ptr(clip)
    return h


def _ahp(hp, clip=None) -> AdamWHParamsC:
    if isinstance(hp, AdamWHParamsC):
        h = AdamWHParamsC.from_buffer_copy(hp)
    else:
        h = AdamWHParamsC(float(hp.lr), float(hp.beta1), float(hp.beta2), float(hp.eps),
                          float(hp.weight_decay))
    if clip is not None:
        h.clip = _ptr(clip)
    return h


# ---------------------------------------------------------------- plan

class MuonPlan:
    """Owns a muon_plan_t (destroyed with the object) and, once uploaded, the
    device tensor holding its tables."""

    def __init__(self, handle: int, workspace_bytes: int, n_mats: int, flat_numel: int = 0,
                 param_dtype: int = MUON_DTYPE_BF16, grad_dtype: int = MUON_DTYPE_BF16):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.n_mats = n_mats
        self.flat_numel = flat_numel
        self.param_dtype = param_dtype
        self.grad_dtype = grad_dtype
        self.tables = None

    @property
    def table_bytes(self) -> int:
        return muon_plan_table_bytes(self)

    def upload(self, device=None, stream=None) -> None:
        """Allocate the table buffer on ``device`` (torch's current device if
        None) and copy the tables into it on ``stream`` (current stream)."""
        import torch
        dev = torch.device("cuda") if device is None else torch.device(device)
        tables = torch.empty(max(1, self.table_bytes), dtype=torch.uint8, device=dev)
        with torch.cuda.device(tables.device):
            muon_plan_upload(self, tables, stream)
        self.tables = tables

    def info(self) -> MuonPlanInfo:
        return muon_plan_get_info(self)

    def alloc_workspace(self, device="cuda"):
        import torch
        return torch.empty(max(1, self.workspace_bytes), dtype=torch.uint8, device=device)

    def close(self):
        if self.handle:
            lib().muon_plan_destroy(ctypes.c_void_p(self.handle))
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def muon_workspace_size(mats, flat_numel: int, param_dtype, grad_dtype, ns_dtype,
                        workspace_cap: int = 0) -> int:
    arr = _mats_array(mats)
    out = ctypes.c_size_t(0)
    _check(lib().muon_workspace_size(arr, len(mats), int(flat_numel), dtype_code(param_dtype),
                                     dtype_code(grad_dtype), dtype_code(ns_dtype),
                                     int(workspace_cap), ctypes.byref(out)))
    return out.value


MUON_PLAN_TILED_ONLY = 1
MUON_PLAN_WHOLE_TILES = 2
MUON_PLAN_FREE_ROUNDS = 4


def muon_plan_create(mats, flat_numel: int, param_dtype, grad_dtype, ns_dtype="bf16",
                     workspace_cap: int = 0, tiled_only: bool = False,
                     whole_tiles: bool = False, free_rounds: bool = False,
                     upload: bool = True) -> MuonPlan:
    """tiled_only: every matrix on the tiled NS path (no fused small-matrix
    kernel); whole_tiles: every NS tile computed whole (no split diagonal
    or edge tiles); free_rounds: the NS kernels never hold an XCD's tile
    rounds together.  Results are bitwise the same either way.
    upload: copy the tables to a new device tensor on torch's current device
    and stream (MuonPlan.upload); without it the plan stays host-only."""
    arr = _mats_array(mats)
    h = ctypes.c_void_p(0)
    ws = ctypes.c_size_t(0)
    _check(lib().muon_plan_create_ex(arr, len(mats), int(flat_numel), dtype_code(param_dtype),
                                     dtype_code(grad_dtype), dtype_code(ns_dtype),
                                     int(workspace_cap),
                                     (MUON_PLAN_TILED_ONLY if tiled_only else 0)
                                     | (MUON_PLAN_WHOLE_TILES if whole_tiles else 0)
                                     | (MUON_PLAN_FREE_ROUNDS if free_rounds else 0),
                                     ctypes.byref(h), ctypes.byref(ws)))
    plan = MuonPlan(h.value, ws.value, len(mats), int(flat_numel), dtype_code(param_dtype),
                    dtype_code(grad_dtype))
    if upload:
        plan.upload()
    return plan


def muon_plan_destroy(plan: MuonPlan) -> None:
    plan.close()


def muon_plan_table_bytes(plan: MuonPlan) -> int:
    return int(lib().muon_plan_table_bytes(ctypes.c_void_p(plan.handle)))


def muon_plan_upload(plan: MuonPlan, tables, stream=None) -> None:
    """tables: a uint8 GPU tensor of at least muon_plan_table_bytes bytes,
    kept alive by the caller while the plan is used (MuonPlan.upload keeps
    it on the plan)."""
    _buf(tables, "tables", muon_plan_table_bytes(plan))
    _check(lib().muon_plan_upload(ctypes.c_void_p(plan.handle), _ptr(tables), _nbytes(tables),
                                  _stream(stream)))


def muon_plan_get_info(plan: MuonPlan) -> MuonPlanInfo:
    info = MuonPlanInfo()
    _check(lib().muon_plan_get_info(ctypes.c_void_p(plan.handle), ctypes.byref(info)))
    return info


F32 = (MUON_DTYPE_FP32,)


def _flat_args(plan: MuonPlan, params=None, grads=None, momentum=None, out_update=None):
    n = plan.flat_numel
    if params is not None:
        _buf(params, "params", n, (plan.param_dtype,))
    if grads is not None:
        _buf(grads, "grads", n, (plan.grad_dtype,))
    if momentum is not None:
        _buf(momentum, "momentum", n, F32)
    _buf(out_update, "out_update", n, F32, optional=True)


def muon_step(plan: MuonPlan, params, grads, momentum, workspace, hp, out_update=None,
              stream=None, clip=None) -> None:
    """clip: optional device clip state from grad_norm_clip (scale and guard)."""
    _flat_args(plan, _buf(params, "params"), _buf(grads, "grads"), _buf(momentum, "momentum"),
               out_update)
    _buf(workspace, "workspace")
    h = _hp(hp, clip)
    _check(lib().muon_step(ctypes.c_void_p(plan.handle), _ptr(params), _ptr(grads),
                           _ptr(momentum), _ptr(workspace), _nbytes(workspace), ctypes.byref(h),
                           _ptr(out_update), _stream(stream)))


def muon_step_noalloc(plan: MuonPlan, params, grads, momentum, hp, out_update=None,
                      stream=None, clip=None) -> None:
    """muon_step on the library's static device workspace (no workspace
    argument, nothing allocated); the plan's workspace_bytes must be at most
    MUON_NOALLOC_WORKSPACE_BYTES (create it with that workspace_cap)."""
    _flat_args(plan, _buf(params, "params"), _buf(grads, "grads"), _buf(momentum, "momentum"),
               out_update)
    h = _hp(hp, clip)
    _check(lib().muon_step_noalloc(ctypes.c_void_p(plan.handle), _ptr(params), _ptr(grads),
                                   _ptr(momentum), ctypes.byref(h), _ptr(out_update),
                                   _stream(stream)))


def muon_stage_momentum(plan: MuonPlan, wave: int, grads, momentum, workspace, hp,
                        stream=None, clip=None) -> None:
    _flat_args(plan, grads=_buf(grads, "grads"), momentum=_buf(momentum, "momentum"))
    _buf(workspace, "workspace")
    h = _hp(hp, clip)
    _check(lib().muon_stage_momentum(ctypes.c_void_p(plan.handle), wave, _ptr(grads),
                                     _ptr(momentum), _ptr(workspace), _nbytes(workspace),
                                     ctypes.byref(h), _stream(stream)))


def muon_stage_ns_phase(plan: MuonPlan, wave: int, workspace, hp, iter: int, phase: int,
                        stream=None) -> None:
    _buf(workspace, "workspace")
    h = _hp(hp)
    _check(lib().muon_stage_ns_phase(ctypes.c_void_p(plan.handle), wave, _ptr(workspace),
                                     _nbytes(workspace), ctypes.byref(h), iter, phase,
                                     _stream(stream)))


def muon_stage_apply(plan: MuonPlan, wave: int, params, workspace, hp, out_update=None,
                     stream=None, clip=None) -> None:
    _flat_args(plan, params=_buf(params, "params"), out_update=out_update)
    _buf(workspace, "workspace")
    h = _hp(hp, clip)
    _check(lib().muon_stage_apply(ctypes.c_void_p(plan.handle), wave, _ptr(params),
                                  _ptr(workspace), _nbytes(workspace), ctypes.byref(h),
                                  _ptr(out_update), _stream(stream)))


def muon_stage_ns_apply(plan: MuonPlan, wave: int, params, workspace, hp, stream=None,
                        clip=None) -> None:
    """Phase 3 of the last NS iteration with the update applied: bitwise
    muon_stage_ns_phase(..., ns_steps - 1, 3) then muon_stage_apply(...)."""
    _flat_args(plan, params=_buf(params, "params"))
    _buf(workspace, "workspace")
    h = _hp(hp, clip)
    _check(lib().muon_stage_ns_apply(ctypes.c_void_p(plan.handle), wave, _ptr(params),
                                     _ptr(workspace), _nbytes(workspace), ctypes.byref(h),
                                     _stream(stream)))


def muon_stage_export_x(plan: MuonPlan, wave: int, workspace, iter_done: int, out,
                        stream=None) -> None:
    """out: fp32, flat_numel elements (the wave's matrices at their offsets)."""
    _buf(workspace, "workspace")
    _buf(out, "out", plan.flat_numel, F32)
    _check(lib().muon_stage_export_x(ctypes.c_void_p(plan.handle), wave, _ptr(workspace),
                                     _nbytes(workspace), iter_done, _ptr(out), _stream(stream)))


def muon_stage_export_norms(plan: MuonPlan, wave: int, workspace, out, stream=None) -> None:
    """out: fp32, at least as many elements as the wave has matrices."""
    _buf(workspace, "workspace")
    _buf(out, "out", 1 if plan.n_mats else 0, F32)
    _check(lib().muon_stage_export_norms(ctypes.c_void_p(plan.handle), wave, _ptr(workspace),
                                         _nbytes(workspace), _ptr(out), _stream(stream)))


def adamw_step(params, master, grads, exp_avg, exp_avg_sq, hp, step: int, stream=None,
               clip=None) -> None:
    """params/grads may be bf16 or fp32 tensors; master (fp32) may be None;
    exp_avg may be fp32 or bf16 and exp_avg_sq fp32, bf16 or fp16 (the
    compressed states of adamw_step_ex); clip: optional device clip state
    from grad_norm_clip."""
    n = _buf(params, "params").numel()
    for name, t in (("grads", grads), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq),
                    ("master", master)):
        _buf(t, name, optional=name == "master")
        if t is not None and t.numel() != n:
            raise MuonError(MUON_ERR_INVALID_ARG, f"{name} has {t.numel()} elements, expected {n}")
    h = _ahp(hp, clip)
    _check(lib().adamw_step_ex(_ptr(params), dtype_code(params.dtype), _ptr(master), _ptr(grads),
                               dtype_code(grads.dtype), _ptr(exp_avg), dtype_code(exp_avg.dtype),
                               _ptr(exp_avg_sq), dtype_code(exp_avg_sq.dtype), n,
                               ctypes.byref(h), int(step), _stream(stream)))


# ------------------------------------------ clipping, step guard, statistics

def grad_norm_clip_workspace_size(n_bufs: int) -> int:
    return int(lib().grad_norm_clip_workspace_size(int(n_bufs)))


def grad_norm_clip(grads: Sequence, max_norm: float, eps: float = 1e-6, out=None,
                   workspace=None, stream=None):
    """Global gradient norm over the given tensors, clip scale and skip flag,
    written to ``out`` (a 16-byte device tensor, allocated if None) and
    returned; pass it as ``clip=`` to the steps of the same iteration."""
    import torch
    bufs = (MuonGradBuffer * max(1, len(grads)))()
    dev = None
    for k, g in enumerate(grads):
        _buf(g, f"grads[{k}]")
        dev = g.device
    dev = dev if dev is not None else torch.device("cuda")
    if out is None:
        out = torch.zeros(16, dtype=torch.uint8, device=dev)
    if _nbytes(_buf(out, "out")) < ctypes.sizeof(MuonClipState):
        raise MuonError(MUON_ERR_INVALID_ARG, "out: 16 bytes of device memory")
    need = grad_norm_clip_workspace_size(len(grads))
    if workspace is None:
        workspace = torch.empty(max(8, need), dtype=torch.uint8, device=dev)
    _buf(workspace, "workspace")
    for k, g in enumerate(grads):
        bufs[k] = MuonGradBuffer(_ptr(g), int(g.numel()), dtype_code(g.dtype), 0)
    _check(lib().grad_norm_clip(bufs, len(grads), float(max_norm), float(eps),
                                _ptr(workspace), _nbytes(workspace), _ptr(out),
                                _stream(stream)))
    return out


def read_clip_state(out) -> dict:
    """Copy a device clip state to the host (synchronises)."""
    c = MuonClipState.from_buffer_copy(bytes(out.cpu().numpy().tobytes()))
    return {"norm": c.norm, "scale": c.scale, "skip": bool(c.skip)}


def state_stats_workspace_size() -> int:
    return int(lib().state_stats_workspace_size())


def state_stats(x, out=None, workspace=None, stream=None):
    """Statistics of a fp32 state tensor into ``out`` (a 56-byte device
    tensor, allocated if None), returned."""
    import torch
    _buf(x, "x", dtypes=F32)
    if out is None:
        out = torch.zeros(ctypes.sizeof(MuonStateStats), dtype=torch.uint8, device=x.device)
    if _nbytes(_buf(out, "out")) < ctypes.sizeof(MuonStateStats):
        raise MuonError(MUON_ERR_INVALID_ARG, "out: 56 bytes of device memory")
    if workspace is None:
        workspace = torch.empty(state_stats_workspace_size(), dtype=torch.uint8, device=x.device)
    _check(lib().state_stats(_ptr(x), int(x.numel()), _ptr(_buf(workspace, "workspace")),
                             _nbytes(workspace), _ptr(out), _stream(stream)))
    return out


def read_state_stats(out) -> dict:
    """Copy device statistics to the host (synchronises)."""
    s = MuonStateStats.from_buffer_copy(bytes(out.cpu().numpy().tobytes()))
    return {k: getattr(s, k) for k, _ in MuonStateStats._fields_}


# ---------------------------------------------------------------- MuonClip

class MuonClipPlan:
    """Owns a muon_clip_plan_t (destroyed with the object) and, once uploaded,
    the device tensor holding its tables."""

    def __init__(self, handle: int, workspace_bytes: int, n_targets: int, n_groups: int,
                 flat_numel: int, param_dtype: int):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.n_targets = n_targets
        self.n_groups = n_groups
        self.flat_numel = flat_numel
        self.param_dtype = param_dtype
        self.tables = None

    def upload(self, device=None, stream=None) -> None:
        import torch
        dev = torch.device("cuda") if device is None else torch.device(device)
        nb = int(lib().muon_clip_plan_table_bytes(ctypes.c_void_p(self.handle)))
        tables = torch.empty(max(1, nb), dtype=torch.uint8, device=dev)
        with torch.cuda.device(tables.device):
            _check(lib().muon_clip_plan_upload(ctypes.c_void_p(self.handle), _ptr(tables),
                                               _nbytes(tables), _stream(stream)))
        self.tables = tables

    def alloc_workspace(self, device="cuda"):
        import torch
        return torch.empty(max(8, self.workspace_bytes), dtype=torch.uint8, device=device)

    def close(self):
        if self.handle:
            lib().muon_clip_plan_destroy(ctypes.c_void_p(self.handle))
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def muon_clip_plan_create(targets, flat_numel: int, param_dtype, n_groups: int = 0,
                          upload: bool = True) -> MuonClipPlan:
    """targets: (offset, rows, cols[, ld[, group]]) per block (ld defaults
    to cols, group to 0).  upload: copy the tables to a new device tensor on
    torch's current device and stream."""
    arr = (MuonClipTarget * max(1, len(targets)))()
    for i, t in enumerate(targets):
        off, rows, cols = int(t[0]), int(t[1]), int(t[2])
        ld = int(t[3]) if len(t) > 3 else cols
        group = int(t[4]) if len(t) > 4 else 0
        arr[i] = MuonClipTarget(off, ld, rows, cols, group, 0)
    h = ctypes.c_void_p(0)
    ws = ctypes.c_size_t(0)
    pd = dtype_code(param_dtype)
    _check(lib().muon_clip_plan_create(arr, len(targets), int(flat_numel), pd, int(n_groups),
                                       ctypes.byref(h), ctypes.byref(ws)))
    plan = MuonClipPlan(h.value, ws.value, len(targets), int(n_groups), int(flat_numel), pd)
    if upload:
        plan.upload()
    return plan


def muon_clip(plan: MuonClipPlan, params, mode, tau: float, max_logits=None, workspace=None,
              norms_out=None, scales_out=None, stream=None) -> None:
    """MuonClip in place on ``params`` (the flat buffer the plan describes).
    mode: "frobenius" / MUON_CLIP_FROBENIUS or "max_logit" / MUON_CLIP_MAX_LOGIT."""
    m = {"frobenius": MUON_CLIP_FROBENIUS, "max_logit": MUON_CLIP_MAX_LOGIT}.get(mode, mode)
    _buf(params, "params", plan.flat_numel, (plan.param_dtype,))
    if m == MUON_CLIP_MAX_LOGIT:
        _buf(max_logits, "max_logits", plan.n_groups, F32)
    _buf(norms_out, "norms_out", plan.n_targets, F32, optional=True)
    _buf(scales_out, "scales_out", plan.n_targets, F32, optional=True)
    if workspace is None and m == MUON_CLIP_FROBENIUS:
        workspace = plan.alloc_workspace(params.device)
    _buf(workspace, "workspace", optional=True)
    _check(lib().muon_clip(ctypes.c_void_p(plan.handle), _ptr(params), int(m), float(tau),
                           _ptr(max_logits), _ptr(workspace),
                           _nbytes(workspace) if workspace is not None else 0,
                           _ptr(norms_out), _ptr(scales_out), _stream(stream)))


# ------------------------------------------- operators that write gradients
#
# They take tensors of one GPU, which need not be torch's current device, and
# run on that GPU's current stream unless ``stream`` names another of its
# streams.  What a call allocates (outputs and workspaces left out) belongs
# to the stream the call runs on.
#
# Like the steps, they are no autograd functions: nothing is recorded, tensors
# that require gradients are read as they are, and an output has no graph.  A
# program calls each gradient itself (or from its own autograd.Function).

TRAIN = (MUON_DTYPE_FP32, MUON_DTYPE_BF16)


def _rows(t, name: str, rows: int, cols: int, dtypes=TRAIN):
    """A GPU tensor of ``rows`` x ``cols`` whose rows are contiguous, with any
    row stride of at least ``cols``.  Returns the row stride."""
    if t is None:
        raise MuonError(MUON_ERR_INVALID_ARG, f"{name} is None")
    if not getattr(t, "is_cuda", False):
        raise MuonError(MUON_ERR_INVALID_ARG, f"{name} must be a GPU tensor")
    if tuple(t.shape) != (rows, cols):
        raise MuonError(MUON_ERR_BAD_SHAPE,
                        f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    if dtype_code(t.dtype) not in dtypes:
        raise MuonError(MUON_ERR_BAD_DTYPE, f"{name} has dtype {t.dtype}")
    if cols > 1 and t.stride(1) != 1:
        raise MuonError(MUON_ERR_INVALID_ARG, f"{name}: a row's elements must be contiguous")
    if rows <= 1:
        return cols
    if t.stride(0) < cols:
        raise MuonError(MUON_ERR_INVALID_ARG, f"{name}: rows overlap (row stride {t.stride(0)})")
    return t.stride(0)


def _block(t, name: str, shape, dtypes=TRAIN):
    """A contiguous GPU tensor of exactly ``shape``."""
    _buf(t, name, dtypes=dtypes)
    if tuple(t.shape) != tuple(shape):
        raise MuonError(MUON_ERR_BAD_SHAPE,
                        f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _index(t, name: str, numel: Optional[int] = None) -> int:
    """A contiguous GPU tensor of int32 or int64.  Returns 1 for int64."""
    import torch
    _buf(t, name)
    if t.dtype not in (torch.int32, torch.int64):
        raise MuonError(MUON_ERR_BAD_DTYPE, f"{name} must be int32 or int64, has {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise MuonError(MUON_ERR_BAD_SHAPE, f"{name} has {t.numel()} elements, expected {numel}")
    return int(t.dtype == torch.int64)


def _one_device(**tensors):
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise MuonError(MUON_ERR_INVALID_ARG, f"{name} is on {t.device}, others on {dev}")
    return dev


def _apart(name: str, out, rows: int, cols: int, ld: int, **inputs):
    """Refuses an output of ``rows`` x ``cols``, row stride ``ld``, that shares
    memory with an input, given as (tensor, rows, cols, row stride): the
    kernels read inputs after they have written outputs.  Columns of one
    buffer beside each other are apart, and so is a vector (one row) that
    lies between two rows' columns."""
    e = out.element_size()
    a, row, step = out.data_ptr(), cols * e, ld * e
    end = a + (rows - 1) * step + row
    for other, (t, r, c, l) in inputs.items():
        if r == 0 or rows == 0:
            continue
        b, e = t.data_ptr(), t.element_size()
        if b >= end or a >= b + ((r - 1) * l + c) * e:
            continue
        if rows > 1 and (r == 1 or l * e == step):
            gap = (b - a) % step
            if gap >= row and gap + c * e <= step:
                continue
        elif rows == 1 and r > 1:
            gap = (a - b) % (l * e)
            if gap >= c * e and gap + row <= l * e:
                continue
        raise MuonError(MUON_ERR_INVALID_ARG, f"{name} shares memory with {other}")


def _vector(t):
    """A contiguous tensor as _apart takes it."""
    n = t.numel()
    return t, 1, n, n


def _apart_workspace(workspace, **tensors):
    """Refuses a caller's workspace that shares memory with a tensor of the
    call."""
    if workspace is not None:
        _buf(workspace, "workspace")
        _apart("workspace", *_vector(workspace), **tensors)


def _current_handle(dev) -> int:
    """hipStream_t of the current stream of ``dev`` (the raw query where torch
    has it: the Stream object costs more than the rest of a small call)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev.index) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


class _Launch:
    """Makes ``dev`` current, and ``stream`` (if given) the stream that torch
    allocates on, around one call; ``handle`` is the hipStream_t."""

    __slots__ = ("handle", "_dev", "_stream")

    def __init__(self, dev, stream):
        import torch
        self._dev = self._stream = None
        if dev.index != torch.cuda.current_device():
            self._dev = torch.cuda.device(dev)
        if stream is None:
            self.handle = _current_handle(dev)
            return
        if isinstance(stream, int):
            stream = (torch.cuda.ExternalStream(stream, device=dev) if stream
                      else torch.cuda.default_stream(dev))
        if stream.device != dev:
            raise MuonError(MUON_ERR_INVALID_ARG, f"stream is on {stream.device}, tensors on {dev}")
        self.handle = stream.cuda_stream
        self._stream = torch.cuda.stream(stream)

    def __enter__(self):
        if self._dev is not None:
            self._dev.__enter__()
        if self._stream is not None:
            self._stream.__enter__()
        return self

    def __exit__(self, *exc):
        if self._stream is not None:
            self._stream.__exit__(*exc)
        if self._dev is not None:
            self._dev.__exit__(*exc)


def _workspace(workspace, need: int, dev):
    """The caller's workspace, checked, or a new one on the call's stream."""
    import torch
    if workspace is None:
        return torch.empty(max(1, need), dtype=torch.uint8, device=dev)
    _buf(workspace, "workspace")
    return workspace


# ---------------------------------------------------------------- embedding

def embed_forward(table, ids, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """``scale * table[ids]`` for ids (int32 or int64) of any shape; zeros for
    an id outside [0, vocab).  out: [ids.numel(), dim], rows may be strided;
    without it a tensor of shape (*ids.shape, dim) and dtype ``out_dtype``
    (the table's by default) is allocated.  Returns the output."""
    import torch
    _buf(table, "table", dtypes=TRAIN)
    if len(table.shape) != 2:
        raise MuonError(MUON_ERR_BAD_SHAPE, f"table must be [vocab, dim], is {tuple(table.shape)}")
    vocab, dim = table.shape
    i64 = _index(ids, "ids")
    n = ids.numel()
    if out_dtype is not None and dtype_code(out_dtype) not in TRAIN:
        raise MuonError(MUON_ERR_BAD_DTYPE, f"out_dtype {out_dtype}")
    ld = dim
    if out is not None:
        ld = _rows(out, "out", n, dim)
        if out_dtype is not None and dtype_code(out_dtype) != dtype_code(out.dtype):
            raise MuonError(MUON_ERR_BAD_DTYPE, f"out has dtype {out.dtype}, not {out_dtype}")
    dev = _one_device(table=table, ids=ids, out=out)
    src = table.data_ptr()
    if out is not None:
        dst = out.data_ptr()  # 4: the largest element (a small call's time is the binding's)
        if dst < src + 4 * vocab * dim and src < dst + 4 * n * ld:
            _apart("out", out, n, dim, ld, table=(table, vocab, dim, dim))
        at = ids.data_ptr()
        if dst < at + 8 * n and at < dst + 4 * n * ld:
            _apart("out", out, n, dim, ld, ids=_vector(ids))
    with _Launch(dev, stream) as on:
        if out is None:
            td = {MUON_DTYPE_FP32: torch.float32, MUON_DTYPE_BF16: torch.bfloat16}
            dt = table.dtype if out_dtype is None else td[dtype_code(out_dtype)]
            out = torch.empty((*ids.shape, dim), dtype=dt, device=dev)
            dst = out.data_ptr()
        _check(lib().embed_forward(src, dtype_code(table.dtype), vocab, dim, _ptr(ids), i64, n,
                                   float(scale), dst, dtype_code(out.dtype), ld, on.handle))
    return out


def embed_backward_workspace_size(n: int, vocab: int, dim: int) -> int:
    return int(lib().embed_backward_workspace_size(int(n), int(vocab), int(dim)))


def embed_backward(dout, ids, dtable, scale: float = 1.0, accumulate: bool = False,
                   workspace=None, stream=None):
    """The dense table gradient: ``dtable[v] = scale * sum of dout[t]`` over the
    positions with ``ids[t] == v`` (added to dtable with ``accumulate``).
    dout: [ids.numel(), dim], rows may be strided; dtable: contiguous
    [vocab, dim], a view of a flat gradient buffer for instance.  Returns
    dtable."""
    _buf(dtable, "dtable", dtypes=TRAIN)
    if len(dtable.shape) != 2:
        raise MuonError(MUON_ERR_BAD_SHAPE,
                        f"dtable must be [vocab, dim], is {tuple(dtable.shape)}")
    vocab, dim = dtable.shape
    i64 = _index(ids, "ids")
    n = ids.numel()
    ld = _rows(dout, "dout", n, dim)
    dev = _one_device(dtable=dtable, ids=ids, dout=dout, workspace=workspace)
    ins = {"dout": (dout, n, dim, ld), "ids": _vector(ids)}
    _apart("dtable", dtable, vocab, dim, dim, **ins)
    _apart_workspace(workspace, dtable=(dtable, vocab, dim, dim), **ins)
    with _Launch(dev, stream) as on:
        ws = _workspace(workspace, embed_backward_workspace_size(n, vocab, dim), dev)
        _check(lib().embed_backward(_ptr(dout), dtype_code(dout.dtype), ld, _ptr(ids), i64, n,
                                    float(scale), _ptr(dtable), dtype_code(dtable.dtype), vocab,
                                    dim, int(bool(accumulate)), _ptr(ws), _nbytes(ws), on.handle))
    return dtable


# --------------------------------------------------------- vocabulary loss

def lm_loss_workspace_size(n: int, vocab: int, dim: int, dtype, backward: bool = True) -> int:
    return int(lib().lm_loss_workspace_size(int(n), int(vocab), int(dim), dtype_code(dtype),
                                            int(bool(backward))))


def _loss_args(hidden, weight, targets):
    _buf(weight, "weight", dtypes=TRAIN)
    if len(weight.shape) != 2:
        raise MuonError(MUON_ERR_BAD_SHAPE,
                        f"weight must be [vocab, dim], is {tuple(weight.shape)}")
    vocab, dim = weight.shape
    t64 = _index(targets, "targets")
    n = targets.numel()
    ld = _rows(hidden, "hidden", n, dim, (dtype_code(weight.dtype),))
    return n, vocab, dim, ld, t64


def lm_loss_forward(hidden, weight, targets, loss=None, lse=None, workspace=None, stream=None):
    """Softmax cross entropy of ``hidden @ weight.T`` per row, without storing
    the logits.  hidden: [n, dim], rows may be strided; weight: contiguous
    [vocab, dim] of the same dtype; targets: n int32 or int64, one outside
    [0, vocab) marks a row without loss.  Returns (loss, lse), fp32 of n."""
    import torch
    n, vocab, dim, ld, t64 = _loss_args(hidden, weight, targets)
    for name, t in (("loss", loss), ("lse", lse)):
        if t is not None:
            _block(t, name, (n,), F32)
    dev = _one_device(weight=weight, hidden=hidden, targets=targets, loss=loss, lse=lse,
                      workspace=workspace)
    outs = {k: _vector(t) for k, t in (("loss", loss), ("lse", lse)) if t is not None}
    if len(outs) == 2:
        _apart("loss", *outs["loss"], lse=outs["lse"])
    ins = {"hidden": (hidden, n, dim, ld), "weight": (weight, vocab, dim, dim),
           "targets": _vector(targets)}
    for name, out in outs.items():
        _apart(name, *out, **ins)
    _apart_workspace(workspace, **outs, **ins)
    with _Launch(dev, stream) as on:
        if loss is None:
            loss = torch.empty(n, dtype=torch.float32, device=dev)
        if lse is None:
            lse = torch.empty(n, dtype=torch.float32, device=dev)
        ws = _workspace(workspace, lm_loss_workspace_size(n, vocab, dim, weight.dtype, False), dev)
        _check(lib().lm_loss_forward(_ptr(hidden), ld, _ptr(weight), dtype_code(weight.dtype),
                                     _ptr(targets), t64, n, vocab, dim, _ptr(loss), _ptr(lse),
                                     _ptr(ws), _nbytes(ws), on.handle))
    return loss, lse


def lm_loss_backward(hidden, weight, targets, lse, dloss, dhidden=None, dweight=None,
                     accumulate: bool = False, workspace=None, stream=None):
    """Gradients of ``sum(dloss * loss)`` by hidden and weight; lse from
    lm_loss_forward, dloss fp32 of n.  dhidden ([n, dim], rows may be strided)
    and dweight (contiguous [vocab, dim], a view of a flat gradient buffer for
    instance; ``accumulate`` adds to it) may be bf16 or fp32, are allocated
    in hidden's dtype where None, and not computed where False.  Returns
    (dhidden, dweight), None for what was not computed."""
    import torch
    n, vocab, dim, ld, t64 = _loss_args(hidden, weight, targets)
    _block(lse, "lse", (n,), F32)
    _block(dloss, "dloss", (n,), F32)
    ld_dh = dim
    if dhidden is not None and dhidden is not False:
        ld_dh = _rows(dhidden, "dhidden", n, dim)
    if dweight is not None and dweight is not False:
        _block(dweight, "dweight", (vocab, dim))
    elif accumulate:
        raise MuonError(MUON_ERR_INVALID_ARG, "accumulate needs a dweight to add to")
    dev = _one_device(weight=weight, hidden=hidden, targets=targets, lse=lse, dloss=dloss,
                      dhidden=None if dhidden is False else dhidden,
                      dweight=None if dweight is False else dweight, workspace=workspace)
    outs = {}
    if dhidden is not None and dhidden is not False:
        outs["dhidden"] = (dhidden, n, dim, ld_dh)
    if dweight is not None and dweight is not False:
        outs["dweight"] = (dweight, vocab, dim, dim)
    if len(outs) == 2:
        _apart("dweight", *outs["dweight"], dhidden=outs["dhidden"])
    ins = {"hidden": (hidden, n, dim, ld), "weight": (weight, vocab, dim, dim),
           "targets": _vector(targets), "lse": _vector(lse), "dloss": _vector(dloss)}
    for name, out in outs.items():
        _apart(name, *out, **ins)
    _apart_workspace(workspace, **outs, **ins)
    with _Launch(dev, stream) as on:
        if dhidden is None:
            dhidden = torch.empty((n, dim), dtype=hidden.dtype, device=dev)
        if dweight is None:
            dweight = torch.empty((vocab, dim), dtype=weight.dtype, device=dev)
        dhidden = None if dhidden is False else dhidden
        dweight = None if dweight is False else dweight
        ws = _workspace(workspace, lm_loss_workspace_size(n, vocab, dim, weight.dtype), dev)
        _check(lib().lm_loss_backward(
            _ptr(hidden), ld, _ptr(weight), dtype_code(weight.dtype), _ptr(targets), t64, n, vocab,
            dim, _ptr(lse), _ptr(dloss), _ptr(dhidden),
            dtype_code(weight.dtype if dhidden is None else dhidden.dtype), ld_dh, _ptr(dweight),
            dtype_code(weight.dtype if dweight is None else dweight.dtype), int(bool(accumulate)),
            _ptr(ws), _nbytes(ws), on.handle))
    return dhidden, dweight


# ---------------------------------------------------------- expert products

def _offsets(t, experts: int):
    import torch
    _buf(t, "offsets")
    if t.dtype != torch.int32:
        raise MuonError(MUON_ERR_BAD_DTYPE, f"offsets must be int32, has {t.dtype}")
    if t.numel() != experts + 1:
        raise MuonError(MUON_ERR_BAD_SHAPE,
                        f"offsets has {t.numel()} elements, expected {experts + 1}")


def expert_matmul(x, w, offsets, trans: bool = False, out=None, out_dtype=None, stream=None):
    """Row r of expert e (offsets[e] <= r < offsets[e + 1], int32 on the GPU)
    times that expert's weight: ``x[r] @ w[e]`` with w [experts, k, n], or with
    ``trans`` ``x[r] @ w[e].T`` with w [experts, n, k].  x: [rows, k] of w's
    dtype, rows may be strided.  out: [rows, n], rows may be strided; its
    rows that belong to no expert are left as they were.  Without it a tensor
    of ``out_dtype`` (x's by default) is allocated, with zeros in those rows.
    Returns the output."""
    import torch
    _buf(w, "w", dtypes=TRAIN)
    if len(w.shape) != 3:
        raise MuonError(MUON_ERR_BAD_SHAPE, f"w must be [experts, ., .], is {tuple(w.shape)}")
    experts, k, n = w.shape
    if trans:
        k, n = n, k
    if x is None or len(x.shape) != 2:
        raise MuonError(MUON_ERR_BAD_SHAPE, "x must be [rows, k]")
    rows = x.shape[0]
    ldx = _rows(x, "x", rows, k, (dtype_code(w.dtype),))
    _offsets(offsets, experts)
    if out_dtype is not None and dtype_code(out_dtype) not in TRAIN:
        raise MuonError(MUON_ERR_BAD_DTYPE, f"out_dtype {out_dtype}")
    ldy = n
    if out is not None:
        ldy = _rows(out, "out", rows, n)
        if out_dtype is not None and dtype_code(out_dtype) != dtype_code(out.dtype):
            raise MuonError(MUON_ERR_BAD_DTYPE, f"out has dtype {out.dtype}, not {out_dtype}")
    dev = _one_device(w=w, x=x, offsets=offsets, out=out)
    if out is not None:
        _apart("out", out, rows, n, ldy, x=(x, rows, k, ldx), w=(w, experts * k, n, n),
               offsets=_vector(offsets))
    with _Launch(dev, stream) as on:
        if out is None:
            td = {MUON_DTYPE_FP32: torch.float32, MUON_DTYPE_BF16: torch.bfloat16}
            dt = x.dtype if out_dtype is None else td[dtype_code(out_dtype)]
            out = torch.zeros((rows, n), dtype=dt, device=dev)
        _check(lib().expert_matmul(_ptr(x), ldx, _ptr(w), dtype_code(w.dtype), _ptr(offsets),
                                   experts, rows, k, n, int(bool(trans)), _ptr(out),
                                   dtype_code(out.dtype), ldy, on.handle))
    return out


def expert_wgrad(a, b, offsets, dw, accumulate: bool = False, stream=None):
    """``dw[e] = a_e.T @ b_e`` over expert e's rows (added to dw with
    ``accumulate``): the weight gradient of ``expert_matmul(x, w, offsets)``
    with (a, b) = (x, dy), and of its trans form with (dy, x).  a: [rows, m],
    b: [rows, n] of one dtype, rows may be strided; dw: contiguous
    [experts, m, n], bf16 or fp32.  Returns dw."""
    _buf(dw, "dw", dtypes=TRAIN)
    if len(dw.shape) != 3:
        raise MuonError(MUON_ERR_BAD_SHAPE, f"dw must be [experts, m, n], is {tuple(dw.shape)}")
    experts, m, n = dw.shape
    if a is None or len(a.shape) != 2:
        raise MuonError(MUON_ERR_BAD_SHAPE, "a must be [rows, m]")
    rows = a.shape[0]
    lda = _rows(a, "a", rows, m)
    ldb = _rows(b, "b", rows, n, (dtype_code(a.dtype),))
    _offsets(offsets, experts)
    dev = _one_device(dw=dw, a=a, b=b, offsets=offsets)
    _apart("dw", dw, experts * m, n, n, a=(a, rows, m, lda), b=(b, rows, n, ldb),
           offsets=_vector(offsets))
    with _Launch(dev, stream) as on:
        _check(lib().expert_wgrad(_ptr(a), lda, _ptr(b), ldb, dtype_code(a.dtype), _ptr(offsets),
                                  experts, rows, m, n, _ptr(dw), dtype_code(dw.dtype),
                                  int(bool(accumulate)), on.handle))
    return dw
