"""Block-wise FP8 W8A8 linear for GB300: Python binding of the C ABI (include/fp8bq.h).

Every function here has the name of the C entry point it calls and does
argument marshalling only: torch tensors become device pointers and sizes, the
current CUDA stream becomes the `stream` argument, and a non-zero status
becomes an :class:`Fp8bqError`.  All computation runs in the CUDA library
``_build/libfp8bq.so`` (build it with ``__graft_entry__.build()``); importing
this package without that library raises ImportError -- there is no fallback.

Tensor conventions: BF16 tensors are ``torch.bfloat16``; E4M3 codes are
``torch.float8_e4m3fn`` or ``torch.uint8``; FP32 scales ``torch.float32``;
UE8M0 scale codes ``torch.uint8``.  Matrices are row-major with unit stride in
the last dimension.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

__all__ = [
    "Fp8bqError", "SCALE_ROW_MAJOR", "SCALE_COL_MAJOR", "OP_GEMM", "OP_LINEAR",
    "OP_MX_GEMM", "OP_MX_LINEAR", "OP_STATIC_GEMM", "OP_STATIC_LINEAR", "OP_CHANNEL_GEMM",
    "OP_CHANNEL_LINEAR", "fp8bq_channel_quant_act", "fp8bq_channel_gemm", "fp8bq_channel_linear",
    "OP_UE8M0_GEMM", "OP_UE8M0_LINEAR", "fp8bq_quant_act_ue8m0", "fp8bq_requant_weight_ue8m0",
    "fp8bq_ue8m0_gemm", "fp8bq_ue8m0_linear",
    "OP_GROUPED_GEMM", "fp8bq_grouped_gemm", "fp8bq_grouped_gemm_masked",
    "fp8bq_check_scales",
    "OP_LORA_ADD", "fp8bq_qk_norm_rope", "fp8bq_lora_group", "fp8bq_lora_add",
    "MOE_SOFTMAX", "MOE_SIGMOID", "MOE_MAX_TOKENS", "fp8bq_moe_layer", "fp8bq_moe_experts",
    "fp8bq_moe_workspace_bytes", "new_moe_workspace",
    "library_path",
    "fp8bq_version", "fp8bq_status_string", "fp8bq_last_cuda_error",
    "fp8bq_workspace_bytes", "fp8bq_workspace_init", "fp8bq_poll_status",
    "fp8bq_quant_act", "fp8bq_gemm", "fp8bq_linear", "fp8bq_gemm_noalloc",
    "fp8bq_noalloc_poll_status",
    "NOALLOC_SCRATCH_BYTES", "fp8bq_mx_quant_act",
    "fp8bq_mx_gemm", "fp8bq_mx_linear", "fp8bq_static_quant_act", "fp8bq_static_gemm",
    "fp8bq_add_rmsnorm_quant_act", "fp8bq_add_rmsnorm_static_quant_act",
    "fp8bq_static_linear", "fp8bq_quant_weight_block", "fp8bq_absmax_scale",
    "new_workspace", "fp8bq_e4m3_from_bits",
]

SCALE_ROW_MAJOR, SCALE_COL_MAJOR = 0, 1
(OP_GEMM, OP_LINEAR, OP_MX_GEMM, OP_MX_LINEAR, OP_STATIC_GEMM,
 OP_STATIC_LINEAR, OP_CHANNEL_GEMM, OP_CHANNEL_LINEAR, OP_UE8M0_GEMM,
 OP_UE8M0_LINEAR, OP_GROUPED_GEMM, OP_LORA_ADD) = range(12)
MOE_SOFTMAX, MOE_SIGMOID = 0, 1               # router scores of fp8bq_moe_layer
MOE_MAX_TOKENS = 64
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024      # FP8BQ_NOALLOC_SCRATCH_BYTES

STATUS_NAMES = {0: "FP8BQ_OK", 1: "FP8BQ_ERR_NULL", 2: "FP8BQ_ERR_SHAPE",
                3: "FP8BQ_ERR_ALIGN", 4: "FP8BQ_ERR_UNSUPPORTED", 5: "FP8BQ_ERR_ARCH",
                6: "FP8BQ_ERR_WORKSPACE", 7: "FP8BQ_ERR_CUDA", 8: "FP8BQ_ERR_TIMEOUT",
                9: "FP8BQ_ERR_BOUNDS"}


class Fp8bqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))
        msg = f"{what}: {self.name} ({_lib.fp8bq_status_string(status).decode()})"
        if status == 7:
            msg += f", cudaError {_lib.fp8bq_last_cuda_error()}"
        super().__init__(msg)


# FP8BQ_LIBRARY selects another build of the same library, e.g. the debug
# build with device-side bounds checks (_build.build(debug=True))
_LIB_PATH = os.environ.get("FP8BQ_LIBRARY") or _build.LIB


def library_path() -> str:
    return _LIB_PATH


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"CUDA library {_LIB_PATH} is not built; run __graft_entry__.build() "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    F32 = ctypes.c_float
    sigs = {
        "fp8bq_version": (I32, []),
        "fp8bq_status_string": (ctypes.c_char_p, [I32]),
        "fp8bq_last_cuda_error": (I32, []),
        "fp8bq_workspace_bytes": (SZ, [I32, I64, I64, I64]),
        "fp8bq_workspace_init": (I32, [P, SZ, P]),
        "fp8bq_poll_status": (I32, [P, P]),
        "fp8bq_quant_act": (I32, [P, I64, I64, I64, P, P, I32, P]),
        "fp8bq_gemm": (I32, [P, P, I32, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_linear": (I32, [P, I64, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_gemm_noalloc": (I32, [P, P, I32, P, P, P, P, I64, I64, I64, P]),
        "fp8bq_noalloc_poll_status": (I32, [P]),
        "fp8bq_mx_quant_act": (I32, [P, I64, I64, I64, P, P, P]),
        "fp8bq_mx_gemm": (I32, [P, P, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_mx_linear": (I32, [P, I64, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_static_quant_act": (I32, [P, I64, I64, I64, P, P, P]),
        "fp8bq_channel_quant_act": (I32, [P, I64, I64, I64, P, P, P]),
        "fp8bq_quant_act_ue8m0": (I32, [P, I64, I64, I64, P, P, P]),
        "fp8bq_requant_weight_ue8m0": (I32, [P, P, I64, I64, P, P, P]),
        "fp8bq_ue8m0_gemm": (I32, [P, P, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_ue8m0_linear": (I32, [P, I64, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_grouped_gemm": (I32, [P, P, I32, P, P, P, I64, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_check_scales": (I32, [P, I64, P, P, P, P]),
        "fp8bq_grouped_gemm_masked": (I32, [P, P, I32, P, P, P, I64, I64, P, I64, I64, P, SZ,
                                            P]),
        "fp8bq_channel_gemm": (I32, [P, P, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_channel_linear": (I32, [P, I64, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_add_rmsnorm_quant_act": (I32, [P, I64, P, I64, P, P, F32, I64, I64, P, P, P,
                                              I32, P]),
        "fp8bq_add_rmsnorm_static_quant_act": (I32, [P, I64, P, I64, P, P, F32, P, I64, I64,
                                                     P, P, P]),
        "fp8bq_static_gemm": (I32, [P, P, P, P, P, I32, P, P, I64, I64, I64, P, SZ, P]),
        "fp8bq_static_linear": (I32, [P, I64, P, P, P, P, I32, P, P, I64, I64, I64, P, SZ,
                                      P]),
        "fp8bq_quant_weight_block": (I32, [P, I64, I64, I64, P, P, P]),
        "fp8bq_absmax_scale": (I32, [P, I64, I64, I64, P, P]),
        # calls of a few microseconds: their 64-bit sizes and strides go as pointers
        # do, the same bits converted in half the time (0.08 against 0.14 us each)
        "fp8bq_qk_norm_rope": (I32, [P] * 10 + [F32] + [P] * 4 + [I32, I32] + [P] * 9),
        "fp8bq_lora_group": (I32, [P] * 6),
        "fp8bq_lora_add": (I32, [P] * 20),
        "fp8bq_moe_workspace_bytes": (SZ, [I64, I64, I64, I64, I64]),
        "fp8bq_moe_layer": (I32, [P, I64, P, P, I32, I32, F32, I64, P, P, P, P, P, P, P, I64, I64,
                                  I64, I64, P, SZ, P]),
        "fp8bq_moe_experts": (I32, [P, I64, P, P, I64, P, P, P, P, P, I64, I64, I64, I64, P, SZ,
                                    P]),
        "fp8bq_e4m3_from_bits": (I32, [ctypes.c_uint32, I64, P, P]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


# ---------------------------------------------------------------- marshalling

def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ld(x) -> int:
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit stride in the last dimension")
    return x.stride(0)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _check(status: int, what: str):
    if status != 0:
        raise Fp8bqError(status, what)


# ---------------------------------------------------------------- argument checks
#
# The C interface takes raw pointers and sizes, so a tensor of the wrong shape,
# dtype or device would be read or written past its end.  Every wrapper below
# describes each tensor it passes and `_validate` checks all of them against the
# sizes before the C call; a mismatch raises ValueError and nothing is launched.

_BF16 = (torch.bfloat16,)
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_F32 = (torch.float32,)
_U8 = (torch.uint8,)
_I32 = (torch.int32,)
_POS = (torch.int32, torch.int64)


def _kb(K: int) -> int:
    return -(-K // 128)


def _sx_shape(M: int, K: int, layout: int):
    """Shape of the FP32 activation scales: [M][ceil(K/128)] or [ceil(K/128)][M rounded up to 4]."""
    if layout == SCALE_ROW_MAJOR:
        return (M, _kb(K))
    if layout == SCALE_COL_MAJOR:
        return (_kb(K), -(-M // 4) * 4)
    raise ValueError(f"s_layout must be SCALE_ROW_MAJOR or SCALE_COL_MAJOR, not {layout!r}")


class _Spec:
    """One tensor argument: name, accepted dtypes and what its shape must be.

    kind "contig": contiguous with exactly `shape` (or `numel` elements when
    shape is None); kind "rows": 2-D [shape] with unit stride in the last
    dimension and any row pitch (the C call takes the pitch); kind "heads": 3-D
    [shape] with unit stride in the last dimension and any other strides."""
    __slots__ = ("name", "t", "dtypes", "shape", "numel", "kind", "optional")

    def __init__(self, name, t, dtypes, shape=None, numel=None, kind="contig", optional=False):
        self.name, self.t, self.dtypes = name, t, dtypes
        self.shape = None if shape is None else tuple(int(v) for v in shape)
        self.numel, self.kind, self.optional = numel, kind, optional


def _validate(what: str, specs, stream=None):
    """Checks every tensor argument of one call before any pointer is taken."""
    present = []
    for sp in specs:
        t = sp.t
        if t is None:
            if sp.optional:
                continue
            raise ValueError(f"{what}: {sp.name} is required")
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{what}: {sp.name} must be a torch.Tensor, not {type(t).__name__}")
        if sp.dtypes is not None and t.dtype not in sp.dtypes:
            names = " or ".join(str(d).replace("torch.", "") for d in sp.dtypes)
            raise ValueError(f"{what}: {sp.name} must be {names}, not "
                             f"{str(t.dtype).replace('torch.', '')}")
        if sp.kind == "rows":
            if t.dim() != 2 or tuple(t.shape) != sp.shape:
                raise ValueError(f"{what}: {sp.name} must have shape {sp.shape}, "
                                 f"not {tuple(t.shape)}")
            if t.numel() and (t.stride(1) != 1 or t.stride(0) < t.shape[1]):
                raise ValueError(f"{what}: {sp.name} needs unit stride in its last dimension "
                                 f"and a row pitch of at least {t.shape[1]}")
        elif sp.kind == "heads":
            if tuple(t.shape) != sp.shape:
                raise ValueError(f"{what}: {sp.name} must have shape {sp.shape}, "
                                 f"not {tuple(t.shape)}")
            if t.numel() and (t.stride(2) != 1 or min(t.stride()) < 0):
                raise ValueError(f"{what}: {sp.name} needs unit stride in its last dimension")
        else:
            if sp.shape is not None and tuple(t.shape) != sp.shape:
                raise ValueError(f"{what}: {sp.name} must have shape {sp.shape}, "
                                 f"not {tuple(t.shape)}")
            if sp.numel is not None and t.numel() != sp.numel:
                raise ValueError(f"{what}: {sp.name} must have {sp.numel} elements, "
                                 f"not {t.numel()}")
            if not t.is_contiguous():
                raise ValueError(f"{what}: {sp.name} must be contiguous")
        present.append(sp)
    # device last, so that shape mistakes are reported even for host tensors
    for sp in present:
        if not sp.t.is_cuda:
            raise ValueError(f"{what}: {sp.name} must be a CUDA tensor, not on {sp.t.device}")
    if present:
        want = _call_device(stream)
        for sp in present:
            if sp.t.device.index != want:
                raise ValueError(f"{what}: {sp.name} is on cuda:{sp.t.device.index} but the "
                                 f"call runs on cuda:{want}")


def _call_device(stream) -> int:
    """The device a call runs on: the stream's, else the current device."""
    if stream is not None and not isinstance(stream, int):
        dev = stream.device
        dev_index = dev.index if isinstance(dev, torch.device) else int(dev)
        if dev_index != torch.cuda.current_device():
            raise ValueError(f"stream is on cuda:{dev_index}, the current device is "
                             f"cuda:{torch.cuda.current_device()}")
        return dev_index
    return torch.cuda.current_device()


def _mat(t, name):
    """(rows, cols) of a 2-D matrix argument whose shape sets the call's sizes."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    rows, cols = t.shape
    return rows, cols


# ---------------------------------------------------------------- utility

def fp8bq_version() -> int:
    return _lib.fp8bq_version()


def fp8bq_status_string(status: int) -> str:
    return _lib.fp8bq_status_string(status).decode()


def fp8bq_last_cuda_error() -> int:
    return _lib.fp8bq_last_cuda_error()


def fp8bq_workspace_bytes(op: int, M: int, N: int, K: int) -> int:
    return _lib.fp8bq_workspace_bytes(op, M, N, K)


def _ws(ws):
    return _Spec("ws", ws, None)


def fp8bq_workspace_init(ws, stream=None):
    _validate("fp8bq_workspace_init", [_ws(ws)], stream)
    _check(_lib.fp8bq_workspace_init(_ptr(ws), _nbytes(ws), _stream(stream)),
           "fp8bq_workspace_init")


def fp8bq_poll_status(ws, stream=None) -> int:
    """Synchronises the stream; returns 0, 8 (FP8BQ_ERR_TIMEOUT) or, from a
    debug build, 9 (FP8BQ_ERR_BOUNDS)."""
    _validate("fp8bq_poll_status", [_ws(ws)], stream)
    return _lib.fp8bq_poll_status(_ptr(ws), _stream(stream))


def new_workspace(op: int, M: int, N: int, K: int, device="cuda", stream=None):
    """A zero-initialised workspace (torch-owned device memory) for `op` at this shape."""
    ws = torch.empty(fp8bq_workspace_bytes(op, M, N, K), dtype=torch.uint8, device=device)
    fp8bq_workspace_init(ws, stream)
    return ws


def _bias(bias, N):
    return _Spec("bias", bias, _BF16, numel=N, optional=True)


# ---------------------------------------------------------------- block path

def fp8bq_quant_act(x, q, s, s_layout: int = SCALE_ROW_MAJOR, stream=None):
    M, K = _mat(x, "x")
    _validate("fp8bq_quant_act", [
        _Spec("x", x, _BF16, (M, K), kind="rows"),
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("s", s, _F32, _sx_shape(M, K, s_layout))], stream)
    _check(_lib.fp8bq_quant_act(_ptr(x), M, K, _ld(x), _ptr(q), _ptr(s), s_layout,
                                _stream(stream)), "fp8bq_quant_act")


def _block_gemm_specs(q, s_x, w, s_w, y, bias, s_layout):
    M, K = _mat(q, "q")
    N = _mat(w, "w")[0]
    return M, N, K, [
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("s_x", s_x, _F32, _sx_shape(M, K, s_layout)),
        _Spec("w", w, _E4M3, (N, K)),
        _Spec("s_w", s_w, _F32, (_kb(N), _kb(K))),
        _Spec("y", y, _BF16, (M, N)),
        _bias(bias, N)]


def fp8bq_gemm(q, s_x, w, s_w, y, ws, bias=None, s_layout: int = SCALE_ROW_MAJOR,
               stream=None):
    M, N, K, specs = _block_gemm_specs(q, s_x, w, s_w, y, bias, s_layout)
    _validate("fp8bq_gemm", specs + [_ws(ws)], stream)
    _check(_lib.fp8bq_gemm(_ptr(q), _ptr(s_x), s_layout, _ptr(w), _ptr(s_w), _ptr(bias),
                           _ptr(y), M, N, K, _ptr(ws), _nbytes(ws), _stream(stream)),
           "fp8bq_gemm")


def fp8bq_gemm_noalloc(q, s_x, w, s_w, y, bias=None, s_layout: int = SCALE_ROW_MAJOR,
                       stream=None):
    """fp8bq_gemm on the library's fixed device scratch instead of a workspace
    (for callers that may not allocate device memory); see include/fp8bq.h."""
    M, N, K, specs = _block_gemm_specs(q, s_x, w, s_w, y, bias, s_layout)
    _validate("fp8bq_gemm_noalloc", specs, stream)
    _check(_lib.fp8bq_gemm_noalloc(_ptr(q), _ptr(s_x), s_layout, _ptr(w), _ptr(s_w),
                                   _ptr(bias), _ptr(y), M, N, K, _stream(stream)),
           "fp8bq_gemm_noalloc")


def _linear_specs(x, w, y, bias):
    M, K = _mat(x, "x")
    N = _mat(w, "w")[0]
    return M, N, K, [
        _Spec("x", x, _BF16, (M, K), kind="rows"),
        _Spec("w", w, _E4M3, (N, K)),
        _Spec("y", y, _BF16, (M, N)),
        _bias(bias, N)]


def fp8bq_noalloc_poll_status(stream=None) -> int:
    """Synchronises the stream; 0, or 8 (FP8BQ_ERR_TIMEOUT) if a wait of an
    fp8bq_gemm_noalloc call on this device ran out."""
    return _lib.fp8bq_noalloc_poll_status(_stream(stream))


def fp8bq_linear(x, w, s_w, y, ws, bias=None, stream=None):
    M, N, K, specs = _linear_specs(x, w, y, bias)
    _validate("fp8bq_linear", specs + [_Spec("s_w", s_w, _F32, (_kb(N), _kb(K))), _ws(ws)],
              stream)
    _check(_lib.fp8bq_linear(_ptr(x), _ld(x), _ptr(w), _ptr(s_w), _ptr(bias), _ptr(y),
                             M, N, K, _ptr(ws), _nbytes(ws), _stream(stream)),
           "fp8bq_linear")


# ---------------------------------------------------------------- MX path

def fp8bq_mx_quant_act(x, q, s, stream=None):
    M, K = _mat(x, "x")
    _validate("fp8bq_mx_quant_act", [
        _Spec("x", x, _BF16, (M, K), kind="rows"),
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("s", s, _U8, (M, K // 32))], stream)
    _check(_lib.fp8bq_mx_quant_act(_ptr(x), M, K, _ld(x), _ptr(q), _ptr(s),
                                   _stream(stream)), "fp8bq_mx_quant_act")


def fp8bq_mx_gemm(q, s_x, w, s_w, y, ws, bias=None, stream=None):
    M, K = _mat(q, "q")
    N = _mat(w, "w")[0]
    _validate("fp8bq_mx_gemm", [
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("s_x", s_x, _U8, (M, K // 32)),
        _Spec("w", w, _E4M3, (N, K)),
        _Spec("s_w", s_w, _U8, (N, K // 32)),
        _Spec("y", y, _BF16, (M, N)), _bias(bias, N), _ws(ws)], stream)
    _check(_lib.fp8bq_mx_gemm(_ptr(q), _ptr(s_x), _ptr(w), _ptr(s_w), _ptr(bias), _ptr(y),
                              M, N, K, _ptr(ws), _nbytes(ws), _stream(stream)),
           "fp8bq_mx_gemm")


def fp8bq_mx_linear(x, w, s_w, y, ws, bias=None, stream=None):
    M, N, K, specs = _linear_specs(x, w, y, bias)
    _validate("fp8bq_mx_linear", specs + [_Spec("s_w", s_w, _U8, (N, K // 32)), _ws(ws)],
              stream)
    _check(_lib.fp8bq_mx_linear(_ptr(x), _ld(x), _ptr(w), _ptr(s_w), _ptr(bias), _ptr(y),
                                M, N, K, _ptr(ws), _nbytes(ws), _stream(stream)),
           "fp8bq_mx_linear")


# ---------------------------------------------------------------- static path

def _parts(part_sizes):
    arr = (ctypes.c_int64 * len(part_sizes))(*[int(p) for p in part_sizes])
    return arr, len(part_sizes)


def fp8bq_static_quant_act(x, s_x, q, stream=None):
    M, K = _mat(x, "x")
    _validate("fp8bq_static_quant_act", [
        _Spec("x", x, _BF16, (M, K), kind="rows"),
        _Spec("s_x", s_x, _F32, numel=1),
        _Spec("q", q, _E4M3, (M, K))], stream)
    _check(_lib.fp8bq_static_quant_act(_ptr(x), M, K, _ld(x), _ptr(s_x), _ptr(q),
                                       _stream(stream)), "fp8bq_static_quant_act")


def fp8bq_channel_quant_act(x, q, s, stream=None):
    """One scale per row (per-token activations, or per-channel weights)."""
    M, K = _mat(x, "x")
    _validate("fp8bq_channel_quant_act", [
        _Spec("x", x, _BF16, (M, K), kind="rows"),
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("s", s, _F32, numel=M)], stream)
    _check(_lib.fp8bq_channel_quant_act(_ptr(x), M, K, _ld(x), _ptr(q), _ptr(s),
                                        _stream(stream)), "fp8bq_channel_quant_act")


def fp8bq_channel_gemm(q, s_x, w, s_w, y, ws, bias=None, stream=None):
    M, K = _mat(q, "q")
    N = _mat(w, "w")[0]
    _validate("fp8bq_channel_gemm", [
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("s_x", s_x, _F32, numel=M),
        _Spec("w", w, _E4M3, (N, K)),
        _Spec("s_w", s_w, _F32, numel=N),
        _Spec("y", y, _BF16, (M, N)), _bias(bias, N), _ws(ws)], stream)
    _check(_lib.fp8bq_channel_gemm(_ptr(q), _ptr(s_x), _ptr(w), _ptr(s_w), _ptr(bias), _ptr(y),
                                   M, N, K, _ptr(ws), _nbytes(ws), _stream(stream)),
           "fp8bq_channel_gemm")


def fp8bq_channel_linear(x, w, s_w, y, ws, bias=None, stream=None):
    M, N, K, specs = _linear_specs(x, w, y, bias)
    _validate("fp8bq_channel_linear", specs + [_Spec("s_w", s_w, _F32, numel=N), _ws(ws)],
              stream)
    _check(_lib.fp8bq_channel_linear(_ptr(x), _ld(x), _ptr(w), _ptr(s_w), _ptr(bias), _ptr(y),
                                     M, N, K, _ptr(ws), _nbytes(ws), _stream(stream)),
           "fp8bq_channel_linear")


def fp8bq_quant_act_ue8m0(x, q, u, stream=None):
    """Group-128 quantisation with power-of-two (UE8M0) scales."""
    M, K = _mat(x, "x")
    _validate("fp8bq_quant_act_ue8m0", [
        _Spec("x", x, _BF16, (M, K), kind="rows"),
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("u", u, _U8, (M, _kb(K)))], stream)
    _check(_lib.fp8bq_quant_act_ue8m0(_ptr(x), M, K, _ld(x), _ptr(q), _ptr(u), _stream(stream)),
           "fp8bq_quant_act_ue8m0")


def fp8bq_requant_weight_ue8m0(q, s_w, q_out, u_w, stream=None):
    """FP32 128x128 block scales -> UE8M0 (rounded up), codes re-encoded."""
    N, K = _mat(q, "q")
    _validate("fp8bq_requant_weight_ue8m0", [
        _Spec("q", q, _E4M3, (N, K)),
        _Spec("s_w", s_w, _F32, (_kb(N), _kb(K))),
        _Spec("q_out", q_out, _E4M3, (N, K)),
        _Spec("u_w", u_w, _U8, (_kb(N), _kb(K)))], stream)
    _check(_lib.fp8bq_requant_weight_ue8m0(_ptr(q), _ptr(s_w), N, K, _ptr(q_out), _ptr(u_w),
                                           _stream(stream)), "fp8bq_requant_weight_ue8m0")


def fp8bq_ue8m0_gemm(q, u_x, w, u_w, y, ws, bias=None, stream=None):
    M, K = _mat(q, "q")
    N = _mat(w, "w")[0]
    _validate("fp8bq_ue8m0_gemm", [
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("u_x", u_x, _U8, (M, _kb(K))),
        _Spec("w", w, _E4M3, (N, K)),
        _Spec("u_w", u_w, _U8, (_kb(N), _kb(K))),
        _Spec("y", y, _BF16, (M, N)), _bias(bias, N), _ws(ws)], stream)
    _check(_lib.fp8bq_ue8m0_gemm(_ptr(q), _ptr(u_x), _ptr(w), _ptr(u_w), _ptr(bias), _ptr(y),
                                 M, N, K, _ptr(ws), _nbytes(ws), _stream(stream)),
           "fp8bq_ue8m0_gemm")


def fp8bq_ue8m0_linear(x, w, u_w, y, ws, bias=None, stream=None):
    M, N, K, specs = _linear_specs(x, w, y, bias)
    _validate("fp8bq_ue8m0_linear",
              specs + [_Spec("u_w", u_w, _U8, (_kb(N), _kb(K))), _ws(ws)], stream)
    _check(_lib.fp8bq_ue8m0_linear(_ptr(x), _ld(x), _ptr(w), _ptr(u_w), _ptr(bias), _ptr(y),
                                   M, N, K, _ptr(ws), _nbytes(ws), _stream(stream)),
           "fp8bq_ue8m0_linear")


def fp8bq_check_scales(s, scratch=None, stream=None) -> dict:
    """Counts unusable FP32 scales in a device tensor: the unloaded sentinel
    (-FLT_MAX), NaN / inf, other values <= 0; and the first bad flat index."""
    if scratch is None and isinstance(s, torch.Tensor):
        scratch = torch.empty(4, dtype=torch.int64, device=s.device)
    _validate("fp8bq_check_scales", [
        _Spec("s", s, _F32, numel=s.numel() if isinstance(s, torch.Tensor) else None),
        _Spec("scratch", scratch, (torch.int64,), numel=4)], stream)
    counts = (ctypes.c_int64 * 3)()
    first = ctypes.c_int64()
    _check(_lib.fp8bq_check_scales(_ptr(s), s.numel(), _ptr(scratch),
                                   ctypes.c_void_p(ctypes.addressof(counts)),
                                   ctypes.c_void_p(ctypes.addressof(first)), _stream(stream)),
           "fp8bq_check_scales")
    return {"sentinel": counts[0], "nonfinite": counts[1], "nonpositive": counts[2],
            "first_bad": first.value}


# ---------------------------------------------------------------- grouped (MoE)

def _experts_w(w):
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be a 3-D tensor [E, N, K]")
    return (int(v) for v in w.shape)


def fp8bq_grouped_gemm(q, s_x, w, s_w, offsets, y, ws, s_layout: int = SCALE_ROW_MAJOR,
                       stream=None):
    """Rows offsets[e] .. offsets[e+1]-1 of q / y use expert e's weight w[e]
    [N, K] and scale grid s_w[e]; offsets is a device int32 tensor [E+1]."""
    M, K = _mat(q, "q")
    E, N, Kw = _experts_w(w)
    if Kw != K:
        raise ValueError(f"fp8bq_grouped_gemm: w has K = {Kw}, q has K = {K}")
    _validate("fp8bq_grouped_gemm", [
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("s_x", s_x, _F32, _sx_shape(M, K, s_layout)),
        _Spec("w", w, _E4M3, (E, N, K)),
        _Spec("s_w", s_w, _F32, (E, _kb(N), _kb(K))),
        _Spec("offsets", offsets, _I32, numel=E + 1),
        _Spec("y", y, _BF16, (M, N)), _ws(ws)], stream)
    _check(_lib.fp8bq_grouped_gemm(_ptr(q), _ptr(s_x), s_layout, _ptr(w), _ptr(s_w),
                                   _ptr(offsets), E, _ptr(y), M, N, K, _ptr(ws), _nbytes(ws),
                                   _stream(stream)), "fp8bq_grouped_gemm")


def fp8bq_grouped_gemm_masked(q, s_x, w, s_w, masked_m, y, ws, s_layout: int = SCALE_ROW_MAJOR,
                              stream=None):
    """q [E, max_m, K] (or [E*max_m, K]); the first masked_m[e] rows of slot e
    use expert e's weight; masked_m is a device int32 tensor [E]."""
    E, N, K = _experts_w(w)
    if not isinstance(q, torch.Tensor) or E == 0 or q.numel() % (K * E):
        raise ValueError(f"fp8bq_grouped_gemm_masked: q must hold E * max_m rows of K = {K}")
    max_m = q.numel() // (K * E)
    rows = E * max_m
    _validate("fp8bq_grouped_gemm_masked", [
        _Spec("q", q, _E4M3, numel=rows * K),
        _Spec("s_x", s_x, _F32, numel=_sx_shape(rows, K, s_layout)[0] *
              _sx_shape(rows, K, s_layout)[1]),
        _Spec("w", w, _E4M3, (E, N, K)),
        _Spec("s_w", s_w, _F32, (E, _kb(N), _kb(K))),
        _Spec("masked_m", masked_m, _I32, numel=E),
        _Spec("y", y, _BF16, numel=rows * N), _ws(ws)], stream)
    _check(_lib.fp8bq_grouped_gemm_masked(_ptr(q), _ptr(s_x), s_layout, _ptr(w), _ptr(s_w),
                                          _ptr(masked_m), E, max_m, _ptr(y), N, K, _ptr(ws),
                                          _nbytes(ws), _stream(stream)),
           "fp8bq_grouped_gemm_masked")


# ---------------------------------------------------------------- beside the linears
#
# Calls of a few microseconds: the checks first run as plain comparisons (about
# 0.4 us a tensor), and `_validate`, which names what is wrong, only where one
# of them fails.

def _fits(dev, contig, rows=()):
    """Whether every (tensor, dtypes, shape) of `contig` is a contiguous tensor,
    and of `rows` a matrix with unit column stride, of that type and shape on
    device `dev`."""
    try:
        for t, dtypes, shape in contig:
            if (t.dtype not in dtypes or t.shape != shape or not t.is_contiguous() or
                    t.get_device() != dev):
                return False
        for t, dtypes, shape in rows:
            if t.dtype not in dtypes or t.shape != shape or t.get_device() != dev:
                return False
            pitch, one = t.stride()
            if one != 1 or pitch < shape[1]:
                return False
    except AttributeError:  # None, or no tensor
        return False
    return True


def _call_stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev if dev >= 0 else torch.cuda.current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _device(t) -> int:
    """Device index of `t` where that is the current device, else -2: the checks
    then say what is wrong."""
    if not isinstance(t, torch.Tensor):
        return -2
    dev = t.get_device()
    return dev if dev >= 0 and dev == torch._C._cuda_getDevice() else -2


def _opt_ptr(t):
    return None if t is None else t.data_ptr()


def _heads(t, name):
    """(tokens, heads, head size) of a 3-D argument whose shape sets the call's sizes."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D tensor [tokens, heads, head size]")
    return t.shape


def _fit_heads(t, shape, dev):
    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.shape != shape or
            t.get_device() != dev):
        return False
    a, b, one = t.stride()
    return one == 1 and a >= 0 and b >= 0


def fp8bq_qk_norm_rope(q, k, q_gamma, k_gamma, table, positions, q_out, k_out, eps: float = 1e-6,
                       interleaved: bool = False, stream=None):
    """RMSNorm of each head of q [T, HQ, D] and k [T, HK, D] (any token and head
    strides: slices of the packed QKV rows) and the rotary embedding, into
    q_out and k_out (which may be q and k).  A gamma of None leaves out the
    norm; k (and k_out) may be None.  table: FP32 [P, rot], a position's
    cosines, then its sines; positions: int32 or int64 [T]."""
    T, HQ, D = _heads(q, "q")
    HK = 0
    if k is not None:
        HK = _heads(k, "k")[1]
    P, rot = _mat(table, "table")
    dev = _device(q)
    contig = [(table, _F32, (P, rot)), (positions, _POS, (T,))]
    if q_gamma is not None:
        contig.append((q_gamma, _BF16, (D,)))
    if k_gamma is not None:
        contig.append((k_gamma, _BF16, (D,)))
    if not (stream is None and _fits(dev, contig) and q_out is not None and
            _fit_heads(q, (T, HQ, D), dev) and _fit_heads(q_out, (T, HQ, D), dev) and
            (k is None) == (k_out is None) and
            (k is None or (_fit_heads(k, (T, HK, D), dev) and _fit_heads(k_out, (T, HK, D), dev)))):
        _validate("fp8bq_qk_norm_rope", [
            _Spec("q", q, _BF16, (T, HQ, D), kind="heads"),
            _Spec("k", k, _BF16, (T, HK, D), kind="heads", optional=True),
            _Spec("q_gamma", q_gamma, _BF16, numel=D, optional=True),
            _Spec("k_gamma", k_gamma, _BF16, numel=D, optional=True),
            _Spec("table", table, _F32, (P, rot)),
            _Spec("positions", positions, _POS, (T,)),
            _Spec("q_out", q_out, _BF16, (T, HQ, D), kind="heads"),
            _Spec("k_out", k_out, _BF16, (T, HK, D), kind="heads", optional=k is None)], stream)
        if k is None and k_out is not None:
            raise ValueError("fp8bq_qk_norm_rope: k_out without k")
    qt, qh, _ = q.stride()
    ot, oh, _ = q_out.stride()
    kp = kop = None
    kt = kh = kot = koh = 0
    if k is not None:
        kp, kop = k.data_ptr(), k_out.data_ptr()
        kt, kh, _ = k.stride()
        kot, koh, _ = k_out.stride()
    status = _lib.fp8bq_qk_norm_rope(
        q.data_ptr(), qt, qh, HQ, kp, kt, kh, HK, _opt_ptr(q_gamma), _opt_ptr(k_gamma), eps,
        table.data_ptr(), P, rot, positions.data_ptr(),
        64 if positions.dtype is torch.int64 else 32, interleaved, q_out.data_ptr(), ot, oh, kop,
        kot, koh, T, D, _call_stream(stream, dev))
    _check(status, "fp8bq_qk_norm_rope")


def fp8bq_lora_group(ids, order, offsets, stream=None):
    """Token indices sorted by adapter (stable) into order [M], and each
    adapter's places in it into offsets [L+1]; ids outside [0, L) come last."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 1:
        raise ValueError("ids must be a 1-D tensor")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be a 1-D tensor of L + 1 elements")
    M, L = ids.shape[0], offsets.shape[0] - 1
    dev = _device(ids)
    if stream is not None or not _fits(dev, ((ids, _I32, (M,)), (order, _I32, (M,)),
                                             (offsets, _I32, (L + 1,)))):
        _validate("fp8bq_lora_group", [
            _Spec("ids", ids, _I32, (M,)), _Spec("order", order, _I32, (M,)),
            _Spec("offsets", offsets, _I32, (L + 1,))], stream)
    status = _lib.fp8bq_lora_group(ids.data_ptr(), M, L, order.data_ptr(), offsets.data_ptr(),
                                   _call_stream(stream, dev))
    _check(status, "fp8bq_lora_group")


def fp8bq_lora_add(x, a, b, scales, order, offsets, base, y, ws, ranks=None, stream=None):
    """y = base + scales[i] * b[i] @ (a[i] @ x[t]) with each token's adapter i
    (a [L, R, K], b [L, N, R]; order and offsets from fp8bq_lora_group); y may
    be base.  Workspace: new_workspace(OP_LORA_ADD, M, R, K)."""
    M, K = _mat(x, "x")
    N = _mat(y, "y")[1]
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise ValueError("a must be a 3-D tensor [L, R, K]")
    L, R, _ = a.shape
    dev = _device(x)
    contig = [(a, _BF16, (L, R, K)), (b, _BF16, (L, N, R)), (scales, _F32, (L,)),
              (order, _I32, (M,)), (offsets, _I32, (L + 1,)), (ws, _U8, (_len(ws),))]
    if ranks is not None:
        contig.append((ranks, _I32, (L,)))
    if stream is not None or not _fits(dev, contig, ((x, _BF16, (M, K)), (base, _BF16, (M, N)),
                                                     (y, _BF16, (M, N)))):
        _validate("fp8bq_lora_add", [
            _Spec("x", x, _BF16, (M, K), kind="rows"),
            _Spec("a", a, _BF16, (L, R, K)), _Spec("b", b, _BF16, (L, N, R)),
            _Spec("scales", scales, _F32, (L,)),
            _Spec("ranks", ranks, _I32, (L,), optional=True),
            _Spec("order", order, _I32, (M,)), _Spec("offsets", offsets, _I32, (L + 1,)),
            _Spec("base", base, _BF16, (M, N), kind="rows"),
            _Spec("y", y, _BF16, (M, N), kind="rows"), _ws(ws)], stream)
    status = _lib.fp8bq_lora_add(
        x.data_ptr(), x.stride(0), a.data_ptr(), b.data_ptr(), scales.data_ptr(), _opt_ptr(ranks),
        order.data_ptr(), offsets.data_ptr(), base.data_ptr(), base.stride(0), y.data_ptr(),
        y.stride(0), M, N, K, L, R, ws.data_ptr(), _nbytes(ws), _call_stream(stream, dev))
    _check(status, "fp8bq_lora_add")


def _len(t):
    return t.shape[0] if isinstance(t, torch.Tensor) and t.dim() else 0


def fp8bq_moe_workspace_bytes(M: int, E: int, H: int, I: int, topk: int) -> int:
    return _lib.fp8bq_moe_workspace_bytes(M, E, H, I, topk)


def new_moe_workspace(M: int, E: int, H: int, I: int, topk: int, device="cuda", stream=None):
    """A zero-initialised workspace for fp8bq_moe_layer and fp8bq_moe_experts at these sizes."""
    ws = torch.empty(fp8bq_moe_workspace_bytes(M, E, H, I, topk), dtype=torch.uint8, device=device)
    fp8bq_workspace_init(ws, stream)
    return ws


def _moe_sizes(x, w13):
    M, H = _mat(x, "x")
    E, I2, _ = _experts_w(w13)
    return M, E, H, I2 // 2


def _moe_check(what, M, E, H, I, x, w13, s13, w2, s2, y, ws, more, stream, dev):
    """`more`: (name, tensor, dtypes, shape) of the form's own arguments, None left out."""
    KI, KH = _kb(I), _kb(H)
    contig = [(w13, _E4M3, (E, 2 * I, H)), (s13, _F32, (E, _kb(2 * I), KH)),
              (w2, _E4M3, (E, H, I)), (s2, _F32, (E, KH, KI)), (y, _BF16, (M, H)),
              (ws, _U8, (_len(ws),))]
    contig += [m[1:] for m in more if m[1] is not None]
    if stream is None and _fits(dev, contig, ((x, _BF16, (M, H)),)):
        return
    _validate(what, [
        _Spec("x", x, _BF16, (M, H), kind="rows"),
        _Spec("w13", w13, _E4M3, (E, 2 * I, H)),
        _Spec("s13", s13, _F32, (E, _kb(2 * I), KH)),
        _Spec("w2", w2, _E4M3, (E, H, I)),
        _Spec("s2", s2, _F32, (E, KH, KI)),
        _Spec("y", y, _BF16, (M, H)), _ws(ws)] +
        [_Spec(n, t, d, sh, optional=n in _MOE_OPTIONAL) for n, t, d, sh in more], stream)


_MOE_OPTIONAL = ("bias", "ids_out", "weights_out")


def fp8bq_moe_layer(x, logits, w13, s13, w2, s2, y, ws, topk: int, score: int = MOE_SOFTMAX,
                    renormalize: bool = True, routed_scale: float = 1.0, bias=None, ids_out=None,
                    weights_out=None, stream=None):
    """A whole mixture-of-experts layer for up to 64 tokens x [M, H] from the
    router's logits [M, E]: top-k routing, w13 [E, 2I, H], SiLU(gate) * up,
    w2 [E, H, I], weighted sum into y.  bias [E] (MOE_SIGMOID): added to the
    score for the choice only.  ids_out / weights_out [M, topk] receive the
    routing.  Workspace: new_moe_workspace(M, E, H, I, topk)."""
    M, E, H, I = _moe_sizes(x, w13)
    dev = _device(x)
    _moe_check("fp8bq_moe_layer", M, E, H, I, x, w13, s13, w2, s2, y, ws, (
        ("logits", logits, _F32, (M, E)), ("bias", bias, _F32, (E,)),
        ("ids_out", ids_out, _I32, (M, topk)), ("weights_out", weights_out, _F32, (M, topk))),
        stream, dev)
    if logits is None:
        raise ValueError("fp8bq_moe_layer: logits is required")
    status = _lib.fp8bq_moe_layer(
        x.data_ptr(), x.stride(0), logits.data_ptr(), _opt_ptr(bias), score, renormalize,
        routed_scale, topk, w13.data_ptr(), s13.data_ptr(), w2.data_ptr(), s2.data_ptr(),
        y.data_ptr(), _opt_ptr(ids_out), _opt_ptr(weights_out), M, E, H, I, ws.data_ptr(),
        _nbytes(ws), _call_stream(stream, dev))
    _check(status, "fp8bq_moe_layer")


def fp8bq_moe_experts(x, ids, weights, w13, s13, w2, s2, y, ws, stream=None):
    """The layer for tokens already routed: ids int32 [M, topk] (values outside
    [0, E) are left out) and weights FP32 [M, topk]."""
    M, E, H, I = _moe_sizes(x, w13)
    topk = _mat(ids, "ids")[1]
    dev = _device(x)
    _moe_check("fp8bq_moe_experts", M, E, H, I, x, w13, s13, w2, s2, y, ws, (
        ("ids", ids, _I32, (M, topk)), ("weights", weights, _F32, (M, topk))), stream, dev)
    if weights is None:
        raise ValueError("fp8bq_moe_experts: weights is required")
    status = _lib.fp8bq_moe_experts(
        x.data_ptr(), x.stride(0), ids.data_ptr(), weights.data_ptr(), topk, w13.data_ptr(),
        s13.data_ptr(), w2.data_ptr(), s2.data_ptr(), y.data_ptr(), M, E, H, I, ws.data_ptr(),
        _nbytes(ws), _call_stream(stream, dev))
    _check(status, "fp8bq_moe_experts")


# ---------------------------------------------------------------- residual add + RMSNorm

def _norm_specs(x, gamma, residual, residual_out, y):
    M, K = _mat(x, "x")
    return M, K, [
        _Spec("x", x, _BF16, (M, K), kind="rows"),
        _Spec("gamma", gamma, _BF16, numel=K),
        _Spec("residual", residual, _BF16, (M, K), kind="rows", optional=True),
        _Spec("residual_out", residual_out, _BF16, (M, K), optional=True),
        _Spec("y", y, _BF16, (M, K), optional=True)]


def fp8bq_add_rmsnorm_quant_act(x, gamma, eps: float, residual=None, residual_out=None,
                                y=None, q=None, s=None, s_layout: int = SCALE_ROW_MAJOR,
                                stream=None):
    """Residual add + RMSNorm (+ group-128 quantisation when q is given)."""
    M, K, specs = _norm_specs(x, gamma, residual, residual_out, y)
    if q is not None:
        specs += [_Spec("q", q, _E4M3, (M, K)), _Spec("s", s, _F32, _sx_shape(M, K, s_layout))]
    _validate("fp8bq_add_rmsnorm_quant_act", specs, stream)
    _check(_lib.fp8bq_add_rmsnorm_quant_act(
        _ptr(x), _ld(x), _ptr(residual), 0 if residual is None else _ld(residual),
        _ptr(residual_out), _ptr(gamma), float(eps), M, K, _ptr(y), _ptr(q), _ptr(s),
        s_layout, _stream(stream)), "fp8bq_add_rmsnorm_quant_act")


def fp8bq_add_rmsnorm_static_quant_act(x, gamma, eps: float, s_x, q, residual=None,
                                       residual_out=None, y=None, stream=None):
    """Residual add + RMSNorm, then static per-tensor quantisation with s_x[0]."""
    M, K, specs = _norm_specs(x, gamma, residual, residual_out, y)
    specs += [_Spec("s_x", s_x, _F32, numel=1), _Spec("q", q, _E4M3, (M, K))]
    _validate("fp8bq_add_rmsnorm_static_quant_act", specs, stream)
    _check(_lib.fp8bq_add_rmsnorm_static_quant_act(
        _ptr(x), _ld(x), _ptr(residual), 0 if residual is None else _ld(residual),
        _ptr(residual_out), _ptr(gamma), float(eps), _ptr(s_x), M, K, _ptr(y), _ptr(q),
        _stream(stream)), "fp8bq_add_rmsnorm_static_quant_act")


# ---------------------------------------------------------------- static GEMM

def fp8bq_static_gemm(q, s_x, w, s_w_part, part_sizes, y, ws, bias=None, stream=None):
    M, K = _mat(q, "q")
    N = _mat(w, "w")[0]
    arr, n = _parts(part_sizes)
    _validate("fp8bq_static_gemm", [
        _Spec("q", q, _E4M3, (M, K)),
        _Spec("s_x", s_x, _F32, numel=1),
        _Spec("w", w, _E4M3, (N, K)),
        _Spec("s_w_part", s_w_part, _F32, numel=n),
        _Spec("y", y, _BF16, (M, N)), _bias(bias, N), _ws(ws)], stream)
    _check(_lib.fp8bq_static_gemm(_ptr(q), _ptr(s_x), _ptr(w), _ptr(s_w_part), arr, n,
                                  _ptr(bias), _ptr(y), M, N, K, _ptr(ws), _nbytes(ws),
                                  _stream(stream)), "fp8bq_static_gemm")


def fp8bq_static_linear(x, s_x, w, s_w_part, part_sizes, y, ws, bias=None, stream=None):
    M, N, K, specs = _linear_specs(x, w, y, bias)
    arr, n = _parts(part_sizes)
    _validate("fp8bq_static_linear", specs + [
        _Spec("s_x", s_x, _F32, numel=1),
        _Spec("s_w_part", s_w_part, _F32, numel=n), _ws(ws)], stream)
    _check(_lib.fp8bq_static_linear(_ptr(x), _ld(x), _ptr(s_x), _ptr(w), _ptr(s_w_part),
                                    arr, n, _ptr(bias), _ptr(y), M, N, K, _ptr(ws),
                                    _nbytes(ws), _stream(stream)), "fp8bq_static_linear")


# ---------------------------------------------------------------- set-up helpers

def fp8bq_quant_weight_block(w, q, s_w, stream=None):
    N, K = _mat(w, "w")
    _validate("fp8bq_quant_weight_block", [
        _Spec("w", w, _BF16, (N, K), kind="rows"),
        _Spec("q", q, _E4M3, (N, K)),
        _Spec("s_w", s_w, _F32, (_kb(N), _kb(K)))], stream)
    _check(_lib.fp8bq_quant_weight_block(_ptr(w), N, K, _ld(w), _ptr(q), _ptr(s_w),
                                         _stream(stream)), "fp8bq_quant_weight_block")


def fp8bq_absmax_scale(x, s, stream=None):
    rows, K = _mat(x, "x")
    _validate("fp8bq_absmax_scale", [
        _Spec("x", x, _BF16, (rows, K), kind="rows"),
        _Spec("s", s, _F32, numel=1)], stream)
    _check(_lib.fp8bq_absmax_scale(_ptr(x), rows, K, _ld(x), _ptr(s), _stream(stream)),
           "fp8bq_absmax_scale")


def fp8bq_e4m3_from_bits(first: int, codes, stream=None):
    """codes[i] = the quantisers' E4M3 conversion of the binary32 value with bit
    pattern first + i, for every element of the uint8 tensor `codes`."""
    _validate("fp8bq_e4m3_from_bits", [_Spec("codes", codes, _U8, numel=codes.numel()
                                             if isinstance(codes, torch.Tensor) else None)],
              stream)
    _check(_lib.fp8bq_e4m3_from_bits(first, codes.numel(), _ptr(codes), _stream(stream)),
           "fp8bq_e4m3_from_bits")
