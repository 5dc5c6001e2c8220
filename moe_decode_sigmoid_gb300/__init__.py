"""Python binding of the Flint decode-MoE C ABI (include/flint_moe.h).

Argument marshalling only: every function below forwards torch tensors' device
pointers and the current CUDA stream to the same-named C entry point in
lib/libflint_moe.so; every step of the layer runs in that library's CUDA
kernels.  There is no fallback: if the library is missing or fails to load,
importing the binding's functions raises.

The C entry points take bare pointers, so the binding checks what they cannot:
each tensor's dtype, shape (as include/flint_moe.h lays it out), contiguity and
device (all on the activations' CUDA device), raising FlintError with
FLINT_ERR_INVALID_ARG before anything is launched.  A plain int is taken as a
raw device pointer the caller vouches for.

Build the library with `python -m moe_decode_sigmoid_gb300.build` (or
`__graft_entry__.build()`).
"""
from __future__ import annotations

import ctypes
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libflint_moe.so")

FLINT_OK = 0
FLINT_ERR_INVALID_ARG = 1
FLINT_ERR_UNSUPPORTED = 2
FLINT_ERR_WORKSPACE = 3
FLINT_ERR_CUDA = 4
FLINT_ERR_DEVICE_TIMEOUT = 5
MAX_BATCH = 256

HIDDEN, N_EXPERTS, TOP_K, INTER, N_SHARED = 2048, 256, 6, 512, 1

# Every symbol include/flint_moe.h declares.
EXPORTS = (
    "flint_status_string", "flint_moe_workspace_bytes", "flint_moe_workspace_init",
    "flint_moe_get_device_status", "flint_moe_route", "flint_moe_bucket",
    "flint_moe_decode_bf16", "flint_moe_decode_nvfp4_w4a16", "flint_moe_rmsnorm_bf16",
    "flint_moe_debug_arm_stall", "flint_moe_gateup_bf16", "flint_moe_down_bf16",
    "flint_moe_decode_bf16_noalloc", "flint_qk_norm_rope_kv_bf16",
    "flint_moe_decode_bf16_prenorm",
    "flint_qk_norm_rope_kv_paged_bf16", "flint_qk_norm_rope_kv_paged_fp8",
    "flint_attn_workspace_bytes", "flint_attn_workspace_init",
    "flint_attn_get_device_status", "flint_attn_debug_arm_stall",
    "flint_attn_paged_bf16", "flint_attn_paged_fp8",
    "flint_prompt_workspace_bytes", "flint_prompt_workspace_init",
    "flint_prompt_get_device_status", "flint_prompt_debug_arm_stall", "flint_linear_bf16",
    "flint_grouped_linear_bf16", "flint_moe_select", "flint_moe_combine_bf16",
    "flint_moe_prompt_bf16",
)
NOALLOC_MAX_BATCH = 8
# Batches up to which flint_moe_decode_bf16_prenorm is one launch (the
# persistent kernel normalises its input itself); 5..8 tokens take the RMSNorm
# kernel + the persistent kernel, larger batches the RMSNorm + three kernels.
PRENORM_FUSED_MAX_BATCH = 4


class FlintError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, status_string(status)))


FLINT_OFFSET_LOGIT = 0    # offsets move ranking and weights (default)
FLINT_OFFSET_SELECT = 1   # offsets steer the ranking only


class Dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("offset_mode", ctypes.c_int32)]


FULL_DIMS = Dims(HIDDEN, N_EXPERTS, TOP_K, INTER, N_SHARED, FLINT_OFFSET_LOGIT)
SELECT_DIMS = Dims(HIDDEN, N_EXPERTS, TOP_K, INTER, N_SHARED, FLINT_OFFSET_SELECT)

# The attention side of a decode step (flint_qk_norm_rope_kv_bf16).
N_Q_HEADS, N_KV_HEADS, HEAD_DIM = 32, 4, 128


class AttnDims(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


ATTN_DIMS = AttnDims(N_Q_HEADS, N_KV_HEADS, HEAD_DIM)

# The paged KV cache (flint_qk_norm_rope_kv_paged_*, flint_attn_paged_*).
KV_BLOCK = 16                  # token rows that share a scale in an E4M3 cache
PAGED_MAX_SEQS, PAGED_MAX_TOKENS = 256, 8192
PAGED_MAX_LENGTH = 1 << 23     # tokens a row of the page table has room for
_INT32_MAX = (1 << 31) - 1

# The linear side of a prompt (flint_linear_bf16, flint_grouped_linear_bf16, flint_moe_select,
# flint_moe_combine_bf16, flint_moe_prompt_bf16).
FLINT_ACT_NONE, FLINT_ACT_SILU, FLINT_ACT_GELU, FLINT_ACT_SWIGLU = 0, 1, 2, 3
LINEAR_MAX_ROWS, LINEAR_MAX_IN, LINEAR_MAX_OUT, LINEAR_MAX_GROUPS = 65536, 65536, 1 << 20, 1024


class LinearDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_in", "n_out", "act", "out_f32")]



class _PagedBatchStruct(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_seqs", "max_q_len", "page_size", "max_pages",
                                               "n_pages")] +
                [(n, ctypes.c_void_p) for n in ("q_start", "kv_len", "page_table")])


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """Loads the CUDA library (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("libflint_moe.so not built (%s); run moe_decode_sigmoid_gb300/build.py"
                          % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    L.flint_status_string.restype = ctypes.c_char_p
    L.flint_status_string.argtypes = [ctypes.c_int]
    L.flint_moe_workspace_bytes.restype = _SZ
    L.flint_moe_workspace_bytes.argtypes = [_P, _I32]
    L.flint_moe_workspace_init.restype = ctypes.c_int
    L.flint_moe_workspace_init.argtypes = [_P, _SZ, ctypes.c_uint64, _P]
    L.flint_moe_get_device_status.restype = ctypes.c_int
    L.flint_moe_get_device_status.argtypes = [_P, _P]
    L.flint_moe_debug_arm_stall.restype = ctypes.c_int
    L.flint_moe_debug_arm_stall.argtypes = [_P, _SZ, _P]
    L.flint_moe_route.restype = ctypes.c_int
    L.flint_moe_route.argtypes = [_P, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]
    L.flint_moe_bucket.restype = ctypes.c_int
    L.flint_moe_bucket.argtypes = [_P, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]
    L.flint_moe_decode_bf16.restype = ctypes.c_int
    L.flint_moe_decode_bf16.argtypes = [_P, _I32] + [_P] * 12 + [_SZ, _P]
    L.flint_moe_decode_nvfp4_w4a16.restype = ctypes.c_int
    L.flint_moe_decode_nvfp4_w4a16.argtypes = [_P, _I32] + [_P] * 20 + [_SZ, _P]
    L.flint_moe_gateup_bf16.restype = ctypes.c_int
    L.flint_moe_gateup_bf16.argtypes = [_P, _I32, _P, _P, _P, _P, _SZ, _P]
    L.flint_moe_down_bf16.restype = ctypes.c_int
    L.flint_moe_down_bf16.argtypes = [_P, _I32, _P, _P, _P, _P, _P, _SZ, _P]
    L.flint_moe_rmsnorm_bf16.restype = ctypes.c_int
    L.flint_moe_rmsnorm_bf16.argtypes = [_P, _I32, _P, _P, ctypes.c_float, _P]
    L.flint_moe_decode_bf16_prenorm.restype = ctypes.c_int
    L.flint_moe_decode_bf16_prenorm.argtypes = ([_P, _I32, _P, ctypes.c_float] + [_P] * 10 +
                                                [_SZ, _P])
    L.flint_moe_decode_bf16_noalloc.restype = ctypes.c_int
    L.flint_moe_decode_bf16_noalloc.argtypes = [_P, _I32] + [_P] * 13
    L.flint_qk_norm_rope_kv_bf16.restype = ctypes.c_int
    L.flint_qk_norm_rope_kv_bf16.argtypes = ([_P, _I32] + [_P] * 5 + [ctypes.c_float] * 2 +
                                             [_P] * 3 + [ctypes.c_int64, _P])
    L.flint_qk_norm_rope_kv_paged_bf16.restype = ctypes.c_int
    L.flint_qk_norm_rope_kv_paged_bf16.argtypes = ([_P, _P, _I32] + [_P] * 3 +
                                                   [ctypes.c_float] * 2 + [_P] * 4)
    L.flint_qk_norm_rope_kv_paged_fp8.restype = ctypes.c_int
    L.flint_qk_norm_rope_kv_paged_fp8.argtypes = ([_P, _P, _I32] + [_P] * 3 +
                                                  [ctypes.c_float] * 2 + [_P] * 6)
    L.flint_attn_workspace_bytes.restype = _SZ
    L.flint_attn_workspace_bytes.argtypes = [_P]
    L.flint_attn_workspace_init.restype = ctypes.c_int
    L.flint_attn_workspace_init.argtypes = [_P, _SZ, _P]
    L.flint_attn_get_device_status.restype = ctypes.c_int
    L.flint_attn_get_device_status.argtypes = [_P, _P]
    L.flint_attn_debug_arm_stall.restype = ctypes.c_int
    L.flint_attn_debug_arm_stall.argtypes = [_P, _SZ, _P]
    L.flint_attn_paged_bf16.restype = ctypes.c_int
    L.flint_attn_paged_bf16.argtypes = ([_P, _P, _I32] + [_P] * 4 + [ctypes.c_float, _I32] +
                                        [_P, _P, _SZ, _P])
    L.flint_attn_paged_fp8.restype = ctypes.c_int
    L.flint_attn_paged_fp8.argtypes = ([_P, _P, _I32] + [_P] * 6 + [ctypes.c_float, _I32] +
                                       [_P, _P, _SZ, _P])
    L.flint_prompt_workspace_bytes.restype = _SZ
    L.flint_prompt_workspace_bytes.argtypes = [_I32]
    L.flint_prompt_workspace_init.restype = ctypes.c_int
    L.flint_prompt_workspace_init.argtypes = [_P, _SZ, _P]
    L.flint_prompt_get_device_status.restype = ctypes.c_int
    L.flint_prompt_get_device_status.argtypes = [_P, _P]
    L.flint_prompt_debug_arm_stall.restype = ctypes.c_int
    L.flint_prompt_debug_arm_stall.argtypes = [_P, _SZ, _P]
    L.flint_linear_bf16.restype = ctypes.c_int
    L.flint_linear_bf16.argtypes = [_P, _I32] + [_P] * 6 + [_SZ, _P]
    L.flint_grouped_linear_bf16.restype = ctypes.c_int
    L.flint_grouped_linear_bf16.argtypes = [_P, _I32, _I32, _P, _P, _I32] + [_P] * 5 + [_SZ, _P]
    L.flint_moe_select.restype = ctypes.c_int
    L.flint_moe_select.argtypes = [_P, _I32] + [_P] * 8 + [_SZ, _P]
    L.flint_moe_combine_bf16.restype = ctypes.c_int
    L.flint_moe_combine_bf16.argtypes = [_P, _I32] + [_P] * 7
    L.flint_moe_prompt_bf16.restype = ctypes.c_int
    L.flint_moe_prompt_bf16.argtypes = [_P, _I32] + [_P] * 12 + [_SZ, _P]
    _lib = L
    return L


def status_string(status: int) -> str:
    try:
        return lib().flint_status_string(int(status)).decode()
    except ImportError:
        return "status %d" % status


def _check(status: int, where: str) -> None:
    if status != FLINT_OK:
        raise FlintError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_BF16, _F32, _I32T, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_Tensor = torch.Tensor


def _bad(where, name, what, t):
    got = ("%s %s%s on %s" % (t.dtype, tuple(t.shape), "" if t.is_contiguous() else
                              " (not contiguous)", t.device)
           if isinstance(t, torch.Tensor) else type(t).__name__)
    raise FlintError(FLINT_ERR_INVALID_ARG, "%s: %s must be %s, got %s" % (where, name, what, got))


def _arg(where, name, t, dtype, shape, dev, optional=False, min_numel=None):
    """Device pointer of t after checking it against the layout the C call
    assumes: dtype, exact shape (or at least min_numel elements), contiguous,
    on device dev."""
    if (type(t) is _Tensor and t.dtype is dtype and t.is_contiguous() and t.device == dev and
            t.shape == shape):
        return t.data_ptr()
    if t is None:
        if optional:
            return None
        raise FlintError(FLINT_ERR_INVALID_ARG, "%s: %s is required" % (where, name))
    if isinstance(t, int):
        return t
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == dev and
            (t.shape == shape if shape is not None else t.numel() >= min_numel) and
            t.is_contiguous()):
        what = "a contiguous %s tensor %s on %s" % (
            dtype, shape if shape is not None else "of >= %d elements" % min_numel, dev)
        _bad(where, name, what, t)
    return t.data_ptr()


def _batch(where, name, t, hidden):
    """(batch, device) of a [batch, hidden] activation tensor on the current
    CUDA device (the library launches on, and sizes its grids for, the
    current device)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2 and t.shape[1] == hidden):
        _bad(where, name, "a [batch, %d] tensor on a CUDA device" % hidden, t)
    _on_current_device(where, name, t)
    return t.shape[0], t.device


def _on_current_device(where, name, t):
    cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise FlintError(FLINT_ERR_INVALID_ARG,
                         "%s: %s is on %s but the current device is cuda:%d (use "
                         "torch.cuda.device(...) around the call)" % (where, name, t.device, cur))


def _ws_arg(where, workspace, dev):
    """(pointer, bytes) of a workspace: a contiguous uint8 tensor on dev."""
    if (type(workspace) is _Tensor and workspace.dtype is _U8 and workspace.dim() == 1 and
            workspace.device == dev and workspace.is_contiguous()):
        return workspace.data_ptr(), workspace.numel()
    if isinstance(workspace, torch.Tensor):
        if not (workspace.dtype == _U8 and workspace.dim() == 1 and workspace.device == dev and
                workspace.is_contiguous()):
            _bad(where, "workspace", "a contiguous 1-D uint8 tensor on %s" % dev, workspace)
    return _ws(workspace)


def _d(dims):
    return FULL_DIMS if dims is None else dims


def _stream(stream):
    if stream is None:  # torch.cuda.current_stream() without the Stream object it makes
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dims(dims):
    return ctypes.byref(FULL_DIMS if dims is None else dims)


# ---------------------------------------------------------------- entry points

def flint_moe_workspace_bytes(max_batch: int, dims: Dims | None = None) -> int:
    return int(lib().flint_moe_workspace_bytes(_dims(dims), int(max_batch)))


def _ws_only(where, workspace):
    """(pointer, bytes) of a workspace passed on its own: a contiguous uint8
    tensor on the current CUDA device."""
    if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda):
        _bad(where, "workspace", "a contiguous 1-D uint8 tensor on a CUDA device", workspace)
    _on_current_device(where, "workspace", workspace)
    return _ws_arg(where, workspace, workspace.device)


def flint_moe_workspace_init(workspace: torch.Tensor, wait_limit_ns: int = 0, stream=None):
    wp, wb = _ws_only("flint_moe_workspace_init", workspace)
    _check(lib().flint_moe_workspace_init(wp, wb, int(wait_limit_ns), _stream(stream)),
           "flint_moe_workspace_init")


def flint_moe_get_device_status(workspace: torch.Tensor, stream=None) -> int:
    wp, _ = _ws_only("flint_moe_get_device_status", workspace)
    return int(lib().flint_moe_get_device_status(wp, _stream(stream)))


def flint_moe_debug_arm_stall(workspace: torch.Tensor, stream=None):
    wp, wb = _ws_only("flint_moe_debug_arm_stall", workspace)
    _check(lib().flint_moe_debug_arm_stall(wp, wb, _stream(stream)), "flint_moe_debug_arm_stall")


def _ws(workspace):
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def flint_moe_route(x, w_router, logit_bias, topk_idx, topk_w, workspace, stream=None,
                    dims: Dims | None = None):
    f, d = "flint_moe_route", _d(dims)
    B, dev = _batch(f, "x", x, d.hidden)
    args = (_arg(f, "x", x, _BF16, (B, d.hidden), dev),
            _arg(f, "w_router", w_router, _BF16, (d.n_experts, d.hidden), dev),
            _arg(f, "logit_bias", logit_bias, _F32, (d.n_experts,), dev, optional=True),
            _arg(f, "topk_idx", topk_idx, _I32T, (B, d.top_k), dev),
            _arg(f, "topk_w", topk_w, _F32, (B, d.top_k), dev))
    wp, wb = _ws_arg(f, workspace, dev)
    _check(lib().flint_moe_route(_dims(dims), B, *args, wp, wb, _stream(stream)), f)


def flint_moe_bucket(topk_idx, uniq, offsets, pairs, n_uniq, workspace, stream=None,
                     dims: Dims | None = None):
    f, d = "flint_moe_bucket", _d(dims)
    B, dev = _batch(f, "topk_idx", topk_idx, d.top_k)
    args = (_arg(f, "topk_idx", topk_idx, _I32T, (B, d.top_k), dev),
            _arg(f, "uniq", uniq, _I32T, None, dev, min_numel=d.n_experts),
            _arg(f, "offsets", offsets, _I32T, None, dev, min_numel=d.n_experts + 1),
            _arg(f, "pairs", pairs, _I32T, None, dev, min_numel=B * d.top_k),
            _arg(f, "n_uniq", n_uniq, _I32T, None, dev, min_numel=1))
    wp, wb = _ws_arg(f, workspace, dev)
    _check(lib().flint_moe_bucket(_dims(dims), B, *args, wp, wb, _stream(stream)), f)


def _layer_args(f, d, B, dev, x, residual, w_router, logit_bias, w13, w2, ws13, ws2, out,
                topk_idx_out, topk_w_out):
    """Checked pointers of the BF16 layer's arguments, in the C call's order."""
    H, E, K, I, S = d.hidden, d.n_experts, d.top_k, d.inter, d.n_shared
    return (_arg(f, "x", x, _BF16, (B, H), dev),
            _arg(f, "residual", residual, _BF16, (B, H), dev),
            _arg(f, "w_router", w_router, _BF16, (E, H), dev),
            _arg(f, "logit_bias", logit_bias, _F32, (E,), dev, optional=True),
            _arg(f, "w13", w13, _BF16, (E, 2 * I, H), dev),
            _arg(f, "w2", w2, _BF16, (E, H, I), dev),
            _arg(f, "ws13", ws13, _BF16, (S, 2 * I, H), dev),
            _arg(f, "ws2", ws2, _BF16, (S, H, I), dev),
            _arg(f, "out", out, _BF16, (B, H), dev),
            _arg(f, "topk_idx_out", topk_idx_out, _I32T, (B, K), dev, optional=True),
            _arg(f, "topk_w_out", topk_w_out, _F32, (B, K), dev, optional=True))


def flint_moe_decode_bf16(x, residual, w_router, logit_bias, w13, w2, ws13, ws2, out, workspace,
                          topk_idx_out=None, topk_w_out=None, stream=None,
                          dims: Dims | None = None):
    f, d = "flint_moe_decode_bf16", _d(dims)
    B, dev = _batch(f, "x", x, d.hidden)
    args = _layer_args(f, d, B, dev, x, residual, w_router, logit_bias, w13, w2, ws13, ws2, out,
                       topk_idx_out, topk_w_out)
    wp, wb = _ws_arg(f, workspace, dev)
    _check(lib().flint_moe_decode_bf16(_dims(dims), B, *args, wp, wb, _stream(stream)), f)


def flint_moe_decode_bf16_prenorm(residual, w_router, logit_bias, w13, w2, ws13, ws2, out,
                                  workspace, norm_eps: float = 1e-6, topk_idx_out=None,
                                  topk_w_out=None, stream=None, dims: Dims | None = None):
    """flint_moe_decode_bf16 whose input is RMSNorm(residual) (unit gain,
    norm_eps), computed inside the call: one launch per layer for batches of
    at most 8 tokens."""
    f, d = "flint_moe_decode_bf16_prenorm", _d(dims)
    B, dev = _batch(f, "residual", residual, d.hidden)
    args = _layer_args(f, d, B, dev, residual, residual, w_router, logit_bias, w13, w2, ws13, ws2,
                       out, topk_idx_out, topk_w_out)
    wp, wb = _ws_arg(f, workspace, dev)
    _check(lib().flint_moe_decode_bf16_prenorm(_dims(dims), B, args[1], float(norm_eps), *args[2:],
                                               wp, wb, _stream(stream)), f)


def flint_moe_decode_bf16_noalloc(x, residual, w_router, logit_bias, w13, w2, ws13, ws2, out,
                                  topk_idx_out=None, topk_w_out=None, device_status_out=None,
                                  stream=None, dims: Dims | None = None):
    """flint_moe_decode_bf16 without a workspace (the library's static device
    array instead; batch <= NOALLOC_MAX_BATCH).  For callers that cannot
    allocate device memory; calls whose GPU work overlaps race."""
    f, d = "flint_moe_decode_bf16_noalloc", _d(dims)
    B, dev = _batch(f, "x", x, d.hidden)
    args = _layer_args(f, d, B, dev, x, residual, w_router, logit_bias, w13, w2, ws13, ws2, out,
                       topk_idx_out, topk_w_out)
    st = _arg(f, "device_status_out", device_status_out, _I32T, None, dev, optional=True,
              min_numel=1)
    _check(lib().flint_moe_decode_bf16_noalloc(_dims(dims), B, *args, st, _stream(stream)), f)


def flint_moe_gateup_bf16(x, w13, ws13, workspace, stream=None, dims: Dims | None = None):
    f, d = "flint_moe_gateup_bf16", _d(dims)
    B, dev = _batch(f, "x", x, d.hidden)
    args = (_arg(f, "x", x, _BF16, (B, d.hidden), dev),
            _arg(f, "w13", w13, _BF16, (d.n_experts, 2 * d.inter, d.hidden), dev),
            _arg(f, "ws13", ws13, _BF16, (d.n_shared, 2 * d.inter, d.hidden), dev))
    wp, wb = _ws_arg(f, workspace, dev)
    _check(lib().flint_moe_gateup_bf16(_dims(dims), B, *args, wp, wb, _stream(stream)), f)


def flint_moe_down_bf16(residual, w2, ws2, out, workspace, stream=None, dims: Dims | None = None):
    f, d = "flint_moe_down_bf16", _d(dims)
    B, dev = _batch(f, "residual", residual, d.hidden)
    args = (_arg(f, "residual", residual, _BF16, (B, d.hidden), dev),
            _arg(f, "w2", w2, _BF16, (d.n_experts, d.hidden, d.inter), dev),
            _arg(f, "ws2", ws2, _BF16, (d.n_shared, d.hidden, d.inter), dev),
            _arg(f, "out", out, _BF16, (B, d.hidden), dev))
    wp, wb = _ws_arg(f, workspace, dev)
    _check(lib().flint_moe_down_bf16(_dims(dims), B, *args, wp, wb, _stream(stream)), f)


NVFP4_KEYS = ("w13_q", "w13_sf", "w13_ts", "w2_q", "w2_sf", "w2_ts",
              "ws13_q", "ws13_sf", "ws13_ts", "ws2_q", "ws2_sf", "ws2_ts")


def flint_moe_decode_nvfp4_w4a16(x, residual, w_router, logit_bias, nv: dict, out, workspace,
                                 topk_idx_out=None, topk_w_out=None, stream=None,
                                 dims: Dims | None = None):
    """nv holds the twelve packed tensors named in NVFP4_KEYS."""
    f, d = "flint_moe_decode_nvfp4_w4a16", _d(dims)
    H, E, K, I, S = d.hidden, d.n_experts, d.top_k, d.inter, d.n_shared
    B, dev = _batch(f, "x", x, H)
    shapes = {}
    for pre, n in (("w", E), ("ws", S)):
        shapes[pre + "13_q"] = (_U8, (n, 2 * I, H // 2))
        shapes[pre + "13_sf"] = (_U8, (n, 2 * I, H // 16))
        shapes[pre + "13_ts"] = (_F32, (n, 2))
        shapes[pre + "2_q"] = (_U8, (n, H, I // 2))
        shapes[pre + "2_sf"] = (_U8, (n, H, I // 16))
        shapes[pre + "2_ts"] = (_F32, (n,))
    packed = [_arg(f, k, nv.get(k), shapes[k][0], shapes[k][1], dev) for k in NVFP4_KEYS]
    args = (_arg(f, "x", x, _BF16, (B, H), dev),
            _arg(f, "residual", residual, _BF16, (B, H), dev),
            _arg(f, "w_router", w_router, _BF16, (E, H), dev),
            _arg(f, "logit_bias", logit_bias, _F32, (E,), dev, optional=True),
            *packed,
            _arg(f, "out", out, _BF16, (B, H), dev),
            _arg(f, "topk_idx_out", topk_idx_out, _I32T, (B, K), dev, optional=True),
            _arg(f, "topk_w_out", topk_w_out, _F32, (B, K), dev, optional=True))
    wp, wb = _ws_arg(f, workspace, dev)
    _check(lib().flint_moe_decode_nvfp4_w4a16(_dims(dims), B, *args, wp, wb, _stream(stream)), f)


def flint_moe_rmsnorm_bf16(inp, out, eps: float = 1e-6, stream=None, dims: Dims | None = None):
    f, d = "flint_moe_rmsnorm_bf16", _d(dims)
    B, dev = _batch(f, "inp", inp, d.hidden)
    args = (_arg(f, "inp", inp, _BF16, (B, d.hidden), dev),
            _arg(f, "out", out, _BF16, (B, d.hidden), dev))
    _check(lib().flint_moe_rmsnorm_bf16(_dims(dims), B, *args, float(eps), _stream(stream)), f)


def flint_qk_norm_rope_kv_bf16(qkv, q_norm, k_norm, positions, slot_mapping, q_out, k_cache,
                               v_cache, rope_theta: float, eps: float = 1e-6, stream=None):
    """Per-head Q/K RMSNorm + RoPE (rope_theta = 0: none) of a decode step's
    projection rows qkv [B, (32 + 2*4) * 128], writing the query heads to
    q_out [B, 32, 128] and the key / value heads to row slot_mapping[t] of
    k_cache / v_cache [slots, 4, 128]; positions and slot_mapping are int32 [B]."""
    f = "flint_qk_norm_rope_kv_bf16"
    row = (N_Q_HEADS + 2 * N_KV_HEADS) * HEAD_DIM
    B, dev = _batch(f, "qkv", qkv, row)
    if not (isinstance(k_cache, torch.Tensor) and k_cache.dim() == 3):
        _bad(f, "k_cache", "a [slots, %d, %d] tensor" % (N_KV_HEADS, HEAD_DIM), k_cache)
    slots = k_cache.shape[0]
    cache = (slots, N_KV_HEADS, HEAD_DIM)
    args = (_arg(f, "qkv", qkv, _BF16, (B, row), dev),
            _arg(f, "q_norm", q_norm, _BF16, (HEAD_DIM,), dev),
            _arg(f, "k_norm", k_norm, _BF16, (HEAD_DIM,), dev),
            _arg(f, "positions", positions, _I32T, (B,), dev),
            _arg(f, "slot_mapping", slot_mapping, _I32T, (B,), dev))
    outs = (_arg(f, "q_out", q_out, _BF16, (B, N_Q_HEADS, HEAD_DIM), dev),
            _arg(f, "k_cache", k_cache, _BF16, cache, dev),
            _arg(f, "v_cache", v_cache, _BF16, cache, dev))
    _check(lib().flint_qk_norm_rope_kv_bf16(ctypes.byref(ATTN_DIMS), B, *args, float(rope_theta),
                                            float(eps), *outs, slots, _stream(stream)), f)


# ---------------------------------------------------------------- the paged KV cache

class PagedBatch:
    """Which tokens a paged call brings and where their sequences' caches lie
    (flint_paged_batch): q_start int32 [n + 1], kv_len int32 [n] (the new tokens
    included) and page_table int32 [n, max_pages], contiguous tensors on one
    CUDA device, which a program may refill in place between calls; page_size
    tokens per page (a power of two, 16 to 1024); max_q_len an upper bound of
    the new tokens of any one sequence (1: the next token of each).  Checked
    here once; the calls only check that they run on its device."""

    def __init__(self, q_start, kv_len, page_table, page_size: int, max_q_len: int):
        f = "PagedBatch"
        page_size, max_q_len = int(page_size), int(max_q_len)
        # The C struct's fields have 32 bits, and ctypes cuts numbers beyond them.
        if (page_size not in (16, 32, 64, 128, 256, 512, 1024) or
                not 1 <= max_q_len <= _INT32_MAX):
            raise FlintError(FLINT_ERR_INVALID_ARG, "%s: page_size %d, max_q_len %d" %
                             (f, page_size, max_q_len))
        if not (isinstance(page_table, torch.Tensor) and page_table.is_cuda and
                page_table.dim() == 2):
            _bad(f, "page_table", "a [sequences, pages] tensor on a CUDA device", page_table)
        n, max_pages = page_table.shape
        dev = page_table.device
        if not (1 <= n <= PAGED_MAX_SEQS and 1 <= max_pages <= PAGED_MAX_LENGTH // page_size):
            _bad(f, "page_table", "of 1 to %d sequences and of 1 to %d pages of %d tokens" %
                 (PAGED_MAX_SEQS, PAGED_MAX_LENGTH // page_size, page_size), page_table)
        self.tensors = (q_start, kv_len, page_table)  # kept alive with the batch
        self.device, self.n_seqs, self.page_size, self.max_q_len = dev, n, page_size, max_q_len
        self.index = dev.index
        self._fields = (n, max_q_len, page_size, max_pages)
        self._pointers = (_arg(f, "q_start", q_start, _I32T, (n + 1,), dev),
                          _arg(f, "kv_len", kv_len, _I32T, (n,), dev),
                          _arg(f, "page_table", page_table, _I32T, (n, max_pages), dev))
        self._for = (0, None)  # the C struct for caches of so many pages

    def _ref(self, n_pages):
        """The C struct, by reference, for caches of n_pages pages."""
        pages, ref = self._for
        if pages != n_pages:
            ref = ctypes.byref(_PagedBatchStruct(*self._fields, n_pages, *self._pointers))
            self._for = (n_pages, ref)
        return ref


def _paged(where, name, rows, batch, k_cache, hd, nkv):
    """(rows, device, pages, C struct) of a paged call after checking its batch
    and device; rows [n_tokens, ...] on the current CUDA device."""
    if type(batch) is not PagedBatch:
        raise FlintError(FLINT_ERR_INVALID_ARG, "%s: batch must be a PagedBatch, got %s" %
                         (where, type(batch).__name__))
    dev = batch.device
    shape = rows.shape if isinstance(rows, _Tensor) else ()
    if not (len(shape) >= 2 and 1 <= shape[0] <= PAGED_MAX_TOKENS and rows.device == dev):
        _bad(where, name, "of 1 to %d token rows on %s" % (PAGED_MAX_TOKENS, dev), rows)
    if batch.index != torch._C._cuda_getDevice():
        _on_current_device(where, name, rows)
    cache = k_cache.shape if isinstance(k_cache, _Tensor) else ()
    if not (len(cache) == 4 and cache[0] >= 1):
        _bad(where, "k_cache", "a [pages, %d, %d, %d] tensor" % (batch.page_size, nkv, hd), k_cache)
    return shape[0], dev, cache[0], batch._ref(cache[0])


def _heads(dims):
    """(query heads, KV heads, head size, C struct by reference) of a call."""
    if dims is None:
        return N_Q_HEADS, N_KV_HEADS, HEAD_DIM, _ATTN_DIMS_REF
    return dims.n_q_heads, dims.n_kv_heads, dims.head_dim, ctypes.byref(dims)


_ATTN_DIMS_REF = ctypes.byref(ATTN_DIMS)


def _append(f, qkv, q_norm, k_norm, batch, q_out, k_cache, v_cache, scales, dtype, rope_theta, eps,
            stream, dims):
    nq, nkv, hd, d = _heads(dims)
    T, dev, pages, b = _paged(f, "qkv", qkv, batch, k_cache, hd, nkv)
    cache = (pages, batch.page_size, nkv, hd)
    args = (_arg(f, "qkv", qkv, _BF16, (T, (nq + 2 * nkv) * hd), dev),
            _arg(f, "q_norm", q_norm, _BF16, (hd,), dev),
            _arg(f, "k_norm", k_norm, _BF16, (hd,), dev), rope_theta, eps,
            _arg(f, "q_out", q_out, _BF16, (T, nq, hd), dev),
            _arg(f, "k_cache", k_cache, dtype, cache, dev),
            _arg(f, "v_cache", v_cache, dtype, cache, dev))
    if scales:
        blocks = (pages, batch.page_size // KV_BLOCK, nkv)
        args += (_arg(f, "k_scale", scales[0], _F32, blocks, dev),
                 _arg(f, "v_scale", scales[1], _F32, blocks, dev))
    _check(getattr(_lib or lib(), f)(d, b, T, *args, _stream(stream)), f)


def flint_qk_norm_rope_kv_paged_bf16(qkv, q_norm, k_norm, batch: PagedBatch, q_out, k_cache,
                                     v_cache, rope_theta: float, eps: float = 1e-6, stream=None,
                                     dims: AttnDims | None = None):
    """Per-head Q/K RMSNorm + RoPE (rope_theta = 0: none) of the projection rows
    qkv [T, (nq + 2 nkv) * 128] of a PagedBatch: query heads to q_out
    [T, nq, 128], keys and values to k_cache / v_cache [pages, page_size, nkv,
    128] (bf16) at the rows the batch's page table gives."""
    _append("flint_qk_norm_rope_kv_paged_bf16", qkv, q_norm, k_norm, batch, q_out, k_cache,
            v_cache, None, _BF16, rope_theta, eps, stream, dims)


def flint_qk_norm_rope_kv_paged_fp8(qkv, q_norm, k_norm, batch: PagedBatch, q_out, k_cache,
                                    v_cache, k_scale, v_scale, rope_theta: float,
                                    eps: float = 1e-6, stream=None, dims: AttnDims | None = None):
    """flint_qk_norm_rope_kv_paged_bf16 into an E4M3 cache: uint8 codes
    [pages, page_size, nkv, 128] and fp32 power-of-two scales
    [pages, page_size / 16, nkv] per 16-token block and head."""
    _append("flint_qk_norm_rope_kv_paged_fp8", qkv, q_norm, k_norm, batch, q_out, k_cache, v_cache,
            (k_scale, v_scale), _U8, rope_theta, eps, stream, dims)


def flint_attn_workspace_bytes(dims: AttnDims | None = None) -> int:
    return int(lib().flint_attn_workspace_bytes(ctypes.byref(ATTN_DIMS if dims is None else dims)))


def flint_attn_workspace_init(workspace: torch.Tensor, stream=None):
    wp, wb = _ws_only("flint_attn_workspace_init", workspace)
    _check(lib().flint_attn_workspace_init(wp, wb, _stream(stream)), "flint_attn_workspace_init")


def flint_attn_get_device_status(workspace: torch.Tensor, stream=None) -> int:
    wp, _ = _ws_only("flint_attn_get_device_status", workspace)
    return int(lib().flint_attn_get_device_status(wp, _stream(stream)))


def flint_attn_debug_arm_stall(workspace: torch.Tensor, stream=None):
    wp, wb = _ws_only("flint_attn_debug_arm_stall", workspace)
    _check(lib().flint_attn_debug_arm_stall(wp, wb, _stream(stream)), "flint_attn_debug_arm_stall")


def _window(where, window):
    """The window as an int of 32 bits, beyond which ctypes would cut it."""
    try:
        w = operator.index(window)
    except TypeError:
        w = -1
    if not 0 <= w <= _INT32_MAX:
        raise FlintError(FLINT_ERR_INVALID_ARG, "%s: window must be a whole number of 0 to %d, "
                         "got %r" % (where, _INT32_MAX, window))
    return w


def _attend(f, q, k_cache, v_cache, scales, dtype, batch, out, workspace, sinks, window,
            softmax_scale, stream, dims):
    if type(window) is not int or not 0 <= window <= _INT32_MAX:
        window = _window(f, window)
    nq, nkv, hd, d = _heads(dims)
    T, dev, pages, b = _paged(f, "q", q, batch, k_cache, hd, nkv)
    cache, rows = (pages, batch.page_size, nkv, hd), (T, nq, hd)
    args = (_arg(f, "q", q, _BF16, rows, dev),
            _arg(f, "k_cache", k_cache, dtype, cache, dev),
            _arg(f, "v_cache", v_cache, dtype, cache, dev))
    if scales:
        blocks = (pages, batch.page_size // KV_BLOCK, nkv)
        args += (_arg(f, "k_scale", scales[0], _F32, blocks, dev),
                 _arg(f, "v_scale", scales[1], _F32, blocks, dev))
    wp, wb = _ws_arg(f, workspace, dev)
    _check(getattr(_lib or lib(), f)(
        d, b, T, *args,
        None if sinks is None else _arg(f, "sinks", sinks, _F32, (nq,), dev),
        hd ** -0.5 if softmax_scale is None else softmax_scale, window,
        _arg(f, "out", out, _BF16, rows, dev), wp, wb, _stream(stream)), f)


def flint_attn_paged_bf16(q, k_cache, v_cache, batch: PagedBatch, out, workspace, sinks=None,
                          window: int = 0, softmax_scale: float | None = None, stream=None,
                          dims: AttnDims | None = None):
    """Grouped-query attention of the rows q [T, nq, 128] of a PagedBatch over
    its bf16 cache [pages, page_size, nkv, 128], causal, over the last `window`
    positions (0: all), with optional learned sinks fp32 [nq] in the softmax's
    denominator, into out [T, nq, 128].  softmax_scale defaults to 128 ** -0.5;
    workspace: new_attn_workspace()."""
    _attend("flint_attn_paged_bf16", q, k_cache, v_cache, None, _BF16, batch, out, workspace, sinks,
            window, softmax_scale, stream, dims)


def flint_attn_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, batch: PagedBatch, out, workspace,
                         sinks=None, window: int = 0, softmax_scale: float | None = None,
                         stream=None, dims: AttnDims | None = None):
    """flint_attn_paged_bf16 over an E4M3 cache (uint8 codes and fp32 scales as
    flint_qk_norm_rope_kv_paged_fp8 writes them)."""
    _attend("flint_attn_paged_fp8", q, k_cache, v_cache, (k_scale, v_scale), _U8, batch, out,
            workspace, sinks, window, softmax_scale, stream, dims)


# ---------------------------------------------------------------- the linear side of a prompt

def flint_prompt_workspace_bytes(max_tokens: int = 0) -> int:
    n = operator.index(max_tokens)
    return int(lib().flint_prompt_workspace_bytes(n)) if 0 <= n <= PAGED_MAX_TOKENS else 0


def flint_prompt_workspace_init(workspace: torch.Tensor, stream=None):
    wp, wb = _ws_only("flint_prompt_workspace_init", workspace)
    _check(lib().flint_prompt_workspace_init(wp, wb, _stream(stream)), "flint_prompt_workspace_init")


def flint_prompt_get_device_status(workspace: torch.Tensor, stream=None) -> int:
    wp, _ = _ws_only("flint_prompt_get_device_status", workspace)
    return int(lib().flint_prompt_get_device_status(wp, _stream(stream)))


def flint_prompt_debug_arm_stall(workspace: torch.Tensor, stream=None):
    wp, wb = _ws_only("flint_prompt_debug_arm_stall", workspace)
    _check(lib().flint_prompt_debug_arm_stall(wp, wb, _stream(stream)),
           "flint_prompt_debug_arm_stall")


_current_gpu, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream

# (C struct by reference, rows of a weight matrix) of a linear call, by its n_in, n_out, act and
# whether out is fp32.
_LINEAR_DIMS = {}


def _linear_dims(f, x, out, act):
    """The entry of _LINEAR_DIMS that x and out need, made; raises if they or act cannot be."""
    if not (isinstance(x, _Tensor) and x.is_cuda and x.dim() == 2 and
            8 <= x.shape[1] <= LINEAR_MAX_IN):
        _bad(f, "x", "[rows, 8 to %d] on a CUDA device" % LINEAR_MAX_IN, x)
    if not (isinstance(out, _Tensor) and out.dim() == 2 and 8 <= out.shape[1] <= LINEAR_MAX_OUT and
            (out.dtype is _BF16 or out.dtype is _F32)):
        _bad(f, "out", "a bf16 or float32 tensor [rows, 8 to %d]" % LINEAR_MAX_OUT, out)
    if type(act) is not int or not FLINT_ACT_NONE <= act <= FLINT_ACT_SWIGLU:
        raise FlintError(FLINT_ERR_UNSUPPORTED, "%s: act must be one of FLINT_ACT_*, got %r" %
                         (f, act))
    k, n, f32 = x.shape[1], out.shape[1], out.dtype is _F32
    return _LINEAR_DIMS.setdefault(
        (k, n, act, f32), (ctypes.byref(LinearDims(k, n, act, int(f32))),
                           2 * n if act == FLINT_ACT_SWIGLU else n))


def _linear(f, x, out, act):
    """(C struct by reference, device, rows of x, n_in, rows of out, n_out, out's type, rows of a
    weight matrix) of a linear call; the calls check what is left of x and out."""
    dtype = getattr(out, "dtype", None)
    try:
        n_x, k = x.shape
        rows, n = out.shape
        if type(act) is not int:   # 1.0 and True would find the entry of 1
            raise KeyError(act)
        ref, m = _LINEAR_DIMS[k, n, act, dtype is _F32]
    except (AttributeError, ValueError, TypeError, KeyError):
        ref, m = _linear_dims(f, x, out, act)
        (n_x, k), (rows, n) = x.shape, out.shape
    if dtype is not _F32:
        dtype = _BF16
    for name, t, r in (("x", x, n_x), ("out", out, rows)):
        if not 1 <= r <= LINEAR_MAX_ROWS:
            _bad(f, name, "of 1 to %d rows" % LINEAR_MAX_ROWS, t)
    dev = x.device
    if dev.index != torch._C._cuda_getDevice():
        _on_current_device(f, "x", x)
    return ref, dev, n_x, k, rows, n, dtype, m


def flint_linear_bf16(x, w, out, workspace, bias=None, residual=None, act: int = FLINT_ACT_NONE,
                      stream=None):
    """out = act(x w^T + bias) + residual: x bf16 [rows, n_in], w bf16 [n_out, n_in]
    (FLINT_ACT_SWIGLU: [2 n_out, n_in], gate rows first), bias fp32 of one value per row
    of w, residual and out [rows, n_out] of one type, bf16 or fp32 (residual may be out
    itself); workspace: new_prompt_workspace()."""
    f = "flint_linear_bf16"
    try:  # everything in order, in one look: half the look-ups of the checks that can say what is not
        rows, k = x.shape
        r, n = out.shape
        f32 = out.dtype is _F32
        ref, m = _LINEAR_DIMS[k, n, act, f32]
        gpu = _current_gpu()
        good = (type(act) is int and r == rows <= LINEAR_MAX_ROWS and x.dtype is _BF16 and
                w.dtype is _BF16 and (f32 or out.dtype is _BF16) and w.shape == (m, k) and x.is_contiguous() and
                w.is_contiguous() and out.is_contiguous() and
                x.get_device() == w.get_device() == out.get_device() == workspace.get_device() == gpu and
                workspace.dtype is _U8 and workspace.dim() == 1 and workspace.is_contiguous())
    except (AttributeError, ValueError, TypeError, LookupError, RuntimeError):
        good = False
    if good and rows > 0:
        dtype, dev = out.dtype, None if bias is None and residual is None else x.device
        args = (x.data_ptr(), w.data_ptr())
        last = (out.data_ptr(), workspace.data_ptr(), workspace.numel())
    else:
        ref, dev, rows, k, _, n, dtype, m = _linear(f, x, out, act)
        args = (_arg(f, "x", x, _BF16, (rows, k), dev), _arg(f, "w", w, _BF16, (m, k), dev))
        last = (_arg(f, "out", out, dtype, (rows, n), dev), *_ws_arg(f, workspace, dev))
        gpu = dev.index
    _check((_lib or lib()).flint_linear_bf16(
        ref, rows, *args,
        None if bias is None else _arg(f, "bias", bias, _F32, (m,), dev),
        None if residual is None else _arg(f, "residual", residual, dtype, (rows, n), dev),
        *last, _raw_stream(gpu) if stream is None else _stream(stream)), f)


def flint_grouped_linear_bf16(x, w, group_start, out, workspace, row_index=None, bias=None,
                              act: int = FLINT_ACT_NONE, stream=None):
    """out[r] = act(x[row_index[r]] w[g]^T + bias[g]) for the rows group_start[g] <= r <
    group_start[g + 1] of every group g: w bf16 [groups, n_out, n_in] (FLINT_ACT_SWIGLU:
    [groups, 2 n_out, n_in]), group_start int32 [groups + 1], row_index int32 of one
    value per row of out (None: x[r]), bias fp32 [groups, rows of a matrix]."""
    f = "flint_grouped_linear_bf16"
    try:  # as flint_linear_bf16
        n_x, k = x.shape
        rows, n = out.shape
        f32 = out.dtype is _F32
        ref, m = _LINEAR_DIMS[k, n, act, f32]
        groups = w.shape[0]
        gpu = _current_gpu()
        good = (type(act) is int and 0 < n_x <= LINEAR_MAX_ROWS and 0 < rows <= LINEAR_MAX_ROWS and
                0 < groups <= LINEAR_MAX_GROUPS and x.dtype is _BF16 and w.dtype is _BF16 and
                (f32 or out.dtype is _BF16) and group_start.dtype is _I32T and
                w.shape == (groups, m, k) and group_start.shape == (groups + 1,) and
                x.is_contiguous() and w.is_contiguous() and out.is_contiguous() and
                group_start.is_contiguous() and
                x.get_device() == w.get_device() == out.get_device() == group_start.get_device() ==
                workspace.get_device() == gpu and
                workspace.dtype is _U8 and workspace.dim() == 1 and workspace.is_contiguous())
    except (AttributeError, ValueError, TypeError, LookupError, RuntimeError):
        good = False
    if good:
        dev = None if bias is None and row_index is None else x.device
        start, xw = group_start.data_ptr(), (x.data_ptr(), w.data_ptr())
        last = (out.data_ptr(), workspace.data_ptr(), workspace.numel())
    else:
        ref, dev, n_x, k, rows, n, dtype, m = _linear(f, x, out, act)
        if not (isinstance(w, _Tensor) and w.dim() == 3 and 1 <= w.shape[0] <= LINEAR_MAX_GROUPS):
            _bad(f, "w", "[1 to %d groups, rows, n_in]" % LINEAR_MAX_GROUPS, w)
        groups = w.shape[0]
        start = _arg(f, "group_start", group_start, _I32T, (groups + 1,), dev)
        xw = (_arg(f, "x", x, _BF16, (n_x, k), dev), _arg(f, "w", w, _BF16, (groups, m, k), dev))
        last = (_arg(f, "out", out, dtype, (rows, n), dev), *_ws_arg(f, workspace, dev))
        gpu = dev.index
    if row_index is None and n_x != rows:
        _bad(f, "x", "of as many rows as out has (%d) without row_index" % rows, x)
    _check((_lib or lib()).flint_grouped_linear_bf16(
        ref, groups, rows, start,
        None if row_index is None else _arg(f, "row_index", row_index, _I32T, (rows,), dev), n_x, *xw,
        None if bias is None else _arg(f, "bias", bias, _F32, (groups, m), dev),
        *last, _raw_stream(gpu) if stream is None else _stream(stream)), f)


def _prompt_tokens(where, name, t):
    """(tokens, device) of a [tokens, width] tensor of a call for prompts; the calls check
    what is left of it."""
    shape = t.shape if isinstance(t, _Tensor) else ()
    if not (len(shape) == 2 and 1 <= shape[0] <= PAGED_MAX_TOKENS):
        _bad(where, name, "of 1 to %d tokens" % PAGED_MAX_TOKENS, t)
    dev = t.device
    if dev.type != "cuda":
        _bad(where, name, "on a CUDA device", t)
    if dev.index != torch._C._cuda_getDevice():
        _on_current_device(where, name, t)
    return shape[0], dev


_FULL_DIMS_REF, _SELECT_DIMS_REF = ctypes.byref(FULL_DIMS), ctypes.byref(SELECT_DIMS)


def _moe_dims(dims):
    """(dims, C struct by reference) of a call for prompts."""
    if dims is None or dims is FULL_DIMS:
        return FULL_DIMS, _FULL_DIMS_REF
    return dims, _SELECT_DIMS_REF if dims is SELECT_DIMS else ctypes.byref(dims)


def flint_moe_select(logits, logit_bias, topk_idx, topk_w, group_start, row_token, pair_row,
                     workspace, stream=None, dims: Dims | None = None):
    """The routing of router scores logits fp32 [T, 256] (topk_idx int32 and topk_w fp32
    [T, 6]) and the order of the T * 6 pairs by expert: group_start int32 [257],
    row_token int32 [T * 6], pair_row int32 [T, 6]."""
    f, (d, ref) = "flint_moe_select", _moe_dims(dims)
    E, K = d.n_experts, d.top_k
    try:  # as flint_linear_bf16
        T, e = logits.shape
        gpu, pairs = _current_gpu(), (T, K)
        good = (0 < T <= PAGED_MAX_TOKENS and e == E and logits.dtype is _F32 and
                topk_w.dtype is _F32 and topk_idx.dtype is _I32T and group_start.dtype is _I32T and
                row_token.dtype is _I32T and pair_row.dtype is _I32T and topk_idx.shape == pairs and
                topk_w.shape == pairs and pair_row.shape == pairs and row_token.shape == (T * K,) and
                group_start.shape == (E + 1,) and logits.is_contiguous() and
                topk_idx.is_contiguous() and topk_w.is_contiguous() and pair_row.is_contiguous() and
                row_token.is_contiguous() and group_start.is_contiguous() and
                logits.get_device() == topk_idx.get_device() == topk_w.get_device() ==
                group_start.get_device() == row_token.get_device() == pair_row.get_device() ==
                workspace.get_device() == gpu and
                workspace.dtype is _U8 and workspace.dim() == 1 and workspace.is_contiguous())
    except (AttributeError, ValueError, TypeError, RuntimeError):
        good = False
    if good:
        bias = logit_bias
        args = (logits.data_ptr(),
                None if bias is None else _arg(f, "logit_bias", bias, _F32, (E,), logits.device),
                topk_idx.data_ptr(), topk_w.data_ptr(), group_start.data_ptr(),
                row_token.data_ptr(), pair_row.data_ptr(), workspace.data_ptr(), workspace.numel())
    else:
        T, dev = _prompt_tokens(f, "logits", logits)
        args = (_arg(f, "logits", logits, _F32, (T, E), dev),
                _arg(f, "logit_bias", logit_bias, _F32, (E,), dev, optional=True),
                _arg(f, "topk_idx", topk_idx, _I32T, (T, K), dev),
                _arg(f, "topk_w", topk_w, _F32, (T, K), dev),
                _arg(f, "group_start", group_start, _I32T, (E + 1,), dev),
                _arg(f, "row_token", row_token, _I32T, (T * K,), dev),
                _arg(f, "pair_row", pair_row, _I32T, (T, K), dev), *_ws_arg(f, workspace, dev))
        gpu = dev.index
    _check((_lib or lib()).flint_moe_select(
        ref, T, *args, _raw_stream(gpu) if stream is None else _stream(stream)), f)


def flint_moe_combine_bf16(residual, y, pair_row, topk_w, y_shared, out, stream=None,
                           dims: Dims | None = None):
    """out[t] = residual[t] + y_shared[t] + sum_j topk_w[t, j] y[pair_row[t, j]]: bf16
    residual, out (may be residual itself) and y_shared (or None) [T, 2048], y
    [T * 6, 2048]."""
    f, (d, ref) = "flint_moe_combine_bf16", _moe_dims(dims)
    H, K = d.hidden, d.top_k
    try:  # as flint_linear_bf16
        T, h = residual.shape
        gpu, pairs, rows = _current_gpu(), (T, K), (T, H)
        good = (0 < T <= PAGED_MAX_TOKENS and h == H and residual.dtype is _BF16 and
                y.dtype is _BF16 and out.dtype is _BF16 and pair_row.dtype is _I32T and
                topk_w.dtype is _F32 and y.shape == (T * K, H) and out.shape == rows and
                pair_row.shape == pairs and topk_w.shape == pairs and residual.is_contiguous() and
                y.is_contiguous() and out.is_contiguous() and pair_row.is_contiguous() and
                topk_w.is_contiguous() and
                residual.get_device() == y.get_device() == out.get_device() ==
                pair_row.get_device() == topk_w.get_device() == gpu)
    except (AttributeError, ValueError, TypeError, RuntimeError):
        good = False
    if good:
        args = (residual.data_ptr(), y.data_ptr(), pair_row.data_ptr(), topk_w.data_ptr(),
                None if y_shared is None else
                _arg(f, "y_shared", y_shared, _BF16, rows, residual.device), out.data_ptr())
    else:
        T, dev = _prompt_tokens(f, "residual", residual)
        args = (_arg(f, "residual", residual, _BF16, (T, H), dev),
                _arg(f, "y", y, _BF16, (T * K, H), dev),
                _arg(f, "pair_row", pair_row, _I32T, (T, K), dev),
                _arg(f, "topk_w", topk_w, _F32, (T, K), dev),
                _arg(f, "y_shared", y_shared, _BF16, (T, H), dev, optional=True),
                _arg(f, "out", out, _BF16, (T, H), dev))
        gpu = dev.index
    _check((_lib or lib()).flint_moe_combine_bf16(
        ref, T, *args, _raw_stream(gpu) if stream is None else _stream(stream)), f)


def flint_moe_prompt_bf16(x, residual, w_router, logit_bias, w13, w2, ws13, ws2, out, workspace,
                          topk_idx_out=None, topk_w_out=None, stream=None,
                          dims: Dims | None = None):
    """flint_moe_decode_bf16 for prompts, 1 to 8192 tokens; workspace:
    new_prompt_workspace(tokens)."""
    f, (d, ref) = "flint_moe_prompt_bf16", _moe_dims(dims)
    T, dev = _prompt_tokens(f, "x", x)
    args = _layer_args(f, d, T, dev, x, residual, w_router, logit_bias, w13, w2, ws13, ws2, out,
                       topk_idx_out, topk_w_out)
    wp, wb = _ws_arg(f, workspace, dev)
    _check((_lib or lib()).flint_moe_prompt_bf16(ref, T, *args, wp, wb, _stream(stream)), f)


# ---------------------------------------------------------------- conveniences

def new_workspace(max_batch: int, device="cuda", wait_limit_ns: int = 0) -> torch.Tensor:
    """Allocates (through torch) and initialises a workspace for max_batch tokens."""
    n = flint_moe_workspace_bytes(max_batch)
    if n == 0:
        raise FlintError(FLINT_ERR_INVALID_ARG, "new_workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    flint_moe_workspace_init(ws, wait_limit_ns)
    return ws


def new_attn_workspace(device="cuda", dims: AttnDims | None = None) -> torch.Tensor:
    """Allocates (through torch) and initialises a workspace of the paged
    attention calls."""
    n = flint_attn_workspace_bytes(dims)
    if n == 0:
        raise FlintError(FLINT_ERR_UNSUPPORTED, "new_attn_workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    flint_attn_workspace_init(ws)
    return ws


def new_prompt_workspace(max_tokens: int = 0, device="cuda") -> torch.Tensor:
    """Allocates (through torch) and initialises a workspace of the linear calls, and of
    flint_moe_prompt_bf16 for up to max_tokens tokens."""
    n = flint_prompt_workspace_bytes(max_tokens)
    if n == 0:
        raise FlintError(FLINT_ERR_INVALID_ARG, "new_prompt_workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    flint_prompt_workspace_init(ws)
    return ws
