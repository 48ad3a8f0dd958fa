"""Python binding of libfp8blk, the MI355X (gfx950) FP8 quantize + block-scaled
FP8 GEMM library.

The functions mirror the C ABI in include/fp8blk.h by name.  They only marshal
arguments: torch tensors supply device memory and the current HIP stream, every
step of the computation runs in the library's HIP kernels.  When the library
is missing or no GPU is present, every call raises; there is no CPU fallback.

Enum values (same as the C header):
  formats        E4M3 = 0, E5M2 = 1
  granularities  GRAN_TENSOR = 0, GRAN_ROW = 1, GRAN_TILE_1x128 = 2,
                 GRAN_BLOCK_128x128 = 3, GRAN_MX32 = 4
  dtypes         DT_F32 = 0, DT_BF16 = 1
  GEMM kernels   GEMM_AUTO = 0, GEMM_TILED = 1, GEMM_SKINNY = 2
  accumulation   ACCUM_FP32 = 0 (exact products, fp32 sums), ACCUM_NATIVE = 1
  KV scales      KV_SCALE_TENSOR = 0, KV_SCALE_HEAD = 1, KV_SCALE_CHANNEL = 2
  FP4 scaling    FP4_MX = 0 (32-element UE8M0), FP4_NV = 1 (16-element E4M3 + fp32 tensor)
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

E4M3, E5M2 = 0, 1
GRAN_TENSOR, GRAN_ROW, GRAN_TILE_1x128, GRAN_BLOCK_128x128, GRAN_MX32 = 0, 1, 2, 3, 4
DT_F32, DT_BF16 = 0, 1
GEMM_AUTO, GEMM_TILED, GEMM_SKINNY = 0, 1, 2
ACCUM_FP32, ACCUM_NATIVE = 0, 1
KV_SCALE_TENSOR, KV_SCALE_HEAD, KV_SCALE_CHANNEL = 0, 1, 2
FP4_MX, FP4_NV = 0, 1

FP8_OK = 0
STATUS_NAMES = {0: "FP8_OK", 1: "FP8_ERR_NULL", 2: "FP8_ERR_ENUM", 3: "FP8_ERR_SHAPE",
                4: "FP8_ERR_UNSUPPORTED", 5: "FP8_ERR_WORKSPACE", 6: "FP8_ERR_HIP", 7: "FP8_ERR_ALIGN"}

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8blk.so")

# Exported symbols and their C signatures (include/fp8blk.h).
_c = ctypes
_SIGS = {
    "fp8_status_string": (_c.c_char_p, [_c.c_int]),
    "fp8_abi_version": (_c.c_int, []),
    "fp8_quantize_workspace_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int64, _c.c_int]),
    "fp8_quantize": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int,
                                _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "fp8_quantize_noalloc": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int,
                                        _c.c_void_p, _c.c_void_p, _c.c_void_p]),
    "fp8_quantize_delayed": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int, _c.c_void_p,
                                        _c.c_int64, _c.c_int64, _c.c_int, _c.c_void_p, _c.c_void_p,
                                        _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "fp8_dequantize": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int,
                                  _c.c_void_p, _c.c_int, _c.c_void_p]),
    "fp8_cast": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int, _c.c_void_p, _c.c_void_p]),
    "fp8_gemm_blockscaled": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p,
                                        _c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p,
                                        _c.c_int64, _c.c_int64, _c.c_int64,
                                        _c.c_void_p, _c.c_int, _c.c_void_p]),
    "fp8_gemm_blockscaled_ex": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p,
                                           _c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p,
                                           _c.c_int64, _c.c_int64, _c.c_int64,
                                           _c.c_void_p, _c.c_int, _c.c_int, _c.c_int, _c.c_void_p]),
    "fp8_gemm_blockscaled_quant": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p,
                                              _c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p,
                                              _c.c_int64, _c.c_int64, _c.c_int64,
                                              _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_void_p]),
    "fp8_kv_append": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64,
                                 _c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int64,
                                 _c.c_void_p]),
    "fp8_kv_gather": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int64,
                                 _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_void_p]),
    "fp8_kv_attention_workspace_bytes": (_c.c_size_t, [_c.c_int64] * 7 + [_c.c_int]),
    "fp8_kv_attention": (_c.c_int, [_c.c_void_p, _c.c_int] + [_c.c_int64] * 5 + [_c.c_void_p] * 2 + [_c.c_int64] +
                         [_c.c_void_p] + [_c.c_int64] * 3 + [_c.c_void_p] * 2 + [_c.c_int64] * 2 + [_c.c_int] * 2 +
                         [_c.c_void_p] * 2 + [_c.c_float, _c.c_void_p, _c.c_int] + [_c.c_void_p] * 3 +
                         [_c.c_int64, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "fp8_kv_evict_select_workspace_bytes": (_c.c_size_t, [_c.c_int64] * 2),
    "fp8_kv_evict_select": (_c.c_int, [_c.c_void_p] + [_c.c_int64] * 3 + [_c.c_void_p] + [_c.c_int64] * 4 +
                            [_c.c_void_p] * 3 + [_c.c_size_t, _c.c_void_p]),
    "fp8_kv_compact": (_c.c_int, [_c.c_void_p] * 2 + [_c.c_int64] * 3 + [_c.c_void_p, _c.c_int64] * 2 +
                       [_c.c_int64] * 2 + [_c.c_void_p] * 2 + [_c.c_int64] + [_c.c_void_p, _c.c_int64] * 2 +
                       [_c.c_void_p]),
    "fp8_prompt_attention_workspace_bytes": (_c.c_size_t, [_c.c_int64] * 6),
    "fp8_prompt_attention": (_c.c_int, [_c.c_void_p, _c.c_int64] * 3 + [_c.c_int64] * 5 +
                             [_c.c_void_p, _c.c_int64, _c.c_float] + [_c.c_void_p] * 3 + [_c.c_size_t, _c.c_void_p]),
    "fp4_quantize_workspace_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int64, _c.c_int]),
    "fp4_quantize": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int, _c.c_void_p,
                                _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "fp4_dequantize": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int,
                                  _c.c_void_p, _c.c_int, _c.c_void_p]),
    "fp4_gemm_blockscaled": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                        _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int, _c.c_void_p,
                                        _c.c_int, _c.c_void_p]),
}
EXPORTS = tuple(_SIGS)

# Measurement probes (include/fp8blk_probe.h): not part of the method; they
# measure the machine's matrix-core, read and copy ceilings.
PROBE_MFMA_BF16, PROBE_MFMA_FP8 = 0, 1
_PROBE_SIGS = {
    "fp8blk_probe_mfma_sink_floats": (_c.c_size_t, [_c.c_int]),
    "fp8blk_probe_mfma": (_c.c_int, [_c.c_int, _c.c_int, _c.c_int, _c.c_void_p, _c.POINTER(_c.c_double),
                                     _c.c_void_p]),
    "fp8blk_probe_read_sink_floats": (_c.c_size_t, []),
    "fp8blk_probe_read": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_void_p]),
    "fp8blk_probe_copy": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_void_p]),
}
PROBE_EXPORTS = tuple(_PROBE_SIGS)

_lib: Optional[ctypes.CDLL] = None


class Fp8Error(RuntimeError):
    """A libfp8blk call returned a non-OK status."""

    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)} ({msg})")
        self.status = status


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libfp8blk.so (built by build.py) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libfp8blk.so not found at {p}: build it with "
                           "`python -m block_scaled_precision_x128_amd.build` (there is no fallback)")
    lib = ctypes.CDLL(p)
    for name, (res, args) in list(_SIGS.items()) + list(_PROBE_SIGS.items()):
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(fn: str, st: int):
    if st != FP8_OK:
        raise Fp8Error(fn, st, load_library().fp8_status_string(st).decode())


def _torch():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("libfp8blk needs a ROCm GPU; torch.cuda.is_available() is False")
    return torch


def _stream(stream) -> int:
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dt_of(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return DT_F32
    if t.dtype == torch.bfloat16:
        return DT_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _torch_dtype(dt: int):
    torch = _torch()
    return torch.float32 if dt == DT_F32 else torch.bfloat16


def scale_shape(gran: int, rows: int, cols: int):
    return {GRAN_TENSOR: (1,), GRAN_ROW: (rows,), GRAN_TILE_1x128: (rows, cols // 128),
            GRAN_BLOCK_128x128: (rows // 128, cols // 128), GRAN_MX32: (rows, cols // 32)}[gran]


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


# ---- raw entry points (pointers and sizes, as in C) -------------------------

def fp8_status_string(status: int) -> str:
    return load_library().fp8_status_string(status).decode()


def fp8_abi_version() -> int:
    return load_library().fp8_abi_version()


def fp8_quantize_workspace_bytes(rows: int, cols: int, gran: int) -> int:
    return load_library().fp8_quantize_workspace_bytes(rows, cols, gran)


# ---- tensor-level wrappers ----------------------------------------------------

def fp8_quantize(x, fmt: int, gran: int, q=None, scales=None, workspace=None, stream=None):
    """Quantize a 2-D fp32/bf16 device tensor.  Returns (codes uint8, scales)."""
    torch = _torch()
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scales is None:
        sdt = torch.uint8 if gran == GRAN_MX32 else torch.float32
        scales = torch.empty(scale_shape(gran, rows, cols), dtype=sdt, device=x.device)
    lib = load_library()
    ws = lib.fp8_quantize_workspace_bytes(rows, cols, gran)
    if ws and workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=x.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.fp8_quantize(x.data_ptr(), _dt_of(x), rows, cols, fmt, gran, q.data_ptr(), scales.data_ptr(),
                          _ptr(workspace), wsb, _stream(stream))
    _check("fp8_quantize", st)
    return q, scales


def fp8_quantize_noalloc(x, fmt: int, gran: int, q, scales, stream=None):
    """fp8_quantize into caller-provided q and scales with no workspace: the
    per-tensor amax partials live in the library's static device scratch
    (calls that overlap on one GPU race).  Returns (q, scales)."""
    rows, cols = x.shape
    st = load_library().fp8_quantize_noalloc(x.data_ptr(), _dt_of(x), rows, cols, fmt, gran, q.data_ptr(),
                                             scales.data_ptr(), _stream(stream))
    _check("fp8_quantize_noalloc", st)
    return q, scales


def fp8_quantize_delayed(x, fmt: int, history, hist_pos: int, margin: int = 0, q=None, scale=None, workspace=None,
                         stream=None):
    """Delayed scaling: quantize x (2-D) with the scale from the amax history
    (device float32 [l]), then store x's amax at history[hist_pos].
    Returns (codes uint8, scale float32 [1])."""
    torch = _torch()
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    lib = load_library()
    ws = lib.fp8_quantize_workspace_bytes(rows, cols, GRAN_TENSOR)
    if ws and workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=x.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.fp8_quantize_delayed(x.data_ptr(), _dt_of(x), rows, cols, fmt, history.data_ptr(), history.numel(),
                                  hist_pos, margin, q.data_ptr(), scale.data_ptr(), _ptr(workspace), wsb,
                                  _stream(stream))
    _check("fp8_quantize_delayed", st)
    return q, scale


def fp8_dequantize(q, scales, fmt: int, gran: int, out_dtype: int = DT_F32, y=None, stream=None):
    """Dequantize codes to fp32 or bf16.  Returns y."""
    torch = _torch()
    rows, cols = q.shape
    if y is None:
        y = torch.empty((rows, cols), dtype=_torch_dtype(out_dtype), device=q.device)
    st = load_library().fp8_dequantize(q.data_ptr(), scales.data_ptr(), rows, cols, fmt, gran, y.data_ptr(),
                                       out_dtype, _stream(stream))
    _check("fp8_dequantize", st)
    return y


def fp8_cast(x, fmt: int, q=None, stream=None):
    """Unscaled saturating cast of a fp32/bf16 device tensor (numel % 8 == 0)."""
    torch = _torch()
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    st = load_library().fp8_cast(x.data_ptr(), _dt_of(x), x.numel(), fmt, q.data_ptr(), _stream(stream))
    _check("fp8_cast", st)
    return q


def fp8_gemm_blockscaled(a, a_fmt: int, a_gran: int, a_scales, b, b_fmt: int, b_gran: int, b_scales,
                         out_dtype: int = DT_BF16, out=None, algo: int = GEMM_AUTO, accum: int = ACCUM_FP32,
                         stream=None):
    """out[M, N] = (a * sA) @ (b * sB)^T for codes a [M, K], b [N, K]."""
    torch = _torch()
    M, K = a.shape
    N = b.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=_torch_dtype(out_dtype), device=a.device)
    lib = load_library()
    if algo == GEMM_AUTO and accum == ACCUM_FP32:
        # the plain entry point (AUTO kernel choice, exact products with fp32 sums)
        st = lib.fp8_gemm_blockscaled(
            a.data_ptr(), a_fmt, a_gran, a_scales.data_ptr(), b.data_ptr(), b_fmt, b_gran, b_scales.data_ptr(),
            M, N, K, out.data_ptr(), out_dtype, _stream(stream))
    else:
        st = lib.fp8_gemm_blockscaled_ex(
            a.data_ptr(), a_fmt, a_gran, a_scales.data_ptr(), b.data_ptr(), b_fmt, b_gran, b_scales.data_ptr(),
            M, N, K, out.data_ptr(), out_dtype, algo, accum, _stream(stream))
    _check("fp8_gemm_blockscaled", st)
    return out


def fp8_gemm_blockscaled_quant(a, a_fmt: int, a_gran: int, a_scales, b, b_fmt: int, b_gran: int, b_scales,
                               out_fmt: int = E4M3, codes=None, scales=None, accum: int = ACCUM_FP32, stream=None):
    """The GEMM with its result quantized in the epilogue to out_fmt codes and
    1x128 tile scales (the layout fp8_quantize writes for GRAN_TILE_1x128).
    Returns (codes uint8 [M, N], scales float32 [M, N/128])."""
    torch = _torch()
    M, K = a.shape
    N = b.shape[0]
    if codes is None:
        codes = torch.empty((M, N), dtype=torch.uint8, device=a.device)
    if scales is None:
        scales = torch.empty((M, N // 128), dtype=torch.float32, device=a.device)
    st = load_library().fp8_gemm_blockscaled_quant(
        a.data_ptr(), a_fmt, a_gran, a_scales.data_ptr(), b.data_ptr(), b_fmt, b_gran, b_scales.data_ptr(),
        M, N, K, out_fmt, codes.data_ptr(), scales.data_ptr(), accum, _stream(stream))
    _check("fp8_gemm_blockscaled_quant", st)
    return codes, scales


def fp8_kv_append(x, slots, cache, scales, fmt: int, scale_kind: int, stream=None):
    """Quantize on append: x [tokens, heads, head_dim] (fp32 or bf16; the
    leading dimension may be strided, e.g. a slice of a fused QKV output)
    written as codes into cache [num_slots, heads, head_dim] at rows slots
    (int64 [tokens]; slots outside the pool are skipped).  Returns cache."""
    tokens, heads, head_dim = x.shape
    if x.stride(2) != 1 or x.stride(1) != head_dim:
        raise ValueError("x must be contiguous within a token ([heads, head_dim] row-major)")
    if tuple(cache.shape[1:]) != (heads, head_dim) or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous [num_slots, heads, head_dim] uint8 tensor")
    st = load_library().fp8_kv_append(x.data_ptr(), _dt_of(x), tokens, heads, head_dim, x.stride(0),
                                      slots.data_ptr(), fmt, scale_kind, scales.data_ptr(), cache.data_ptr(),
                                      cache.shape[0], _stream(stream))
    _check("fp8_kv_append", st)
    return cache


def fp8_kv_gather(cache, slots, scales, fmt: int, scale_kind: int, out_dtype: int = DT_BF16, out=None,
                  stream=None):
    """Dequantize on read: rows slots (int64 [n]) of cache [num_slots, heads,
    head_dim] as fp32 or bf16 [n, heads, head_dim] (zeros for slots outside the
    pool).  Returns out."""
    torch = _torch()
    num_slots, heads, head_dim = cache.shape
    n = slots.shape[0]
    if out is None:
        out = torch.empty((n, heads, head_dim), dtype=_torch_dtype(out_dtype), device=cache.device)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    st = load_library().fp8_kv_gather(cache.data_ptr(), num_slots, heads, head_dim, slots.data_ptr(), n, fmt,
                                      scale_kind, scales.data_ptr(), out.data_ptr(), _dt_of(out), _stream(stream))
    _check("fp8_kv_gather", st)
    return out


def _placed(fn):
    """Run fn on its first argument's device (a launch goes to the current one)
    and on `stream` (a stream or its handle; None: that device's current one),
    which is made current, so that what the call allocates belongs to the
    stream it runs on."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw[name]
        if not first.is_cuda:
            _torch()
            raise ValueError(f"the tensors must be on a GPU, not on {first.device}")
        import torch
        if stream is None and first.get_device() == torch.cuda.current_device():
            return fn(*args, **kw)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=first.device)
        with torch.cuda.device(first.device), torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _need(t, name: str, index: int, dtype, shape=None):
    """The address of a tensor argument, checked: contiguous, of this dtype and shape, on GPU `index`."""
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, not {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")


def _need_states(t, name: str, index: int, dtypes, shape):
    """Check t [tokens, heads, head_dim], contiguous within a token; its dtype code and row stride."""
    if t.dtype not in dtypes:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    tokens, heads, head_dim = shape
    ld, head, one = t.stride()
    if tokens > 0 and ((head_dim > 1 and one != 1) or (heads > 1 and head != head_dim)):
        raise ValueError(f"{name} must be contiguous within a token ([heads, head_dim] row-major)")
    return dtypes.index(t.dtype), ld if tokens > 1 else heads * head_dim


def _need_weights(t, name: str, index: int, batch: int, kv_heads: int):
    """Check an attention-weight tensor; its address and row length."""
    import torch
    at = _need(t, name, index, torch.float32)
    if t.dim() != 3 or t.shape[0] != batch or t.shape[1] != kv_heads:
        raise ValueError(f"{name} must be [{batch}, {kv_heads}, positions], not {tuple(t.shape)}")
    return at, t.shape[2]


def _need_scales(t, name: str, index: int, kind: int, heads: int, head_dim: int):
    import torch
    at = _need(t, name, index, torch.float32)
    n = heads if kind == KV_SCALE_HEAD else heads * head_dim if kind == KV_SCALE_CHANNEL else 1
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} scales, not {n}")
    return at


def _need_workspace(ws, nbytes: int, index: int):
    """The given workspace, checked, or a new one: the tensor (kept alive by the caller), its address and size."""
    import torch
    if ws is None:
        if not nbytes:
            return None, None, 0
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    elif ws.get_device() != index or not ws.is_contiguous():
        raise ValueError("workspace must be contiguous and on the inputs' device")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def fp8_kv_attention_workspace_bytes(q_tokens: int, heads: int, kv_heads: int, head_dim: int, batch: int, max_q: int,
                                     max_kv: int, with_weights: bool = False) -> int:
    return int(load_library().fp8_kv_attention_workspace_bytes(q_tokens, heads, kv_heads, head_dim, batch, max_q,
                                                               max_kv, int(with_weights)))


@_placed
def fp8_kv_attention(q, k_cache, v_cache, block_table, block_size: int, q_starts, kv_lens, k_scales, v_scales,
                     fmt: int, scale_kind: int, max_q: int, max_kv: int, softmax_scale: Optional[float] = None,
                     out_dtype: int = DT_BF16, out=None, lse=None, weights_in=None, weights_out=None, workspace=None):
    """Attention of the newest tokens of every sequence over the paged FP8
    cache: one token each (a decode step), a few, or a chunk of a prompt.

    q [tokens, heads, head_dim] (fp32 or bf16; rows may be strided) holds
    sequence b's tokens at q_starts[b] .. q_starts[b+1]-1 (int64 [batch + 1]),
    k_cache and v_cache [num_slots, kv_heads, head_dim] the codes, these
    tokens' own among them; position j of sequence b is slot
    block_table[b, j // block_size] * block_size + j % block_size (int64
    [batch, max_blocks]; entries outside the pool are left out).  kv_lens
    int64 [batch].  max_q and max_kv bound the lengths.  softmax_scale defaults
    to head_dim ** -0.5.

    weights_out (fp32 [batch, kv_heads, >= max_kv]) receives weights_in (None:
    zeros; may be weights_out) plus the attention weight of this call that each
    position got from its kv head's query heads.  `stream` (keyword): a stream
    or its handle instead of the current one.

    Returns (out [tokens, heads, head_dim], lse fp32 [tokens, heads])."""
    import torch
    if q.dim() != 3 or k_cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q and the caches are [.., heads, head_dim], block_table [batch, max_blocks]")
    dev, i64, pool = q.get_device(), torch.int64, k_cache.shape
    tokens, heads, head_dim = q.shape
    num_slots, kv_heads, _ = pool
    batch, max_blocks = block_table.shape
    if pool[2] != head_dim:
        raise ValueError(f"the cache has heads of {pool[2]}, q of {head_dim}")
    q_dt, ld_q = _need_states(q, "q", dev, (torch.float32, torch.bfloat16), q.shape)
    kp = _need(k_cache, "k_cache", dev, torch.uint8)
    vp = _need(v_cache, "v_cache", dev, torch.uint8, pool)
    table = _need(block_table, "block_table", dev, i64)
    starts = _need(q_starts, "q_starts", dev, i64, (batch + 1,))
    lens = _need(kv_lens, "kv_lens", dev, i64, (batch,))
    ks = _need_scales(k_scales, "k_scales", dev, scale_kind, kv_heads, head_dim)
    vs = _need_scales(v_scales, "v_scales", dev, scale_kind, kv_heads, head_dim)
    wi = wo = None
    ld_w = 0
    if weights_out is not None:
        wo, ld_w = _need_weights(weights_out, "weights_out", dev, batch, kv_heads)
    if weights_in is not None:
        wi, ld_in = _need_weights(weights_in, "weights_in", dev, batch, kv_heads)
        if wo is None or ld_in != ld_w:
            raise ValueError("weights_in goes with a weights_out of its shape")
    if out is None:
        out = torch.empty(tokens, heads, head_dim, dtype=torch.float32 if out_dtype == DT_F32 else torch.bfloat16,
                          device="cuda")
    else:
        out_dtype = _need_states(out, "out", dev, (torch.float32, torch.bfloat16), q.shape)[0]
        _need(out, "out", dev, out.dtype)
    if lse is None:
        lse = torch.empty(tokens, heads, dtype=torch.float32, device="cuda")
    lib = load_library()
    ws, wsp, wsb = _need_workspace(workspace, lib.fp8_kv_attention_workspace_bytes(
        tokens, heads, kv_heads, head_dim, batch, max_q, max_kv, wo is not None), dev)
    st = lib.fp8_kv_attention(
        q.data_ptr(), q_dt, tokens, heads, kv_heads, head_dim, ld_q, kp, vp, num_slots, table, max_blocks, block_size,
        batch, starts, lens, max_q, max_kv, fmt, scale_kind, ks, vs,
        head_dim ** -0.5 if softmax_scale is None else softmax_scale, out.data_ptr(), out_dtype,
        _need(lse, "lse", dev, torch.float32, (tokens, heads)), wi, wo, ld_w, wsp, wsb,
        torch.cuda.current_stream(dev).cuda_stream)
    if st:
        _check("fp8_kv_attention", st)
    return out, lse


def fp8_kv_evict_select_workspace_bytes(batch: int, max_kv: int) -> int:
    return int(load_library().fp8_kv_evict_select_workspace_bytes(batch, max_kv))


@_placed
def fp8_kv_evict_select(weights, kv_lens, keep: int, first: int = 0, recent: int = 0, max_kv: Optional[int] = None,
                        kept=None, kept_lens=None, workspace=None):
    """Choose the positions of every sequence to keep: the first `first` and the
    last `recent`, and of the others those with the largest weight summed over
    the kv heads (weights fp32 [batch, kv_heads, positions], as
    fp8_kv_attention collects them), ties to the lowest position.  kv_lens
    int64 [batch]; max_kv (default: the row length) bounds it.  `stream`
    (keyword) as for fp8_kv_attention.  Returns (kept int64 [batch, keep],
    ascending and -1 behind the last; kept_lens int64 [batch])."""
    import torch
    dev, i64 = weights.get_device(), torch.int64
    if weights.dim() != 3:
        raise ValueError("weights must be [batch, kv_heads, positions]")
    batch, kv_heads, ld_w = weights.shape
    wp = _need(weights, "weights", dev, torch.float32)
    lens = _need(kv_lens, "kv_lens", dev, i64, (batch,))
    if max_kv is None:
        max_kv = ld_w
    if kept is None:
        kept = torch.empty(batch, max(keep, 0), dtype=i64, device="cuda")
    if kept_lens is None:
        kept_lens = torch.empty(batch, dtype=i64, device="cuda")
    lib = load_library()
    ws, wsp, wsb = _need_workspace(workspace, lib.fp8_kv_evict_select_workspace_bytes(batch, max_kv), dev)
    st = lib.fp8_kv_evict_select(wp, ld_w, batch, kv_heads, lens, max_kv, keep, first, recent,
                                 _need(kept, "kept", dev, i64, (batch, max(keep, 0))),
                                 _need(kept_lens, "kept_lens", dev, i64, (batch,)), wsp, wsb,
                                 torch.cuda.current_stream(dev).cuda_stream)
    if st:
        _check("fp8_kv_evict_select", st)
    return kept, kept_lens


@_placed
def fp8_kv_compact(k_cache, v_cache, src_table, dst_table, block_size: int, kept, kept_lens, weights_in=None,
                   weights_out=None):
    """Move the rows of the kept positions together in both caches (uint8
    [num_slots, kv_heads, head_dim]) and, if given, in the weights: position i
    under dst_table becomes position kept[b, i] under src_table (int64 tables
    [batch, blocks]).  dst_table may be src_table: compaction in place.  A table
    of its own names pages that are no source of the call, or the page that
    src_table has in the same place.
    `stream` (keyword) as for fp8_kv_attention.  Returns (k_cache, v_cache)."""
    import torch
    dev, i64, pool = k_cache.get_device(), torch.int64, k_cache.shape
    if k_cache.dim() != 3 or src_table.dim() != 2 or dst_table.dim() != 2 or kept.dim() != 2:
        raise ValueError("caches are [num_slots, kv_heads, head_dim], tables [batch, blocks], kept [batch, keep]")
    num_slots, kv_heads, head_dim = pool
    batch, keep = kept.shape
    src_blocks, dst_blocks = src_table.shape[1], dst_table.shape[1]
    wi = wo = None
    ld_in = ld_out = 0
    if (weights_in is None) != (weights_out is None):
        raise ValueError("weights_in and weights_out go together")
    if weights_in is not None:
        wi, ld_in = _need_weights(weights_in, "weights_in", dev, batch, kv_heads)
        wo, ld_out = _need_weights(weights_out, "weights_out", dev, batch, kv_heads)
    st = load_library().fp8_kv_compact(
        _need(k_cache, "k_cache", dev, torch.uint8), _need(v_cache, "v_cache", dev, torch.uint8, pool), num_slots,
        kv_heads, head_dim, _need(src_table, "src_table", dev, i64, (batch, src_blocks)), src_blocks,
        _need(dst_table, "dst_table", dev, i64, (batch, dst_blocks)), dst_blocks, block_size, batch,
        _need(kept, "kept", dev, i64), _need(kept_lens, "kept_lens", dev, i64, (batch,)), keep, wi, ld_in, wo, ld_out,
        torch.cuda.current_stream(dev).cuda_stream)
    if st:
        _check("fp8_kv_compact", st)
    return k_cache, v_cache


def fp8_prompt_attention_workspace_bytes(tokens: int, heads: int, kv_heads: int, head_dim: int, batch: int,
                                         max_len: int) -> int:
    return int(load_library().fp8_prompt_attention_workspace_bytes(tokens, heads, kv_heads, head_dim, batch, max_len))


@_placed
def fp8_prompt_attention(q, k, v, seq_starts, max_len: int, softmax_scale: Optional[float] = None, out=None, lse=None,
                         workspace=None):
    """Causal attention of whole prompts, packed one behind the other, over
    their bf16 states: q [tokens, heads, head_dim], k and v [tokens, kv_heads,
    head_dim] (rows may be strided, as in a fused QKV output); sequence b is the
    tokens seq_starts[b] .. seq_starts[b+1]-1 (int64 [batch + 1]), of at most
    max_len.  softmax_scale defaults to head_dim ** -0.5.  `stream` (keyword) as
    for fp8_kv_attention.  Returns (out bf16 [tokens, heads, head_dim], lse fp32
    [tokens, heads])."""
    import torch
    dev = q.get_device()
    if q.dim() != 3 or k.dim() != 3 or seq_starts.dim() != 1 or seq_starts.numel() < 1:
        raise ValueError("q, k and v are [tokens, heads, head_dim], seq_starts [batch + 1]")
    tokens, heads, head_dim = q.shape
    kv_heads = k.shape[1]
    kv = (tokens, kv_heads, head_dim)
    _, ld_q = _need_states(q, "q", dev, (torch.bfloat16,), q.shape)
    _, ld_k = _need_states(k, "k", dev, (torch.bfloat16,), kv)
    _, ld_v = _need_states(v, "v", dev, (torch.bfloat16,), kv)
    starts = _need(seq_starts, "seq_starts", dev, torch.int64)
    if out is None:
        out = torch.empty(tokens, heads, head_dim, dtype=torch.bfloat16, device="cuda")
    if lse is None:
        lse = torch.empty(tokens, heads, dtype=torch.float32, device="cuda")
    lib, batch = load_library(), seq_starts.shape[0] - 1
    ws, wsp, wsb = _need_workspace(workspace, lib.fp8_prompt_attention_workspace_bytes(
        tokens, heads, kv_heads, head_dim, batch, max_len), dev)
    st = lib.fp8_prompt_attention(
        q.data_ptr(), ld_q, k.data_ptr(), ld_k, v.data_ptr(), ld_v, tokens, heads, kv_heads, head_dim, batch, starts,
        max_len, head_dim ** -0.5 if softmax_scale is None else softmax_scale,
        _need(out, "out", dev, torch.bfloat16, q.shape), _need(lse, "lse", dev, torch.float32, (tokens, heads)), wsp, wsb,
        torch.cuda.current_stream(dev).cuda_stream)
    if st:
        _check("fp8_prompt_attention", st)
    return out, lse


def fp4_block(kind: int) -> int:
    return 32 if kind == FP4_MX else 16


def fp4_quantize_workspace_bytes(rows: int, cols: int, kind: int) -> int:
    return int(load_library().fp4_quantize_workspace_bytes(rows, cols, kind))


def fp4_quantize(x, kind: int, q=None, block_scales=None, tensor_scale=None, workspace=None, stream=None):
    """Quantize x [rows, cols] to packed E2M1 codes.  Returns (q [rows, cols/2]
    uint8, block_scales uint8 [rows, cols/32 or cols/16], tensor_scale float32
    [1] or None for MX)."""
    torch = _torch()
    rows, cols = x.shape
    dev = x.device
    if q is None:
        q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    if block_scales is None:
        block_scales = torch.empty((rows, cols // fp4_block(kind)), dtype=torch.uint8, device=dev)
    if kind == FP4_NV and tensor_scale is None:
        tensor_scale = torch.empty(1, dtype=torch.float32, device=dev)
    wsb = fp4_quantize_workspace_bytes(rows, cols, kind)
    if workspace is None and wsb:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    st = load_library().fp4_quantize(x.data_ptr(), _dt_of(x), rows, cols, kind, q.data_ptr(),
                                     block_scales.data_ptr(), _ptr(tensor_scale), _ptr(workspace),
                                     workspace.numel() if workspace is not None else 0, _stream(stream))
    _check("fp4_quantize", st)
    return q, block_scales, tensor_scale


def fp4_dequantize(q, block_scales, tensor_scale, kind: int, out_dtype: int = DT_F32, y=None, stream=None):
    """Dequantize packed E2M1 codes [rows, cols/2] to fp32 or bf16 [rows, cols]."""
    torch = _torch()
    rows, half = q.shape
    if y is None:
        y = torch.empty((rows, 2 * half), dtype=_torch_dtype(out_dtype), device=q.device)
    st = load_library().fp4_dequantize(q.data_ptr(), block_scales.data_ptr(), _ptr(tensor_scale), rows, 2 * half,
                                       kind, y.data_ptr(), _dt_of(y), _stream(stream))
    _check("fp4_dequantize", st)
    return y


def fp4_gemm_blockscaled(a, a_scales, a_tensor_scale, b, b_scales, b_tensor_scale, kind: int,
                         out_dtype: int = DT_F32, out=None, stream=None):
    """FP4 block-scaled GEMM of packed E2M1 operands a [M, K/2], b [N, K/2]
    (K-contiguous) with their block (and, NV, tensor) scales.  MXFP4 runs on
    the FP4 matrix cores, NVFP4 on exact fp16 expansions; M <= 64 takes the
    skinny (decode) kernel.  Returns out [M, N]."""
    torch = _torch()
    M, half = a.shape
    N = b.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=_torch_dtype(out_dtype), device=a.device)
    st = load_library().fp4_gemm_blockscaled(a.data_ptr(), a_scales.data_ptr(), _ptr(a_tensor_scale), b.data_ptr(),
                                             b_scales.data_ptr(), _ptr(b_tensor_scale), M, N, 2 * half, kind,
                                             out.data_ptr(), _dt_of(out), _stream(stream))
    _check("fp4_gemm_blockscaled", st)
    return out


# ---- measurement probes (include/fp8blk_probe.h) -------------------------------

def probe_mfma(kind: int, waves_per_simd: int, iters: int, sink=None, stream=None) -> float:
    """Enqueue the back-to-back MFMA probe; returns the launch's FLOP count."""
    torch = _torch()
    lib = load_library()
    if sink is None:
        sink = torch.empty(int(lib.fp8blk_probe_mfma_sink_floats(waves_per_simd)), dtype=torch.float32,
                           device="cuda")
    flops = ctypes.c_double(0.0)
    st = lib.fp8blk_probe_mfma(kind, waves_per_simd, iters, sink.data_ptr(), ctypes.byref(flops), _stream(stream))
    _check("fp8blk_probe_mfma", st)
    return flops.value


def probe_read(src, sink=None, stream=None):
    """Enqueue a streaming read of every byte of the device tensor src."""
    torch = _torch()
    lib = load_library()
    if sink is None:
        sink = torch.empty(int(lib.fp8blk_probe_read_sink_floats()), dtype=torch.float32, device=src.device)
    st = lib.fp8blk_probe_read(src.data_ptr(), src.numel() * src.element_size(), sink.data_ptr(), _stream(stream))
    _check("fp8blk_probe_read", st)
    return sink


def probe_copy(src, dst, stream=None):
    """Enqueue a device copy of src into dst (same byte size, no overlap)."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst must have the same byte size")
    st = load_library().fp8blk_probe_copy(src.data_ptr(), dst.data_ptr(), nbytes, _stream(stream))
    _check("fp8blk_probe_copy", st)
    return dst
