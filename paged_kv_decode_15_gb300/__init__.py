"""Attention over a paged KV cache on GB300 (sm_103a): Python binding of libpkd.

Argument marshalling only.  Every step runs in the library's CUDA kernels;
torch supplies device memory and the current stream.  There is no CPU path:
if libpkd.so is missing or a GPU is absent, the calls raise.

Entry points (same names as the C ABI in include/pkd.h, without the prefix):
  paged_decode(q, kv_cache, block_table, seq_lens, scale, window, out, lse, ...)
  segmented_attention(q, k, v, used, bias, bs, local, out, ...)
  lse_merge(part_out, part_lse, prior=None, live=None, out=None, lse_out=None)
  workspace_size(...), workspace_init(ws), workspace_check(ws=None), release_workspaces()
  rope_cache_write(q, key, value, positions, cos_sin, slot_mapping, kv_cache, ...)
  paged_attention(q, kv_cache, block_table, seq_lens, query_start, scale, ...)
  prefix_decode(q, kv_cache, prefix_table, prefix_lens, block_table, seq_lens, scale, ...)
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkd.so")

OK, EINVAL, EUNSUPPORTED, ECUDA, EDEVICE_BOUNDS, ETIMEOUT = range(6)
BF16, FP16, FP8_E4M3, FP32 = 0, 1, 2, 3
FLAG_CAUSAL, FLAG_MMA_SMALL_M, FLAG_FMA, FLAG_GRID, FLAG_FLAT, FLAG_BALANCED = 1, 2, 4, 8, 16, 32
FLAG_TEST_TIMEOUT = 64
FLAG_HOST_IO = 128

SYMBOLS = ("pkd_version", "pkd_last_error", "pkd_paged_decode_workspace_size", "pkd_paged_decode_kernel_name",
           "pkd_workspace_init",
           "pkd_workspace_check", "pkd_paged_decode", "pkd_paged_decode_static", "pkd_paged_decode_static_check",
           "pkd_cache_write",
           "pkd_segmented_attention", "pkd_segmented_attention_paged", "pkd_lse_merge",
           "pkd_rope_cache_write", "pkd_paged_attention_workspace_size", "pkd_paged_attention_kernel_name",
           "pkd_paged_attention", "pkd_prefix_decode_workspace_size", "pkd_prefix_decode")


class ScoreOptions(ctypes.Structure):
    """pkd_score_options of the C ABI."""
    _fields_ = [("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p), ("window", ctypes.c_int),
                ("prefix_lens", ctypes.c_void_p), ("doc_start", ctypes.c_void_p)]


class PkdError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pkd status {status}: {message}")
        self.status = status


_lib = None


def build(force: bool = False) -> str:
    """Compile libpkd.so in-tree for sm_103a."""
    from . import _build
    return _build.build(force=force)


def load_library(path: str = LIB_PATH):
    """Load libpkd.so and declare its C signatures (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with paged_kv_decode_15_gb300.build() "
                          "(nvcc for sm_103a); there is no fallback implementation")
    lib = ctypes.CDLL(path)
    P, I, I64, F, U, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_uint,
                           ctypes.c_size_t)
    lib.pkd_version.restype = I
    lib.pkd_last_error.restype = ctypes.c_char_p
    lib.pkd_paged_decode_workspace_size.argtypes = [I, I, I, I, I, I, I, I, I, I, U]
    lib.pkd_paged_decode_workspace_size.restype = SZ
    lib.pkd_paged_decode_kernel_name.argtypes = [I, I, I, I, I, I, I, I, I, I, U]
    lib.pkd_paged_decode_kernel_name.restype = ctypes.c_char_p
    lib.pkd_workspace_init.argtypes = [P, SZ, P]
    lib.pkd_workspace_check.argtypes = [P, SZ, P]
    lib.pkd_paged_decode.argtypes = [P, I, P, I, I64, P, I64, P, I, I, I, I, I, I, I, F, F, F, F, I,
                                     P, I, P, P, SZ, I, U, P]
    lib.pkd_paged_decode_static.argtypes = [P, I, P, I, I64, P, I64, P, I, I, I, I, I, I, I, F, F, F, F, I,
                                            P, I, P, I, U, P]
    lib.pkd_paged_decode_static_check.argtypes = [P]
    lib.pkd_cache_write.argtypes = [P, P, I, I64, I64, P, I64, I, I, I, I64, P, I, F, F, P]
    lib.pkd_segmented_attention.argtypes = [P, P, P, I, P, P, I, I, I, I, I, I, I, P, P, P, P]
    lib.pkd_segmented_attention_paged.argtypes = [P, I, P, I64, P, I64, P, P, P, I, I, I, I, I, I, I, I, I,
                                                  P, P, P, P]
    lib.pkd_lse_merge.argtypes = [P, P, P, P, I, I, I, I, P, I, P, P]
    O = ctypes.POINTER(ScoreOptions)
    lib.pkd_rope_cache_write.argtypes = [P, I64, P, I64, P, I64, I, P, P, I64, I, I, P, I64, I, I, I, I, I64, P, I, F,
                                         F, P, I64, I, F, P]
    lib.pkd_paged_attention_workspace_size.argtypes = [I, I64, I, I, I, I, I, I, I, O]
    lib.pkd_paged_attention_workspace_size.restype = SZ
    lib.pkd_paged_attention_kernel_name.argtypes = [I, I64, I, I, I, I, I, I, I, O]
    lib.pkd_paged_attention_kernel_name.restype = ctypes.c_char_p
    lib.pkd_paged_attention.argtypes = [P, I, I64, P, I, I64, P, I64, P, P, I, I64, I, I, I, I, I, I, F, F, F, F, O, P,
                                        I, P, P, SZ, U, P]
    lib.pkd_prefix_decode_workspace_size.argtypes = [I, I, I, I, I, I, I, I, I, I]
    lib.pkd_prefix_decode_workspace_size.restype = SZ
    lib.pkd_prefix_decode.argtypes = [P, I, P, I, I64, P, I64, P, P, I, I, P, I64, P, I, I, I, I, I, I, I, F, F, F, F,
                                      F, P, I, P, P, SZ, U, P]
    for name in ("pkd_rope_cache_write", "pkd_paged_attention", "pkd_prefix_decode", "pkd_workspace_init", "pkd_workspace_check", "pkd_paged_decode", "pkd_paged_decode_static",
                 "pkd_paged_decode_static_check", "pkd_cache_write", "pkd_segmented_attention", "pkd_segmented_attention_paged", "pkd_lse_merge"):
        getattr(lib, name).restype = I
    _lib = lib
    return lib


def _check(status: int):
    if status != OK:
        raise PkdError(status, load_library().pkd_last_error().decode())


def dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return BF16
    if t == torch.float16:
        return FP16
    if t in (torch.uint8, getattr(torch, "float8_e4m3fn", None)):
        return FP8_E4M3
    if t == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _cuda(t, name):
    if t is not None and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t


def version() -> int:
    return load_library().pkd_version()


def workspace_size(batch, sq, num_heads, num_kv_heads, head_dim, page_size, max_kv_len, kv_dtype, window=0,
                   chunk_tokens=0, flags=0) -> int:
    n = load_library().pkd_paged_decode_workspace_size(batch, sq, num_heads, num_kv_heads, head_dim, page_size,
                                                       max_kv_len, int(kv_dtype), int(window), int(chunk_tokens),
                                                       int(flags))
    if n == 0:
        raise PkdError(EINVAL, load_library().pkd_last_error().decode())
    return n


def kernel_name(batch, sq, num_heads, num_kv_heads, head_dim, page_size, max_kv_len, kv_dtype, window=0,
                chunk_tokens=0, flags=0) -> str:
    """The kernel paged_decode launches for these shapes and flags."""
    name = load_library().pkd_paged_decode_kernel_name(batch, sq, num_heads, num_kv_heads, head_dim, page_size,
                                                       max_kv_len, int(kv_dtype), int(window), int(chunk_tokens),
                                                       int(flags))
    if name is None:
        raise PkdError(EINVAL, load_library().pkd_last_error().decode())
    return name.decode()


def workspace_init(ws: torch.Tensor, stream=None):
    _check(load_library().pkd_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def workspace_check(ws: torch.Tensor = None, stream=None) -> int:
    """Synchronise, read and clear the workspace status word; returns the status code.

    Without ws: that of the workspace which paged_attention and prefix_decode
    keep for this host thread and stream (default: the current one) when they
    are given none.  Such a workspace is ready for the next call afterwards,
    also after ETIMEOUT (its counters are zeroed again).  A call captured into
    a graph has its workspace in the graph: pass it one of your own to read
    its status.
    """
    if ws is not None:
        return load_library().pkd_workspace_check(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    s = stream if stream is not None else torch.cuda.current_stream()
    index = s.device.index
    kept = _kept.workspaces.get((index, s.cuda_stream))
    if kept is None:
        return OK
    with torch.cuda.device(index):
        status = load_library().pkd_workspace_check(kept[0], kept[1], s.cuda_stream)
        if status == ETIMEOUT:
            _check(load_library().pkd_workspace_init(kept[0], _WS_HEAD, s.cuda_stream))
    return status


def release_workspaces():
    """Free the workspaces that paged_attention and prefix_decode keep for this host
    thread (the next call makes a new one); those of other threads go with their
    threads.  Calls already queued keep theirs until they are done."""
    _kept.workspaces.clear()


_ws_cache: dict = {}


def _workspace(nbytes: int, device) -> torch.Tensor:
    key = (str(device), nbytes)
    ws = _ws_cache.get(key)
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        workspace_init(ws)
        _ws_cache[key] = ws
    return ws


def paged_decode(q, kv_cache, block_table, seq_lens, scale, window=0, out=None, lse=None, *, q_scale=1.0,
                 k_scale=1.0, v_scale=1.0, max_kv_len=None, workspace=None, chunk_tokens=0, causal=False,
                 mma_small_m=False, force_fma=False, grid=False, flat=False, balanced=False, out_dtype=None,
                 test_timeout=False, host_io=False, stream=None):
    """Attention of each request's query block over its paged keys.

    q [B, sq, Hq, D]; kv_cache [num_pages, Hkv, P, 2*D] (bf16, fp16, or uint8 /
    float8_e4m3fn for fp8, with q of the same type); block_table int32 [B, W];
    seq_lens int32 [B].  Returns (out [B, sq, Hq, D], lse fp32 [B, sq, Hq]).
    max_kv_len defaults to the table's capacity W * P (no host sync).
    test_timeout sets the diagnostic PKD_FLAG_TEST_TIMEOUT.  host_io sets
    PKD_FLAG_HOST_IO: q, block_table, seq_lens (and out, lse, allocated pinned
    when not given) are pinned host tensors that the kernels read and write in
    place; kv_cache and the workspace stay on the device.
    """
    lib = load_library()
    _cuda(kv_cache, "kv_cache")
    io = ((q, "q"), (block_table, "block_table"), (seq_lens, "seq_lens"), (out, "out"), (lse, "lse"))
    for t, n in io:
        if host_io:
            if t is not None and (t.is_cuda or not t.is_pinned()):
                raise ValueError(f"{n} must be a pinned host tensor with host_io")
        else:
            _cuda(t, n)
    B, sq, Hq, D = q.shape
    num_pages, Hkv, P, twoD = kv_cache.shape
    if twoD != 2 * D:
        raise ValueError(f"kv_cache last dim {twoD} != 2 * head_dim {2 * D}")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    if not (q.is_contiguous() and kv_cache.is_contiguous() and seq_lens.is_contiguous()):
        raise ValueError("q, kv_cache and seq_lens must be contiguous")
    if block_table.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")
    kv_dt = dtype_code(kv_cache.dtype)
    q_dt = dtype_code(q.dtype)
    place = dict(pin_memory=True) if host_io else dict(device=q.device)
    if out is None:
        odt = out_dtype or (torch.bfloat16 if kv_dt == FP8_E4M3 else q.dtype)
        out = torch.empty((B, sq, Hq, D), dtype=odt, **place)
    if lse is None:
        lse = torch.empty((B, sq, Hq), dtype=torch.float32, **place)
    if max_kv_len is None:
        max_kv_len = block_table.shape[1] * P
    flags = (FLAG_CAUSAL if causal else 0) | (FLAG_MMA_SMALL_M if mma_small_m else 0) | \
        (FLAG_FMA if force_fma else 0) | (FLAG_GRID if grid else 0) | (FLAG_FLAT if flat else 0) | \
        (FLAG_BALANCED if balanced else 0) | (FLAG_TEST_TIMEOUT if test_timeout else 0) | \
        (FLAG_HOST_IO if host_io else 0)
    need = workspace_size(B, sq, Hq, Hkv, D, P, max_kv_len, kv_dt, window, chunk_tokens, flags)
    if workspace is None:
        workspace = _workspace(need, kv_cache.device)
    _check(lib.pkd_paged_decode(
        _ptr(q), q_dt, _ptr(kv_cache), kv_dt, num_pages, _ptr(block_table), block_table.stride(0), _ptr(seq_lens),
        B, sq, Hq, Hkv, D, P, int(max_kv_len), float(scale), float(q_scale), float(k_scale), float(v_scale),
        int(window), _ptr(out), dtype_code(out.dtype), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), int(chunk_tokens), flags, _stream(stream)))
    return out, lse


def segmented_attention(q, k, v, used, bias, bs, local, out=None, *, seg_out=None, seg_lse=None,
                        return_segments=False, stream=None):
    """DASH segmented attention + combine.

    q [n, Hq, D]; k, v [n*(topk*bs+local), Hkv, D]; used int32 [n*(topk+1)];
    bias fp32 [n, topk].  Returns out [n, Hq, D] (and the per-segment fp32
    (seg_out [n, topk+1, Hq, D], seg_lse [n, topk+1, Hq]) when asked).
    """
    lib = load_library()
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    topk = bias.shape[1] if bias is not None else 0
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (used, "used"), (bias, "bias")):
        _cuda(t, name)
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if used.dtype != torch.int32 or (bias is not None and bias.dtype != torch.float32):
        raise TypeError("used must be int32 and bias float32")
    if out is None:
        out = torch.empty_like(q)
    if return_segments and seg_out is None:
        seg_out = torch.empty((n, topk + 1, Hq, D), dtype=torch.float32, device=q.device)
        seg_lse = torch.empty((n, topk + 1, Hq), dtype=torch.float32, device=q.device)
    _check(lib.pkd_segmented_attention(
        _ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(used), _ptr(bias), n, Hq, Hkv, D, topk, int(bs),
        int(local), _ptr(out), _ptr(seg_out), _ptr(seg_lse), _stream(stream)))
    return (out, seg_out, seg_lse) if return_segments else out


def segmented_attention_paged(q, kv_cache, block_table, seg_start, used, bias, bs, local, out=None, *,
                              max_kv_len=None, return_segments=False, stream=None):
    """DASH segmented attention over key ranges of each query's request in a paged cache.

    q [n, Hq, D]; kv_cache [num_pages, Hkv, P, 2D]; block_table int32 [n, W];
    seg_start, used int32 [n, topk+1]; bias fp32 [n, topk].
    """
    lib = load_library()
    n, Hq, D = q.shape
    num_pages, Hkv, P, _ = kv_cache.shape
    topk = bias.shape[1] if bias is not None else 0
    for t, name in ((q, "q"), (kv_cache, "kv_cache"), (block_table, "block_table"), (seg_start, "seg_start"),
                    (used, "used"), (bias, "bias")):
        _cuda(t, name)
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out is None:
        out = torch.empty_like(q)
    seg_out = seg_lse = None
    if return_segments:
        seg_out = torch.empty((n, topk + 1, Hq, D), dtype=torch.float32, device=q.device)
        seg_lse = torch.empty((n, topk + 1, Hq), dtype=torch.float32, device=q.device)
    if max_kv_len is None:
        max_kv_len = block_table.shape[1] * P
    _check(lib.pkd_segmented_attention_paged(
        _ptr(q), dtype_code(q.dtype), _ptr(kv_cache), num_pages, _ptr(block_table), block_table.stride(0),
        _ptr(seg_start), _ptr(used), _ptr(bias), n, Hq, Hkv, D, P, topk, int(bs), int(local), int(max_kv_len),
        _ptr(out), _ptr(seg_out), _ptr(seg_lse), _stream(stream)))
    return (out, seg_out, seg_lse) if return_segments else out


def lse_merge(part_out, part_lse, prior=None, live=None, out=None, lse_out=None, out_dtype=torch.float32,
              stream=None):
    """Merge partials part_out [N, S, H, D] fp32 by their LSE [N, S, H]."""
    lib = load_library()
    N, S, H, D = part_out.shape
    for t, name in ((part_out, "part_out"), (part_lse, "part_lse"), (prior, "prior"), (live, "live")):
        _cuda(t, name)
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out is None:
        out = torch.empty((N, H, D), dtype=out_dtype, device=part_out.device)
    if lse_out is None:
        lse_out = torch.empty((N, H), dtype=torch.float32, device=part_out.device)
    _check(lib.pkd_lse_merge(_ptr(part_out), _ptr(part_lse), _ptr(prior), _ptr(live), N, S, H, D, _ptr(out),
                             dtype_code(out.dtype), _ptr(lse_out), _stream(stream)))
    return out, lse_out


def cache_write(key, value, slot_mapping, kv_cache, k_scale=1.0, v_scale=1.0, stream=None):
    """Write key/value rows [T, Hkv, D] (bf16/fp16) into their slots of kv_cache
    [num_pages, Hkv, P, 2D] (same dtype, or uint8 / float8_e4m3fn for fp8)."""
    lib = load_library()
    for t, n in ((key, "key"), (value, "value"), (slot_mapping, "slot_mapping"), (kv_cache, "kv_cache")):
        _cuda(t, n)
    T, Hkv, D = key.shape
    num_pages, Hkv2, P, twoD = kv_cache.shape
    if Hkv2 != Hkv or twoD != 2 * D:
        raise ValueError("kv_cache shape does not match key")
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    if key.stride(2) != 1 or key.stride(1) != D or value.stride(2) != 1 or value.stride(1) != D:
        raise ValueError("rows of one token must be contiguous")
    _check(lib.pkd_cache_write(_ptr(key), _ptr(value), dtype_code(key.dtype), key.stride(0), value.stride(0),
                               _ptr(slot_mapping), T, Hkv, D, P, num_pages, _ptr(kv_cache), dtype_code(kv_cache.dtype),
                               float(k_scale), float(v_scale), _stream(stream)))
    return kv_cache


# The host time of the calls below is most of a small step's: they compare device
# indexes, take raw stream handles, enter a device or stream context only where it
# differs from the current one, and check what is right in few expressions; the
# helpers that say what is wrong run only then.
_I32, _I64, _F32, _BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
_CODES = {torch.bfloat16: BF16, torch.float16: FP16, torch.uint8: FP8_E4M3, torch.float8_e4m3fn: FP8_E4M3,
          torch.float32: FP32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_capturing = torch.cuda.is_current_stream_capturing


def _device_error(**tensors):
    """Raise for tensors that are not all on one CUDA device."""
    index = None
    for name, t in tensors.items():
        if t is not None:
            d = t.get_device()
            if d < 0:
                raise ValueError(f"{name} must be a CUDA tensor")
            if index is None:
                index = d
            elif d != index:
                raise ValueError(f"{name} is on cuda:{d}, other arguments on cuda:{index}")


def _code(dtype):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _elsewhere(index, stream):
    """The context of a call whose device or stream is not the current one, or None."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
        if stream.cuda_stream != _raw_stream(index) or _current_device() != index:
            return torch.cuda.stream(stream)
    elif _current_device() != index:
        return torch.cuda.device(index)
    return None


def _token_stride(t, T, H, D, name):
    """Token stride of t [T, H, D], whose tokens must be contiguous rows of H * D."""
    a, b, c = t.stride()
    if c != 1 or (b != D and H > 1):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with contiguous rows per token")
    return a if T > 1 else max(a, H * D)


class _Kept(threading.local):
    """Workspaces of a host thread's calls: (device index, stream) -> (address, bytes, tensor)."""

    def __init__(self):
        self.workspaces = {}


_kept = _Kept()
_WS_HEAD = 256 + 4 * 65536  # PKD_ATTENTION_WORKSPACE_HEAD


def _call_workspace(nbytes, index, stream):
    """A zeroed workspace for a call on the current stream: one kept per stream and
    host thread (grown as needed; launches of two threads' calls may alternate on a
    stream; freed with its thread or by release_workspaces(); workspace_check()
    reads its status), or, while the stream is capturing, one of the graph's own (zeroed by
    the graph), so that two graphs never share one."""
    if not _capturing():
        key = (index, stream)
        ws = _kept.workspaces.get(key)
        if ws is not None and ws[1] >= nbytes:
            return ws
    else:
        key = None
    t = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
    _check(load_library().pkd_workspace_init(t.data_ptr(), _WS_HEAD, stream))
    ws = (t.data_ptr(), nbytes, t)
    if key is not None:
        _kept.workspaces[key] = ws
    return ws


def rope_cache_write(q, key, value, positions, cos_sin, slot_mapping, kv_cache, *, interleaved=False, q_out=None,
                     q_out_dtype=None, q_scale=1.0, k_scale=1.0, v_scale=1.0, stream=None):
    """Rotate q and key by position and append key and value to the paged cache.

    q [T, Hq, D] (or None), key, value [T, Hkv, D] (bf16/fp16; rows of a token
    contiguous, any token stride); positions, slot_mapping int64 [T]; cos_sin
    fp32 [max_position, rotary_dim]; kv_cache [num_pages, Hkv, P, 2D] (the input
    type, or uint8 / float8_e4m3fn).  Returns the rotated q (q_out, allocated
    when not given; of type q_out_dtype: q's, or e4m3(q / q_scale)).
    """
    index = key.get_device()
    if index < 0 or value.get_device() != index or positions.get_device() != index or \
            cos_sin.get_device() != index or slot_mapping.get_device() != index or kv_cache.get_device() != index or \
            (q is not None and q.get_device() != index) or (q_out is not None and q_out.get_device() != index):
        _device_error(key=key, q=q, value=value, positions=positions, cos_sin=cos_sin, slot_mapping=slot_mapping,
                      kv_cache=kv_cache, q_out=q_out)
    if stream is not None or _current_device() != index:
        ctx = _elsewhere(index, stream)
        if ctx is not None:
            with ctx:
                return rope_cache_write(q, key, value, positions, cos_sin, slot_mapping, kv_cache,
                                        interleaved=interleaved, q_out=q_out, q_out_dtype=q_out_dtype, q_scale=q_scale,
                                        k_scale=k_scale, v_scale=v_scale)
    shape = key.shape
    T, Hkv, D = shape
    num_pages, cache_heads, P, twoD = kv_cache.shape
    max_position, rotary_dim = cos_sin.shape
    dtype = key.dtype
    if value.shape != shape or value.dtype != dtype:
        raise ValueError("value must have key's shape and dtype")
    if cache_heads != Hkv or twoD != 2 * D or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous [num_pages, num_kv_heads, page_size, 2 * head_dim]")
    if positions.dtype is not _I64 or slot_mapping.dtype is not _I64 or cos_sin.dtype is not _F32:
        raise TypeError("positions and slot_mapping must be int64, cos_sin float32")
    if positions.dim() != 1 or slot_mapping.dim() != 1 or positions.numel() != T or slot_mapping.numel() != T or not (
            positions.is_contiguous() and slot_mapping.is_contiguous() and cos_sin.is_contiguous()):
        raise ValueError("positions and slot_mapping must be contiguous [T], cos_sin contiguous")
    ks, vs = _token_stride(key, T, Hkv, D, "key"), _token_stride(value, T, Hkv, D, "value")
    Hq = qs = qos = 0
    qp = qop = None
    in_dt = q_dt = _code(dtype)
    if q is not None:
        qT, Hq, qD = qshape = q.shape
        if q.dtype != dtype or qT != T or qD != D:
            raise ValueError("q must be [T, num_heads, head_dim] of key's dtype")
        qs, qp = _token_stride(q, T, Hq, D, "q"), q.data_ptr()
        if q_out is None:
            q_out = torch.empty(qshape, dtype=q_out_dtype or dtype, device=q.device)
            qos = Hq * D
        else:
            if q_out.shape != qshape:
                raise ValueError("q_out must have q's shape")
            qos = _token_stride(q_out, T, Hq, D, "q_out")
        q_dt, qop = _code(q_out.dtype), q_out.data_ptr()
    status = (_lib or load_library()).pkd_rope_cache_write(
        qp, qs, key.data_ptr(), ks, value.data_ptr(), vs, in_dt, positions.data_ptr(), cos_sin.data_ptr(), max_position,
        rotary_dim, 1 if interleaved else 0, slot_mapping.data_ptr(), T, Hq, Hkv, D, P, num_pages, kv_cache.data_ptr(),
        _code(kv_cache.dtype), k_scale, v_scale, qop, qos, q_dt, q_scale, _raw_stream(index))
    if status:
        _check(status)
    return q_out


def _options(T, Hq, B, window, softcap, alibi_slopes, prefix_lens, doc_start):
    if alibi_slopes is prefix_lens is doc_start is None and not window and not softcap:
        return None
    if alibi_slopes is prefix_lens is doc_start is None:
        return ScoreOptions(softcap, None, window, None, None)
    for name, t, dtype, n in (("alibi_slopes", alibi_slopes, _F32, Hq), ("prefix_lens", prefix_lens, _I32, B),
                              ("doc_start", doc_start, _I32, T)):
        if t is not None and (t.dtype is not dtype or t.dim() != 1 or t.numel() != n or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n}")
    return ScoreOptions(softcap, alibi_slopes.data_ptr() if alibi_slopes is not None else None, window,
                        prefix_lens.data_ptr() if prefix_lens is not None else None,
                        doc_start.data_ptr() if doc_start is not None else None)


def _check_table(block_table, seq_lens, what="block_table"):
    """(rows, columns, row stride) of a block table, checked with its lengths."""
    if block_table.dtype is not _I32 or seq_lens.dtype is not _I32:
        raise TypeError(f"{what} and its lengths must be int32")
    if block_table.dim() != 2:
        raise ValueError(f"{what} must be [batch, columns]")
    rows, columns = block_table.shape
    a, b = block_table.stride()
    if (b != 1 and columns > 1) or seq_lens.dim() != 1 or seq_lens.numel() != rows or not seq_lens.is_contiguous():
        raise ValueError(f"{what} must be [batch, columns] with contiguous rows, its lengths contiguous [batch]")
    return rows, columns, a if rows > 1 else max(a, columns)


def _check_cache(D, kv_cache):
    """(pages, kv heads, page size) of a cache of heads of D."""
    if kv_cache.dim() != 4 or kv_cache.shape[3] != 2 * D or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous [num_pages, num_kv_heads, page_size, 2 * head_dim]")
    return kv_cache.shape[:3]


def _results(out, lse, shape, dtype, device):
    """out and lse of a call: the given ones, checked, or new ones."""
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    elif out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be contiguous {tuple(shape)}")
    if lse is None:
        lse = torch.empty(shape[:-1], dtype=_F32, device=device)
    elif lse.shape != shape[:-1] or not lse.is_contiguous() or lse.dtype is not _F32:
        raise ValueError(f"lse must be contiguous float32 {tuple(shape[:-1])}")
    return out, lse


@functools.lru_cache(maxsize=4096)
def _attention_bytes(*plan):
    """Workspace bytes of a paged_attention plan (window and prefix mask last)."""
    opt = ScoreOptions(0.0, None, plan[-2], 16 if plan[-1] else None, None)
    n = load_library().pkd_paged_attention_workspace_size(*plan[:-2], opt)
    if n == 0:
        raise PkdError(EUNSUPPORTED, load_library().pkd_last_error().decode())
    return n


@functools.lru_cache(maxsize=4096)
def _prefix_bytes(*plan):
    """Workspace bytes of a prefix_decode plan."""
    n = load_library().pkd_prefix_decode_workspace_size(*plan)
    if n == 0:
        raise PkdError(EUNSUPPORTED, load_library().pkd_last_error().decode())
    return n


def paged_attention(q, kv_cache, block_table, seq_lens, query_start, scale, *, causal=True, window=0, softcap=0.0,
                    alibi_slopes=None, prefix_lens=None, doc_start=None, max_query_len=None, max_kv_len=None,
                    q_scale=1.0, k_scale=1.0, v_scale=1.0, out=None, lse=None, out_dtype=None, workspace=None,
                    test_timeout=False, stream=None):
    """Attention of ragged query tokens over the paged cache (prompts, chunks, steps).

    q [T, Hq, D] (the cache's type; any token stride); request b's tokens are
    rows query_start[b] : query_start[b + 1] (int32 [B + 1]), the last of its
    seq_lens[b] keys.  softcap: c * tanh(s / c); alibi_slopes fp32 [Hq]: minus
    slope * distance; window: keys from position - (window - 1) on; prefix_lens
    int32 [B]: keys that all of a request's tokens see; doc_start int32 [T]:
    first key of each token's document.  max_query_len (default T) and
    max_kv_len (default the table's capacity) bound the lengths on the host and
    with them choose the kernel and the split of the keys: give the batch's own
    (1 for single tokens, which have a kernel of their own; without it T tokens
    may be one request's).
    Lengths, pages or starts out of range are clamped or skipped; workspace_check
    (of workspace, or of the one kept for calls without) then says so.
    test_timeout sets the diagnostic PKD_FLAG_TEST_TIMEOUT.
    Returns (out [T, Hq, D], lse fp32 [T, Hq]); rows of no request keep what was
    in out and lse (nothing in particular where the call allocates them).
    """
    index = q.get_device()
    if index < 0 or kv_cache.get_device() != index or block_table.get_device() != index or \
            seq_lens.get_device() != index or query_start.get_device() != index or \
            not (alibi_slopes is prefix_lens is doc_start is out is lse is workspace is None):
        _device_error(q=q, kv_cache=kv_cache, block_table=block_table, seq_lens=seq_lens, query_start=query_start,
                      alibi_slopes=alibi_slopes, prefix_lens=prefix_lens, doc_start=doc_start, out=out, lse=lse,
                      workspace=workspace)
    if stream is not None or _current_device() != index:
        ctx = _elsewhere(index, stream)
        if ctx is not None:
            with ctx:
                return paged_attention(q, kv_cache, block_table, seq_lens, query_start, scale, causal=causal,
                                       window=window, softcap=softcap, alibi_slopes=alibi_slopes,
                                       prefix_lens=prefix_lens, doc_start=doc_start, max_query_len=max_query_len,
                                       max_kv_len=max_kv_len, q_scale=q_scale, k_scale=k_scale, v_scale=v_scale,
                                       out=out, lse=lse, out_dtype=out_dtype, workspace=workspace,
                                       test_timeout=test_timeout)
    T, Hq, D = shape = q.shape
    qs = _token_stride(q, T, Hq, D, "q")
    num_pages, Hkv, P = _check_cache(D, kv_cache)
    B, columns, stride = _check_table(block_table, seq_lens)
    if query_start.dtype is not _I32 or query_start.dim() != 1 or query_start.numel() != B + 1 or \
            not query_start.is_contiguous():
        raise ValueError("query_start must be a contiguous int32 tensor [batch + 1]")
    opt = _options(T, Hq, B, window, softcap, alibi_slopes, prefix_lens, doc_start)
    if max_query_len is None:
        max_query_len = max(T, 1)
    if max_kv_len is None:
        max_kv_len = columns * P
    if window >> 31 or max_query_len >> 31 or max_kv_len >> 31:
        raise ValueError("window, max_query_len and max_kv_len must lie in [0, 2^31)")
    dtype = q.dtype
    q_dt, kv_dt = _code(dtype), _code(kv_cache.dtype)
    out, lse = _results(out, lse, shape, out_dtype or (_BF16 if kv_dt == FP8_E4M3 else dtype), q.device)
    s = _raw_stream(index)
    if workspace is None:
        ws, ws_bytes, keep = _call_workspace(_attention_bytes(B, T, max_query_len, Hq, Hkv, D, P, max_kv_len, kv_dt,
                                                              window, prefix_lens is not None), index, s)
    else:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    status = (_lib or load_library()).pkd_paged_attention(
        q.data_ptr(), q_dt, qs, kv_cache.data_ptr(), kv_dt, num_pages, block_table.data_ptr(), stride,
        seq_lens.data_ptr(), query_start.data_ptr(), B, T, max_query_len, Hq, Hkv, D, P, max_kv_len, scale, q_scale,
        k_scale, v_scale, opt, out.data_ptr(), _code(out.dtype), lse.data_ptr(), ws, ws_bytes,
        (FLAG_CAUSAL if causal else 0) | (FLAG_TEST_TIMEOUT if test_timeout else 0), s)
    if status:
        _check(status)
    return out, lse


def prefix_decode(q, kv_cache, prefix_table, prefix_lens, block_table, seq_lens, scale, *, group_start=None,
                  causal=False, softcap=0.0, max_prefix_len=None, max_kv_len=None, q_scale=1.0, k_scale=1.0,
                  v_scale=1.0, out=None, lse=None, out_dtype=None, workspace=None, test_timeout=False, stream=None):
    """Decode of a batch whose requests share prefixes, each computed once.

    q [B, sq, Hq, D]; prefix_table int32 [groups, columns] and prefix_lens int32
    [groups]: the shared prefixes' pages; group_start int32 [groups + 1]: requests
    group_start[g] : group_start[g + 1] follow prefix g (default: one group of
    all); block_table, seq_lens: the requests' own keys behind the prefix.
    workspace_check reads the status, as for paged_attention.
    test_timeout sets the diagnostic PKD_FLAG_TEST_TIMEOUT.
    Returns (out [B, sq, Hq, D], lse fp32 [B, sq, Hq]) over both.
    """
    index = q.get_device()
    if index < 0 or kv_cache.get_device() != index or prefix_table.get_device() != index or \
            prefix_lens.get_device() != index or block_table.get_device() != index or \
            seq_lens.get_device() != index or (group_start is not None and group_start.get_device() != index) or \
            not (out is lse is workspace is None):
        _device_error(q=q, kv_cache=kv_cache, prefix_table=prefix_table, prefix_lens=prefix_lens,
                      block_table=block_table, seq_lens=seq_lens, group_start=group_start, out=out, lse=lse,
                      workspace=workspace)
    if stream is not None or _current_device() != index:
        ctx = _elsewhere(index, stream)
        if ctx is not None:
            with ctx:
                return prefix_decode(q, kv_cache, prefix_table, prefix_lens, block_table, seq_lens, scale,
                                     group_start=group_start, causal=causal, softcap=softcap,
                                     max_prefix_len=max_prefix_len, max_kv_len=max_kv_len, q_scale=q_scale,
                                     k_scale=k_scale, v_scale=v_scale, out=out, lse=lse, out_dtype=out_dtype,
                                     workspace=workspace, test_timeout=test_timeout)
    if q.dim() != 4 or not q.is_contiguous():
        raise ValueError("q must be contiguous [batch, sq, num_heads, head_dim]")
    B, sq, Hq, D = shape = q.shape
    num_pages, Hkv, P = _check_cache(D, kv_cache)
    rows, columns, stride = _check_table(block_table, seq_lens)
    groups, pcolumns, pstride = _check_table(prefix_table, prefix_lens, "prefix_table")
    if rows != B:
        raise ValueError("block_table must have one row per request")
    if group_start is None:
        if groups != 1:
            raise ValueError("group_start is needed with more than one prefix")
    elif group_start.dtype is not _I32 or group_start.dim() != 1 or group_start.numel() != groups + 1 or \
            not group_start.is_contiguous():
        raise ValueError("group_start must be a contiguous int32 tensor [groups + 1]")
    if max_prefix_len is None:
        max_prefix_len = pcolumns * P
    if max_kv_len is None:
        max_kv_len = columns * P
    if max_prefix_len >> 31 or max_kv_len >> 31:
        raise ValueError("max_prefix_len and max_kv_len must lie in [0, 2^31)")
    dtype = q.dtype
    q_dt, kv_dt = _code(dtype), _code(kv_cache.dtype)
    out, lse = _results(out, lse, shape, out_dtype or (_BF16 if kv_dt == FP8_E4M3 else dtype), q.device)
    s = _raw_stream(index)
    if workspace is None:
        ws, ws_bytes, keep = _call_workspace(_prefix_bytes(B, sq, Hq, Hkv, D, P, groups, max_prefix_len, max_kv_len,
                                                           kv_dt), index, s)
    else:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    status = (_lib or load_library()).pkd_prefix_decode(
        q.data_ptr(), q_dt, kv_cache.data_ptr(), kv_dt, num_pages, prefix_table.data_ptr(), pstride,
        prefix_lens.data_ptr(), group_start.data_ptr() if group_start is not None else None, groups, max_prefix_len,
        block_table.data_ptr(), stride, seq_lens.data_ptr(), B, sq, Hq, Hkv, D, P, max_kv_len, scale, q_scale, k_scale,
        v_scale, softcap, out.data_ptr(), _code(out.dtype), lse.data_ptr(), ws, ws_bytes,
        (FLAG_CAUSAL if causal else 0) | (FLAG_TEST_TIMEOUT if test_timeout else 0), s)
    if status:
        _check(status)
    return out, lse
