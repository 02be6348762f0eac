"""GB300 (sm_103a) DeepSeek-Sparse-Attention prefill over an MLA latent KV cache.

A thin ctypes binding over ``libdsa.so`` (C ABI in ``include/dsa.h``).  The
functions carry the C names and only marshal arguments: they check tensor
dtypes/devices, allocate outputs with torch when none are given, pass raw
device pointers and the current CUDA stream, and raise ``DSAError`` on a
non-zero status.  All arithmetic happens in the library's CUDA kernels;
there is no CPU fallback: without the built library every call raises.

Forms (see the header for the exact contracts):
  dsa_sparse_prefill      per-token sparse attention over each token's top-k rows
  dsa_sparse_prefill_host the same from and to host memory, copies overlapped with the kernel
  dsa_sparse_prefill_host_noalloc  the same without a workspace (fixed library scratch)
  dsa_union_build         sorted union per group + head-group membership mask
  dsa_grouped_prefill     G = 128/H tokens as 128 pseudo-heads over the union
  dsa_topk_to_key_mask    packed per-token key mask from the top-k rows
  dsa_masked_mha_prefill  masked dense MHA with per-head q/k/v
  dsa_masked_mha_prefill_strided  the same on strided views, RoPE key columns shared
  dsa_choose_form         predicted time of each form and the fastest (host only)
  dsa_kv_fp8_quantize / dsa_kv_fp8_dequantize  FP8 latent rows of the KV cache

The decode step over the same paged cache:
  dsa_rope                rotary positions and their gradient (frequencies from dsa_rope_freqs)
  dsa_kv_append           new tokens' latent rows into the cache, bf16 or FP8, RoPE columns rotated
  dsa_paged_decode        attention of one new token per request, whole context or its top-k positions
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")
MAX_REQUESTS = 512

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_CUDA, DSA_ERR_DEVICE = range(5)


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


_lib_handle = None

_VP = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_D = ctypes.c_double
_I32P = ctypes.POINTER(ctypes.c_int32)
_L = ctypes.c_int64

FORMS = ("per_token", "grouped", "masked")


class FormCalibration(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in (
        "hbm_gbs", "bf16_tflops", "per_token_frac", "per_token_ms0", "union_frac", "union_ms0",
        "grouped_frac_576", "grouped_frac_512", "grouped_ms0", "masked_frac_192", "masked_frac_256", "masked_ms0",
        "key_mask_frac", "key_mask_ms0", "union_growth")]


class FormQuery(ctypes.Structure):
    _fields_ = [("num_req", ctypes.c_int), ("q_lens", ctypes.POINTER(ctypes.c_int32)),
                ("kv_lens", ctypes.POINTER(ctypes.c_int32)), ("H", ctypes.c_int), ("k", ctypes.c_int),
                ("d_qk", ctypes.c_int), ("masked_d_qk", ctypes.c_int), ("masked_d_v", ctypes.c_int),
                ("union_rows", ctypes.c_double)]


class FormEstimate(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * 3), ("form", ctypes.c_int), ("union_rows", ctypes.c_double)]


class RopeFreqs(ctypes.Structure):
    """Rotary frequencies (dsa_rope_freqs)."""
    _fields_ = [("d_rope", ctypes.c_int32), ("layout", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * 128)]


ROPE_LAYOUTS = ("interleaved", "half")
ROPE_SCALINGS = ("none", "linear", "yarn")

_SIGNATURES = {
    "dsa_status_string": (ctypes.c_char_p, [_I]),
    "dsa_version": (_I, []),
    "dsa_union_pad": (ctypes.c_int64, [_I, _I, _I]),
    "dsa_num_groups": (_I, [_I32P, _I, _I, _I, ctypes.POINTER(ctypes.c_int)]),
    "dsa_union_build": (_I, [_VP, _I, _I, _I, _I, _I32P, _I, _I, _VP, _VP, _VP, _I, _VP]),
    "dsa_sparse_prefill": (_I, [_VP, _VP, _I, _I, _VP, _I, _I, _I, _I, _I, _I, _F, _VP, _VP, _VP]),
    "dsa_grouped_prefill": (_I, [_VP, _VP, _I, _I, _VP, _VP, _VP, _I, _I, _I32P, _I, _I, _I, _I, _I, _F, _VP,
                                 _VP, _VP]),
    "dsa_topk_to_key_mask": (_I, [_VP, _I, _I, _I, _I32P, _I32P, _I, _VP, _I, _VP]),
    "dsa_local_to_global": (_I, [_VP, _I, _I, _I, _I32P, _I32P, _I, _VP, _I, _I, _I, _VP, _VP]),
    "dsa_masked_mha_prefill": (_I, [_VP, _VP, _VP, _VP, _I, _I32P, _I32P, _I, _I, _I, _I, _I, _F, _VP, _VP,
                                    _VP]),
    "dsa_masked_mha_prefill_strided": (_I, [_VP, _L, _L, _VP, _L, _L, _VP, _L, _VP, _L, _L, _VP, _I, _I32P, _I32P,
                                            _I, _I, _I, _I, _I, _I, _F, _VP, _VP, _VP]),
    "dsa_sparse_prefill_host_workspace": (_L, [_I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "dsa_sparse_prefill_host_plan": (_I, [_I, _I, _I, _I32P, _I, ctypes.POINTER(ctypes.c_int)]),
    "dsa_sparse_prefill_host": (_I, [_VP, _VP, _I, _I, _I, _VP, _I, _I, _I, _I, _I, _I, _F, _VP, _VP, _VP, _L, _I,
                                     _VP]),
    "dsa_sparse_prefill_host_noalloc": (_I, [_VP, _VP, _I, _I, _I, _VP, _I, _I, _I, _I, _I, _I, _F, _VP, _VP, _I,
                                             _VP]),
    "dsa_kv_fp8_row_bytes": (_L, [_I]),
    "dsa_kv_fp8_quantize": (_I, [_VP, _I, _I, _I, _VP, _VP]),
    "dsa_kv_fp8_dequantize": (_I, [_VP, _I, _I, _VP, _I, _VP]),
    "dsa_sparse_prefill_fp8": (_I, [_VP, _VP, _I, _I, _VP, _I, _I, _I, _I, _I, _I, _F, _VP, _VP, _VP]),
    "dsa_rope_freqs_init": (_I, [ctypes.POINTER(RopeFreqs), _I, _D, _I, _I, _D, _I, _D, _D, _F]),
    "dsa_rope": (_I, [_VP, _L, _L, _VP, _L, _L, _I, _VP, _I, _I, ctypes.POINTER(RopeFreqs), _I, _VP]),
    "dsa_kv_append": (_I, [_VP, _L, _VP, _L, _I, _I, _VP, _VP, _VP, _I, _I, _I, ctypes.POINTER(RopeFreqs), _VP, _I, _I,
                           _I, _VP]),
    "dsa_paged_decode_workspace": (_L, [_I, _I, _L]),
    "dsa_paged_decode": (_I, [_VP, _VP, _I, _I, _I, _VP, _I, _I, _VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP, _VP, _VP,
                              _L, _VP]),
    "dsa_form_calibration_default": (_I, [ctypes.POINTER(FormCalibration)]),
    "dsa_choose_form": (_I, [ctypes.POINTER(FormQuery), ctypes.POINTER(FormCalibration),
                             ctypes.POINTER(FormEstimate)]),
    "dsa_last_device_error": (_I, [_VP, ctypes.POINTER(ctypes.c_uint32)]),
    "dsa_debug_trace": (_I, [_VP, _I]),
    "dsa_debug_wait_timeout": (_I, [_VP]),
}

EXPORTED = tuple(_SIGNATURES)


def lib() -> ctypes.CDLL:
    """The loaded ``libdsa.so`` (raises if it has not been built)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m dsa_sparse_mla_prefill_gb300.build` "
                               "(the library has no CPU fallback)")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib_handle = h
    return _lib_handle


def status_string(status: int) -> str:
    return lib().dsa_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != DSA_OK:
        raise DSAError(status, where)


def _host_i32(arr):
    """Host int32 array for a cu_seqlens argument (None stays None)."""
    if arr is None:
        return None, None
    try:
        import torch
        if isinstance(arr, torch.Tensor):
            arr = arr.detach().cpu().numpy()
    except ImportError:  # pragma: no cover
        pass
    a = np.ascontiguousarray(np.asarray(arr, dtype=np.int32))
    return a, a.ctypes.data_as(_I32P)


def _stream(stream, device):
    if stream is None:
        torch = _torch or _load_torch()
        if device.type != "cuda":
            raise ValueError(f"expected CUDA tensors, got one on {device}")
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device() if device.index is None else device.index))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _empty(shape, dtype, device, stream):
    """A new tensor for a call on `stream` (None: the current one) to write.  Another stream's is made
    as that stream's own memory: the current stream's may have been freed there while its queued
    kernels still use it, and nothing orders the call behind them.  The current stream, which the
    caller most likely reads the tensor on, is recorded as its user."""
    torch = _torch or _load_torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle == here.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):   # a handle: 0 and 1 are names of the default stream
        stream = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _need(t, dtype, name, ndim=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    return t


def dsa_union_pad(G: int, k: int, union_block: int = 128) -> int:
    return int(lib().dsa_union_pad(G, k, union_block))


def dsa_num_groups(cu_seqlens_q, T: int, G: int) -> int:
    arr, ptr = _host_i32(cu_seqlens_q)
    n = ctypes.c_int(0)
    nreq = 0 if arr is None else len(arr) - 1
    _check(lib().dsa_num_groups(ptr, nreq, T, G, ctypes.byref(n)), "dsa_num_groups")
    return n.value


def dsa_union_build(idx, k: int, G: int, N: int, cu_seqlens_q=None, union_pad: int | None = None,
                    union_block: int = 128, out=None, stream=None):
    """Returns (union_idx [groups, union_pad] int32, union_len [groups] int32,
    mask [groups, union_pad] uint8)."""
    import torch
    _need(idx, torch.int32, "idx", 2)
    T, ld = idx.shape
    if union_pad is None:
        union_pad = dsa_union_pad(G, k, union_block)
    ng = dsa_num_groups(cu_seqlens_q, T, G)
    if out is None:
        u = _empty((ng, union_pad), torch.int32, idx.device, stream)
        ul = _empty((ng,), torch.int32, idx.device, stream)
        m = _empty((ng, union_pad), torch.uint8, idx.device, stream)
    else:
        u, ul, m = out
    arr, ptr = _host_i32(cu_seqlens_q)
    nreq = 0 if arr is None else len(arr) - 1
    _check(lib().dsa_union_build(idx.data_ptr(), T, k, ld, G, ptr, nreq, N, u.data_ptr(), ul.data_ptr(),
                                 m.data_ptr(), union_pad, _stream(stream, idx.device)), "dsa_union_build")
    return u, ul, m


def dsa_sparse_prefill(q, kv, idx, k: int, scale: float, d_v: int = 512, out=None, lse=None, stream=None):
    """Per-token sparse prefill.  q [T, H, d_qk] bf16, kv [N, ld_kv] bf16 (the
    first d_qk columns are the latent key, the first d_v the value), idx
    [T, ld] int32 global rows.  Returns (out [T, H, d_v] bf16, lse [T, H] fp32)."""
    import torch
    _need(q, torch.bfloat16, "q", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(idx, torch.int32, "idx", 2)
    T, H, d_qk = q.shape
    N, ld_kv = kv.shape
    if idx.shape[0] != T:
        raise ValueError("idx rows must match q tokens")
    if out is None:
        out = _empty((T, H, d_v), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty((T, H), torch.float32, q.device, stream)
    _check(lib().dsa_sparse_prefill(q.data_ptr(), kv.data_ptr(), N, ld_kv, idx.data_ptr(), T, H, d_qk, d_v, k,
                                    idx.shape[1], float(scale), out.data_ptr(), lse.data_ptr(),
                                    _stream(stream, q.device)), "dsa_sparse_prefill")
    return out, lse


def _host_tensor(t, dtype, name, ndim):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != ndim:
        raise TypeError(f"{name} must be a {ndim}-D {dtype} tensor")
    if t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous host tensor (pinned for overlapped copies)")
    return t


def dsa_sparse_prefill_host_workspace(T: int, N: int, ld_kv: int, H: int, d_qk: int, ld: int, chunk_tokens: int,
                                      kv_on_host: bool = True, d_v: int = 512) -> int:
    """Device workspace bytes dsa_sparse_prefill_host needs for these shapes."""
    n = lib().dsa_sparse_prefill_host_workspace(T, N, ld_kv, H, d_qk, d_v, ld, chunk_tokens, int(bool(kv_on_host)))
    if n < 0:
        raise DSAError(DSA_ERR_INVALID_ARG, "dsa_sparse_prefill_host_workspace")
    return int(n)


def dsa_sparse_prefill_host_plan(T: int, chunk_tokens: int, num_sms: int) -> list:
    """Chunk sizes the host-buffer call uses for T tokens on num_sms SMs (host only)."""
    n = ctypes.c_int(0)
    st = lib().dsa_sparse_prefill_host_plan(T, chunk_tokens, num_sms, None, 0, ctypes.byref(n))
    if st != DSA_OK and n.value == 0:
        _check(st, "dsa_sparse_prefill_host_plan")   # bad sizes
    buf = (ctypes.c_int32 * max(1, n.value))()
    _check(lib().dsa_sparse_prefill_host_plan(T, chunk_tokens, num_sms, buf, n.value, ctypes.byref(n)),
           "dsa_sparse_prefill_host_plan")
    return [int(buf[i]) for i in range(n.value)]


def dsa_sparse_prefill_host(q, kv, idx, k: int, scale: float, out, lse, workspace, chunk_tokens: int = 2048,
                            stream=None):
    """Per-token sparse prefill from and to host memory: q [T, H, d_qk] bf16, idx [T, ld] int32,
    out [T, H, 512] bf16 and lse [T, H] fp32 are host tensors (pinned, for the copies to overlap
    the kernel), kv [N, ld_kv] bf16 a host or CUDA tensor, workspace a CUDA uint8 tensor of
    dsa_sparse_prefill_host_workspace bytes.  A workspace sized with chunk_tokens >= T selects
    the streamed form (one kernel launch, copies in chunks of at most chunk_tokens); a smaller
    one the ring of chunk launches.  Asynchronous on `stream` (synchronize before reading out
    and lse)."""
    import torch
    _host_tensor(q, torch.bfloat16, "q", 3)
    _host_tensor(idx, torch.int32, "idx", 2)
    _host_tensor(out, torch.bfloat16, "out", 3)
    _host_tensor(lse, torch.float32, "lse", 2)
    if kv.dtype != torch.bfloat16 or kv.dim() != 2 or not kv.is_contiguous():
        raise TypeError("kv must be a contiguous 2-D bf16 tensor")
    _need(workspace, torch.uint8, "workspace", 1)
    T, H, d_qk = q.shape
    N, ld_kv = kv.shape
    if idx.shape[0] != T or out.shape[0] != T or lse.shape != (T, H):
        raise ValueError("q, idx, out and lse must cover the same tokens")
    _check(lib().dsa_sparse_prefill_host(q.data_ptr(), kv.data_ptr(), 0 if kv.is_cuda else 1, N, ld_kv,
                                         idx.data_ptr(), T, H, d_qk, out.shape[2], k, idx.shape[1], float(scale),
                                         out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                         int(chunk_tokens), _stream(stream, workspace.device)),
           "dsa_sparse_prefill_host")
    return out, lse


HOST_NOALLOC_SCRATCH_BYTES = 64 << 20


def dsa_sparse_prefill_host_noalloc(q, kv, idx, k: int, scale: float, out, lse, chunk_tokens: int = 152,
                                    stream=None):
    """dsa_sparse_prefill_host for callers that cannot allocate device memory: the same
    arguments without a workspace; the library's fixed 64 MiB device scratch holds the
    chunks in flight.  Shapes whose buffers need more (dsa_sparse_prefill_host_workspace)
    raise DSAError(DSA_ERR_UNSUPPORTED); lower chunk_tokens then.  Calls that overlap on
    the GPU share the scratch and race: keep them on one stream."""
    import torch
    _host_tensor(q, torch.bfloat16, "q", 3)
    _host_tensor(idx, torch.int32, "idx", 2)
    _host_tensor(out, torch.bfloat16, "out", 3)
    _host_tensor(lse, torch.float32, "lse", 2)
    if kv.dtype != torch.bfloat16 or kv.dim() != 2 or not kv.is_contiguous():
        raise TypeError("kv must be a contiguous 2-D bf16 tensor")
    T, H, d_qk = q.shape
    N, ld_kv = kv.shape
    if idx.shape[0] != T or out.shape[0] != T or lse.shape != (T, H):
        raise ValueError("q, idx, out and lse must cover the same tokens")
    dev = kv.device if kv.is_cuda else torch.device("cuda", torch.cuda.current_device())
    _check(lib().dsa_sparse_prefill_host_noalloc(q.data_ptr(), kv.data_ptr(), 0 if kv.is_cuda else 1, N, ld_kv,
                                                 idx.data_ptr(), T, H, d_qk, out.shape[2], k, idx.shape[1],
                                                 float(scale), out.data_ptr(), lse.data_ptr(), int(chunk_tokens),
                                                 _stream(stream, dev)),
           "dsa_sparse_prefill_host_noalloc")
    return out, lse


def dsa_grouped_prefill(q, kv, union_idx, union_len, mask, G: int, scale: float, cu_seqlens_q=None,
                        d_v: int = 512, out=None, lse=None, stream=None):
    """Grouped sparse prefill over (union_idx, union_len, mask) from dsa_union_build."""
    import torch
    _need(q, torch.bfloat16, "q", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(union_idx, torch.int32, "union_idx", 2)
    _need(union_len, torch.int32, "union_len", 1)
    _need(mask, torch.uint8, "mask", 2)
    T, H, d_qk = q.shape
    N, ld_kv = kv.shape
    if out is None:
        out = _empty((T, H, d_v), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty((T, H), torch.float32, q.device, stream)
    arr, ptr = _host_i32(cu_seqlens_q)
    nreq = 0 if arr is None else len(arr) - 1
    _check(lib().dsa_grouped_prefill(q.data_ptr(), kv.data_ptr(), N, ld_kv, union_idx.data_ptr(),
                                     union_len.data_ptr(), mask.data_ptr(), union_idx.shape[1], G, ptr, nreq, T,
                                     H, d_qk, d_v, float(scale), out.data_ptr(), lse.data_ptr(),
                                     _stream(stream, q.device)), "dsa_grouped_prefill")
    return out, lse


def dsa_topk_to_key_mask(idx, k: int, words: int, cu_seqlens_q=None, cu_seqlens_kv=None, out=None, stream=None):
    """Packed key mask [T, words] uint32 (viewed as int32 in torch)."""
    import torch
    _need(idx, torch.int32, "idx", 2)
    T, ld = idx.shape
    if out is None:
        out = _empty((T, words), torch.int32, idx.device, stream)
    aq, pq = _host_i32(cu_seqlens_q)
    ak, pk = _host_i32(cu_seqlens_kv)
    nreq = 0 if aq is None else len(aq) - 1
    _check(lib().dsa_topk_to_key_mask(idx.data_ptr(), T, k, ld, pq, pk, nreq, out.data_ptr(), words,
                                      _stream(stream, idx.device)), "dsa_topk_to_key_mask")
    return out


def dsa_local_to_global(idx_local, k: int, kv_lens, block_table, block_size: int, N: int, cu_seqlens_q=None,
                        out=None, stream=None):
    """Request-local KV positions [T, ld] -> physical rows of a paged KV cache
    through block_table [num_req, max_blocks] (device int32).  kv_lens: host
    KV length per request.  Returns idx_global [T, ld] (may be ``out`` =
    ``idx_local`` for in place)."""
    import torch
    _need(idx_local, torch.int32, "idx_local", 2)
    _need(block_table, torch.int32, "block_table", 2)
    T, ld = idx_local.shape
    if out is None:
        out = _empty(idx_local.shape, torch.int32, idx_local.device, stream)
    aq, pq = _host_i32(cu_seqlens_q)
    al, pl = _host_i32(kv_lens)
    nreq = 0 if aq is None else len(aq) - 1
    _check(lib().dsa_local_to_global(idx_local.data_ptr(), T, k, ld, pq, pl, nreq, block_table.data_ptr(),
                                     block_table.shape[1], block_size, N, out.data_ptr(),
                                     _stream(stream, idx_local.device)), "dsa_local_to_global")
    return out


def dsa_masked_mha_prefill(q, k, v, key_mask, scale: float, cu_seqlens_q=None, cu_seqlens_kv=None, out=None,
                           lse=None, stream=None):
    """Masked dense MHA.  q [T, H, d_qk], k [Nk, H, d_qk], v [Nk, H, d_v] bf16;
    key_mask [T, words] (int32/uint32 bits).  Returns (out [T, H, d_v], lse [T, H])."""
    import torch
    _need(q, torch.bfloat16, "q", 3)
    _need(k, torch.bfloat16, "k", 3)
    _need(v, torch.bfloat16, "v", 3)
    if key_mask.dtype not in (torch.int32,):
        raise TypeError("key_mask must be int32 (bit pattern of uint32 words)")
    _need(key_mask, key_mask.dtype, "key_mask", 2)
    T, H, d_qk = q.shape
    d_v = v.shape[2]
    if out is None:
        out = _empty((T, H, d_v), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty((T, H), torch.float32, q.device, stream)
    aq, pq = _host_i32(cu_seqlens_q)
    ak, pk = _host_i32(cu_seqlens_kv)
    nreq = 0 if aq is None else len(aq) - 1
    _check(lib().dsa_masked_mha_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), key_mask.data_ptr(),
                                        key_mask.shape[1], pq, pk, nreq, T, H, d_qk, d_v, float(scale),
                                        out.data_ptr(), lse.data_ptr(), _stream(stream, q.device)),
           "dsa_masked_mha_prefill")
    return out, lse


def dsa_masked_mha_prefill_strided(q, k, v, key_mask, scale: float, k_pe=None, cu_seqlens_q=None,
                                   cu_seqlens_kv=None, out=None, lse=None, stream=None):
    """Masked dense MHA on strided views.  q [T, H, d_qk], k [Nk, H, d_qk - d_rope] and
    v [Nk, H, d_v] bf16 with unit stride in the last dimension (e.g. k = kv[..., :256] and
    v = kv[..., 256:] of one [Nk, H, 512] projection output, no copies); k_pe [Nk, d_rope]
    (d_rope = 64) holds the RoPE key columns shared by all heads, or None (d_rope = 0).
    Returns (out [T, H, d_v], lse [T, H])."""
    import torch
    for name, x in (("q", q), ("k", k), ("v", v)):
        if x.dtype != torch.bfloat16 or x.dim() != 3 or x.stride(2) != 1:
            raise TypeError(f"{name} must be a 3-D bf16 tensor with unit stride in its last dimension")
    if key_mask.dtype != torch.int32 or key_mask.dim() != 2 or not key_mask.is_contiguous():
        raise TypeError("key_mask must be a contiguous 2-D int32 tensor (bit pattern of uint32 words)")
    d_rope, pe_ptr, pe_stride = 0, None, 0
    if k_pe is not None:
        if k_pe.dtype != torch.bfloat16 or k_pe.dim() != 2 or k_pe.stride(1) != 1:
            raise TypeError("k_pe must be a 2-D bf16 tensor with unit stride in its last dimension")
        d_rope, pe_ptr, pe_stride = k_pe.shape[1], k_pe.data_ptr(), k_pe.stride(0)
    T, H, d_qk = q.shape
    d_v = v.shape[2]
    if k.shape[2] + d_rope != d_qk:
        raise ValueError("k columns + k_pe columns must equal q's head dim")
    if out is None:
        out = _empty((T, H, d_v), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty((T, H), torch.float32, q.device, stream)
    aq, pq = _host_i32(cu_seqlens_q)
    ak, pk = _host_i32(cu_seqlens_kv)
    nreq = 0 if aq is None else len(aq) - 1
    _check(lib().dsa_masked_mha_prefill_strided(
        q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1), pe_ptr, pe_stride,
        v.data_ptr(), v.stride(0), v.stride(1), key_mask.data_ptr(), key_mask.shape[1], pq, pk, nreq, T, H,
        d_qk, d_rope, d_v, float(scale), out.data_ptr(), lse.data_ptr(), _stream(stream, q.device)),
        "dsa_masked_mha_prefill_strided")
    return out, lse


def dsa_kv_fp8_row_bytes(d_rope: int) -> int:
    n = int(lib().dsa_kv_fp8_row_bytes(int(d_rope)))
    if n < 0:
        raise DSAError(DSA_ERR_UNSUPPORTED, "dsa_kv_fp8_row_bytes")
    return n


def dsa_kv_fp8_quantize(kv, d_rope: int = 64, out=None, stream=None):
    """bf16 latent rows kv [N, ld_kv] (CUDA) to FP8 rows [N, dsa_kv_fp8_row_bytes(d_rope)] uint8."""
    import torch
    _need(kv, torch.bfloat16, "kv", 2)
    N, ld = kv.shape
    if out is None:
        out = _empty((N, dsa_kv_fp8_row_bytes(d_rope)), torch.uint8, kv.device, stream)
    _need(out, torch.uint8, "out", 2)
    _check(lib().dsa_kv_fp8_quantize(kv.data_ptr(), N, ld, int(d_rope), out.data_ptr(), _stream(stream, kv.device)),
           "dsa_kv_fp8_quantize")
    return out


def dsa_kv_fp8_dequantize(fp8, d_rope: int = 64, out=None, stream=None):
    """FP8 rows [N, row_bytes] uint8 (CUDA) to bf16 latent rows [N, 512 + d_rope] (or into out [N, ld_kv])."""
    import torch
    _need(fp8, torch.uint8, "fp8", 2)
    N = fp8.shape[0]
    if fp8.shape[1] != dsa_kv_fp8_row_bytes(d_rope):
        raise ValueError("fp8 rows must be dsa_kv_fp8_row_bytes(d_rope) bytes wide")
    if out is None:
        out = _empty((N, 512 + d_rope), torch.bfloat16, fp8.device, stream)
    _need(out, torch.bfloat16, "out", 2)
    _check(lib().dsa_kv_fp8_dequantize(fp8.data_ptr(), N, int(d_rope), out.data_ptr(), out.shape[1],
                                       _stream(stream, fp8.device)), "dsa_kv_fp8_dequantize")
    return out


def dsa_form_calibration_default() -> FormCalibration:
    """The GB300 calibration of the form model (fields as in include/dsa.h)."""
    c = FormCalibration()
    _check(lib().dsa_form_calibration_default(ctypes.byref(c)), "dsa_form_calibration_default")
    return c


def dsa_choose_form(q_lens, kv_lens, H: int, k: int, d_qk: int = 576, masked_dims=None, union_rows=None,
                    calibration: FormCalibration = None):
    """Predicted ms of each form and the fastest applicable one (host only).  q_lens / kv_lens
    per request (queries are the last q_len positions); masked_dims = (d_qk, d_v) of the per-head
    tensors when the masked form can run; union_rows = sum of union_len after dsa_union_build
    (else estimated).  Returns (form name, {form name: ms or None}, union rows used)."""
    ql = np.ascontiguousarray(q_lens, dtype=np.int32)
    kl = np.ascontiguousarray(kv_lens, dtype=np.int32)
    if ql.shape != kl.shape or ql.ndim != 1:
        raise ValueError("q_lens and kv_lens must be 1-D of the same length")
    md = (0, 0) if masked_dims is None else tuple(int(x) for x in masked_dims)
    q = FormQuery(len(ql), ql.ctypes.data_as(_I32P), kl.ctypes.data_as(_I32P), int(H), int(k), int(d_qk), md[0],
                  md[1], -1.0 if union_rows is None else float(union_rows))
    e = FormEstimate()
    _check(lib().dsa_choose_form(ctypes.byref(q), None if calibration is None else ctypes.byref(calibration),
                                 ctypes.byref(e)), "dsa_choose_form")
    ms = {name: (e.ms[i] if e.ms[i] >= 0 else None) for i, name in enumerate(FORMS)}
    return FORMS[e.form], ms, e.union_rows


def dsa_debug_wait_timeout(stream=None, device=None):
    """Queues the failure-path check: one CTA whose bounded wait runs out (about 2 s)."""
    import torch
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    _check(lib().dsa_debug_wait_timeout(_stream(stream, dev)), "dsa_debug_wait_timeout")


def dsa_last_device_error(stream=None, device=None):
    """Synchronizes the stream and returns (status, [bad_index, timeout, union_overflow, reserved]),
    clearing the device counters."""
    import torch
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    counts = (ctypes.c_uint32 * 4)()
    st = lib().dsa_last_device_error(_stream(stream, dev), counts)
    return st, [int(c) for c in counts]


def dsa_debug_trace(buffer=None, capacity: int = 0):
    """Diagnostic timeline: record per-tile clock64 stamps of CTAs 0 and 1 into
    ``buffer`` (an int64 CUDA tensor of >= 2 * capacity * 8 elements); call with
    no buffer to switch recording off."""
    if buffer is None:
        _check(lib().dsa_debug_trace(None, 0), "dsa_debug_trace")
        return
    if buffer.numel() < 2 * capacity * 8 or not buffer.is_cuda:
        raise ValueError("trace buffer too small or not on the GPU")
    _check(lib().dsa_debug_trace(buffer.data_ptr(), capacity), "dsa_debug_trace")


def dsa_sparse_prefill_fp8(q, kv_fp8, idx, k: int, scale: float, d_rope: int = 64, d_v: int = 512, out=None,
                           lse=None, stream=None):
    """Per-token sparse prefill over FP8 latent rows kv_fp8 [N, dsa_kv_fp8_row_bytes(d_rope)] uint8, read
    and dequantized inside the kernel.  q [T, H, 512 + d_rope] bf16, idx [T, ld] int32 global rows.
    Returns (out [T, H, d_v] bf16, lse [T, H] fp32), bit-equal to dsa_kv_fp8_dequantize followed by
    dsa_sparse_prefill."""
    import torch
    _need(q, torch.bfloat16, "q", 3)
    _need(kv_fp8, torch.uint8, "kv_fp8", 2)
    _need(idx, torch.int32, "idx", 2)
    T, H, d_qk = q.shape
    N, rb = kv_fp8.shape
    if rb != dsa_kv_fp8_row_bytes(d_rope):
        raise ValueError("kv_fp8 rows must be dsa_kv_fp8_row_bytes(d_rope) bytes")
    if idx.shape[0] != T:
        raise ValueError("idx rows must match q tokens")
    if out is None:
        out = _empty((T, H, d_v), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty((T, H), torch.float32, q.device, stream)
    _check(lib().dsa_sparse_prefill_fp8(q.data_ptr(), kv_fp8.data_ptr(), N, int(d_rope), idx.data_ptr(), T, H, d_qk,
                                        d_v, k, idx.shape[1], float(scale), out.data_ptr(), lse.data_ptr(),
                                        _stream(stream, q.device)), "dsa_sparse_prefill_fp8")
    return out, lse


# ---------------------------------------------------------------------------
# the decode step: calls of a few microseconds of GPU work, so the checks are
# written out flat (a call through these functions costs the host about twice
# the bare library call)
# ---------------------------------------------------------------------------
_torch = _raw_stream = _current_device = None


def _load_torch():
    global _torch, _raw_stream, _current_device
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch
    return torch


def _queue(fn, where, args, dev, stream):
    """Calls the library function on `stream` (None: the current one) with `dev` current, which a
    library call works on."""
    if stream is not None:
        stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if dev == _current_device():
        st = fn(*args, _raw_stream(dev) if stream is None else stream)
    else:
        with _torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev) if stream is None else stream)
    if st:
        raise DSAError(st, where)


def _int_tensor(t, name, ndim, dev):
    if not isinstance(t, _torch.Tensor) or t.dtype is not _torch.int32:
        raise TypeError(f"{name} must be an int32 tensor")
    if t.dim() != ndim or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor on CUDA device {dev}")


@functools.lru_cache(maxsize=64)
def _rope_table(d_rope, base, layout, scaling, factor, original_len, beta_fast, beta_slow, mscale) -> bytes:
    f = RopeFreqs()
    _check(lib().dsa_rope_freqs_init(ctypes.byref(f), int(d_rope), float(base), ROPE_LAYOUTS.index(layout),
                                     ROPE_SCALINGS.index(scaling), float(factor), int(original_len), float(beta_fast),
                                     float(beta_slow), float(mscale)), "dsa_rope_freqs_init")
    return bytes(f)


def dsa_rope_freqs(d_rope: int, base: float = 10000.0, layout: str = "interleaved", scaling: str = "none",
                   factor: float = 1.0, original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                   mscale: float = 1.0) -> RopeFreqs:
    """Rotary frequencies for dsa_rope and dsa_kv_append (host only): pairs of ``layout``
    "interleaved" (2i, 2i+1) or "half" (i, i + d_rope/2), frequencies base^(-2i/d_rope),
    ``scaling`` "none", "linear" (divided by factor) or "yarn" (fast pairs kept, slow ones
    divided, mixed between beta_fast and beta_slow turns over original_len positions); mscale
    multiplies cos and sin.  The table depends on these numbers alone (and is kept by them); every
    call returns a copy of its own."""
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {ROPE_LAYOUTS}")
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {ROPE_SCALINGS}")
    return RopeFreqs.from_buffer_copy(_rope_table(d_rope, base, layout, scaling, factor, original_len, beta_fast,
                                                  beta_slow, mscale))


def dsa_rope(x, positions, freqs: RopeFreqs, out=None, gradient: bool = False, stream=None):
    """Rotary positions on x [T, H, d_rope] (bf16 or fp32, any strides with unit last stride: the
    RoPE columns of a wider head are passed as that view), positions [T] int32.  ``out``: a tensor
    or view of the same shape and dtype, x itself for in place; a new contiguous one if None.
    gradient=True turns back: the gradient of the forward with respect to x, given the gradient
    of its result.  Returns out.  (As with every call of the library, autograd does not see this one:
    out is detached from an x that requires a gradient.)"""
    torch = _torch or _load_torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a bf16 or fp32 tensor")
    dtype = x.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("x must be a bf16 or fp32 tensor")
    dev = x.get_device()
    if dev < 0 or x.dim() != 3:
        raise ValueError("x must be a 3-D CUDA tensor")
    if not isinstance(freqs, RopeFreqs):
        raise TypeError("freqs must come from dsa_rope_freqs")
    _int_tensor(positions, "positions", 1, dev)
    shape = x.shape
    T, H, d = shape
    xs = x.stride()
    if T > 0x7fffffff or H > 0x7fffffff:   # (the library counts them in 32 bits)
        raise DSAError(DSA_ERR_UNSUPPORTED, "dsa_rope")
    if d != freqs.d_rope or positions.shape[0] != T:
        raise ValueError(f"x is {tuple(shape)}: it must have {freqs.d_rope} columns, and positions one entry per token")
    if out is None:
        out = _empty(shape, dtype, x.device, stream)
    elif out.dtype is not dtype or out.shape != shape or out.get_device() != dev:
        raise ValueError("out must have x's shape, dtype and device")
    ys = out.stride()
    if xs[2] != 1 or ys[2] != 1:
        raise ValueError("x and out must have unit stride in their last dimension")
    _queue(lib().dsa_rope, "dsa_rope",
           (x.data_ptr(), xs[0], xs[1], out.data_ptr(), ys[0], ys[1], 1 if dtype is torch.float32 else 0,
            positions.data_ptr(), T, H, freqs, 1 if gradient else 0), dev, stream)
    return out


def _cache_of(cache, d_rope, dev):
    """(format, rows, ld) of a bf16 or FP8 cache tensor."""
    if not isinstance(cache, _torch.Tensor) or cache.dim() != 2 or cache.get_device() != dev or \
            not cache.is_contiguous():
        raise ValueError("cache must be a contiguous 2-D CUDA tensor on the device of the other arguments")
    N, ld = cache.shape
    if cache.dtype is _torch.bfloat16:
        return 0, N, ld
    if cache.dtype is not _torch.uint8:
        raise TypeError("cache must be bf16 rows or FP8 rows as uint8")
    if ld != 528 + 2 * d_rope:
        raise ValueError("FP8 cache rows must be dsa_kv_fp8_row_bytes(d_rope) bytes")
    return 1, N, 0


def dsa_kv_append(c_kv, k_pe, positions, block_table, block_size: int, cache, rope: RopeFreqs = None, token_req=None,
                  stream=None):
    """New tokens' latent rows into a paged cache: token t of request r (token_req [T] int32, or
    r = t) at positions[t] (int32, -1 = padding token) goes to row block_table[r][p // block_size] *
    block_size + p % block_size.  c_kv [T, 512] and k_pe [T, d_rope] bf16 (row-strided views, k_pe
    None without RoPE columns) are stored with k_pe rotated by ``rope`` (None: as it is).  cache:
    bf16 [N, ld_kv] or FP8 rows [N, dsa_kv_fp8_row_bytes(d_rope)] uint8.  Returns cache."""
    torch = _torch or _load_torch()
    if not isinstance(c_kv, torch.Tensor) or c_kv.dtype is not torch.bfloat16:
        raise TypeError("c_kv must be a bf16 tensor")
    dev = c_kv.get_device()
    cs = c_kv.stride()
    if dev < 0 or c_kv.dim() != 2 or c_kv.shape[1] != 512 or cs[1] != 1:
        raise ValueError("c_kv must be a [T, 512] CUDA tensor with unit stride in its last dimension")
    T = c_kv.shape[0]
    d_rope = pe = ps = 0
    if k_pe is not None:
        if not isinstance(k_pe, torch.Tensor) or k_pe.dtype is not torch.bfloat16:
            raise TypeError("k_pe must be a bf16 tensor")
        if k_pe.dim() != 2 or k_pe.shape[0] != T or k_pe.get_device() != dev:
            raise ValueError("k_pe must be a [T, d_rope] tensor on c_kv's device")
        d_rope = k_pe.shape[1]
        if d_rope:
            pe = k_pe.data_ptr()
            ps, last = k_pe.stride()
            if last != 1:
                raise ValueError("k_pe must have unit stride in its last dimension")
    if rope is not None and not isinstance(rope, RopeFreqs):
        raise TypeError("rope must come from dsa_rope_freqs")
    _int_tensor(positions, "positions", 1, dev)
    _int_tensor(block_table, "block_table", 2, dev)
    if token_req is not None:
        _int_tensor(token_req, "token_req", 1, dev)
    if positions.shape[0] != T or (token_req is not None and token_req.shape[0] != T):
        raise ValueError("positions and token_req must have one entry per token")
    fmt, N, ld = _cache_of(cache, d_rope, dev)
    num_req, max_blocks = block_table.shape
    _queue(lib().dsa_kv_append, "dsa_kv_append",
           (c_kv.data_ptr(), cs[0], pe, ps, T, d_rope, positions.data_ptr(),
            None if token_req is None else token_req.data_ptr(), block_table.data_ptr(), num_req, max_blocks,
            int(block_size), rope, cache.data_ptr(), fmt, N, ld), dev, stream)
    return cache


@functools.lru_cache(maxsize=1024)
def dsa_paged_decode_workspace(B: int, H: int, max_positions: int) -> int:
    """Device workspace bytes dsa_paged_decode needs for B requests of H heads; max_positions: k with
    idx, else the block table's columns * block_size."""
    n = int(lib().dsa_paged_decode_workspace(B, H, max_positions))
    if n < 0:
        raise DSAError(DSA_ERR_UNSUPPORTED, "dsa_paged_decode_workspace")
    return n


def dsa_paged_decode(q, cache, block_table, kv_lens, block_size: int, scale: float, idx=None, k: int | None = None,
                     d_v: int = 512, out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per request over a paged latent cache.  q [B, H, d_qk] bf16 (d_qk =
    576 or 512, H <= 128), cache bf16 [N, ld_kv] or FP8 rows uint8, block_table [B, max_blocks] and
    kv_lens [B] int32 on the device.  idx [B, ld] int32 (first k columns): the token's own top-k
    positions instead of the whole context.  workspace: a CUDA uint8 tensor of
    dsa_paged_decode_workspace(...) bytes (calls sharing one must not overlap on the GPU); one per
    call if None.  Returns (out [B, H, 512] bf16, lse [B, H] fp32)."""
    torch = _torch or _load_torch()
    if not isinstance(q, torch.Tensor) or q.dtype is not torch.bfloat16:
        raise TypeError("q must be a bf16 tensor")
    dev = q.get_device()
    if dev < 0 or q.dim() != 3 or not q.is_contiguous():
        raise ValueError("q must be a contiguous 3-D CUDA tensor")
    B, H, d_qk = q.shape
    if d_qk != 576 and d_qk != 512 or d_v != 512:
        raise DSAError(DSA_ERR_UNSUPPORTED, "dsa_paged_decode")
    _int_tensor(block_table, "block_table", 2, dev)
    _int_tensor(kv_lens, "kv_lens", 1, dev)
    fmt, N, ld_kv = _cache_of(cache, d_qk - 512, dev)
    block_size = int(block_size)
    rows, max_blocks = block_table.shape
    if rows != B or kv_lens.shape[0] != B:
        raise ValueError("block_table and kv_lens must have one row per request")
    ld, idx_ptr = 0, None
    if idx is not None:
        _int_tensor(idx, "idx", 2, dev)
        rows, ld = idx.shape
        if rows != B:
            raise ValueError("idx must have one row per request")
        idx_ptr = idx.data_ptr() or kv_lens.data_ptr()   # (an empty idx has no address, and means no keys)
        k = ld if k is None else int(k)
    elif k is not None:
        raise ValueError("k without idx")
    device = q.device
    if out is None:
        out = _empty((B, H, 512), torch.bfloat16, device, stream)
    elif out.dtype is not torch.bfloat16 or out.shape != (B, H, 512) or out.get_device() != dev or \
            not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 [B, H, 512] tensor on q's device")
    if lse is None:
        lse = _empty((B, H), torch.float32, device, stream)
    elif lse.dtype is not torch.float32 or lse.shape != (B, H) or lse.get_device() != dev or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H] tensor on q's device")
    if workspace is None:
        nbytes = dsa_paged_decode_workspace(B, H, max_blocks * block_size if idx is None else k)
        workspace = _empty(nbytes, torch.uint8, device, stream)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    else:
        nbytes = workspace.numel()
    _queue(lib().dsa_paged_decode, "dsa_paged_decode",
           (q.data_ptr(), cache.data_ptr(), fmt, N, ld_kv, block_table.data_ptr(), max_blocks, block_size,
            kv_lens.data_ptr(), idx_ptr, k or 0, ld, B, H, d_qk, 512, float(scale), out.data_ptr(), lse.data_ptr(),
            workspace.data_ptr(), nbytes), dev, stream)
    return out, lse
