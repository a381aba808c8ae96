"""Python binding of the C ABI in include/fa2.h (argument marshalling only).

Every entry point forwards raw device pointers, sizes and the CUDA stream
handle to ``libfa2.so``; all compute runs in the library's sm_103a kernel.
If the library cannot be loaded the call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfa2.so")

FA2_BF16 = 0
FA2_FP16 = 1

FA2_OK = 0
FA2_ERR_INVALID_ARG = 1
FA2_ERR_UNSUPPORTED = 2
FA2_ERR_CUDA = 3
FA2_ERR_TIMEOUT = 4
FA2_ERR_BOUNDS = 5   # a device-side bounds check failed (KV cache: every build; others: debug builds)

# symbols declared in include/fa2.h
EXPORTS = ("fa2_fwd", "fa2_fwd_gqa", "fa2_fwd_ex", "fa2_fwd_fp8", "fa2_fwd_fp8_ex", "fa2_bwd", "fa2_bwd_noalloc",
           "fa2_kv4_plan", "fa2_kv4_append", "fa2_kv4_gather", "fa2_fwd_kv4", "fa2_fwd_kv4_workspace",
           "fa2_check_status", "fa2_status_string",
           "fa2_set_wait_limit_ns", "fa2_set_debug_flags", "fa2_set_tile_config", "fa2_version")

_lib = None


class FA2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where} failed: {status_string(status)}")


def load(path: str = LIB_PATH):
    """Load libfa2.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"CUDA library {path} is missing: run __graft_entry__.build() "
                          "(python -m attention_fa2_forward_03_gb300.build)")
    lib = ctypes.CDLL(path)
    p, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa2_fwd.argtypes = [p, p, p, p, p, i, i, i, i, f, i, p]
    lib.fa2_fwd.restype = i
    lib.fa2_fwd_gqa.argtypes = [p, p, p, p, p, i, i, i, i, i, f, i, p]
    lib.fa2_fwd_gqa.restype = i
    lib.fa2_fwd_ex.argtypes = [p, p, p, p, p, i, i, i, i, i, i, f, i, i, p]
    lib.fa2_fwd_ex.restype = i
    lib.fa2_fwd_fp8.argtypes = [p, p, p, p, p, p, p, p, i, i, i, i, i, f, p]
    lib.fa2_fwd_fp8.restype = i
    lib.fa2_fwd_fp8_ex.argtypes = [p, p, p, p, p, p, p, p, i, i, i, i, i, i, f, i, p]
    lib.fa2_fwd_fp8_ex.restype = i
    lib.fa2_bwd.argtypes = [p, p, p, p, p, p, p, p, p, p, i, i, i, i, i, f, i, i, p]
    lib.fa2_bwd.restype = i
    lib.fa2_bwd_noalloc.argtypes = [p, p, p, p, p, p, p, p, p, i, i, i, i, i, f, i, i, p]
    lib.fa2_bwd_noalloc.restype = i
    ll = ctypes.c_int64
    lib.fa2_kv4_plan.argtypes = [p, p, p, p, p, p, p, p, p, i, i, i, i, i, p]
    lib.fa2_kv4_plan.restype = i
    lib.fa2_kv4_append.argtypes = [p, p, p, p, p, p, i, i, i, i, ll, ll, ll, ll, ll, ll, i, i, i, p]
    lib.fa2_kv4_append.restype = i
    lib.fa2_kv4_gather.argtypes = [p, p, p, p, p, p, p, p, i, i, i, i, i, i, i, i, p]
    lib.fa2_kv4_gather.restype = i
    lib.fa2_fwd_kv4.argtypes = [p, p, p, p, p, p, p, p, p, ll, i, i, i, i, i, i, i, i, f, i, i, p]
    lib.fa2_fwd_kv4.restype = i
    lib.fa2_fwd_kv4_workspace.argtypes = [i, i, i, i, i, i, i]
    lib.fa2_fwd_kv4_workspace.restype = ll
    lib.fa2_check_status.argtypes = [p]
    lib.fa2_check_status.restype = i
    lib.fa2_status_string.argtypes = [i]
    lib.fa2_status_string.restype = ctypes.c_char_p
    lib.fa2_set_wait_limit_ns.argtypes = [ctypes.c_int64]
    lib.fa2_set_wait_limit_ns.restype = ctypes.c_int64
    lib.fa2_set_debug_flags.argtypes = [i]
    lib.fa2_set_debug_flags.restype = i
    lib.fa2_set_tile_config.argtypes = [i]
    lib.fa2_set_tile_config.restype = i
    lib.fa2_version.argtypes = []
    lib.fa2_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().fa2_status_string(int(status)).decode()


# ------------------------------------------------------------------ raw pointer API

def fa2_fwd_gqa_ptr(q, k, v, o, lse, B, H_q, H_kv, N, d, scale, dtype, stream=0) -> int:
    """fa2_fwd_gqa on raw device addresses (ints); returns the status code."""
    return load().fa2_fwd_gqa(q, k, v, o, lse, B, H_q, H_kv, N, d, float(scale), int(dtype),
                              stream or None)


def fa2_fwd_ptr(q, k, v, o, lse, B, H, N, d, scale, dtype, stream=0) -> int:
    """fa2_fwd on raw device addresses (ints); returns the status code."""
    return load().fa2_fwd(q, k, v, o, lse, B, H, N, d, float(scale), int(dtype), stream or None)


def fa2_fwd_ex_ptr(q, k, v, o, lse, B, H_q, H_kv, N_q, N_k, d, scale, causal, dtype, stream=0) -> int:
    """fa2_fwd_ex on raw device addresses (ints); returns the status code."""
    return load().fa2_fwd_ex(q, k, v, o, lse, B, H_q, H_kv, N_q, N_k, d, float(scale), int(causal),
                             int(dtype), stream or None)


def fa2_fwd_fp8_ptr(q, k, v, q_descale, k_descale, v_descale, o, lse, B, H_q, H_kv, N, d, scale,
                    stream=0) -> int:
    """fa2_fwd_fp8 on raw device addresses (ints); returns the status code."""
    return load().fa2_fwd_fp8(q, k, v, q_descale, k_descale, v_descale, o, lse, B, H_q, H_kv, N, d,
                              float(scale), stream or None)


def fa2_fwd_fp8_ex_ptr(q, k, v, q_descale, k_descale, v_descale, o, lse, B, H_q, H_kv, N_q, N_k, d, scale,
                       causal, stream=0) -> int:
    """fa2_fwd_fp8_ex on raw device addresses (ints); returns the status code."""
    return load().fa2_fwd_fp8_ex(q, k, v, q_descale, k_descale, v_descale, o, lse, B, H_q, H_kv, N_q, N_k, d,
                                 float(scale), int(causal), stream or None)


def fa2_bwd_ptr(q, k, v, o, lse, dout, dq, dk, dv, delta, B, H_q, H_kv, N, d, scale, causal, dtype,
                stream=0) -> int:
    """fa2_bwd on raw device addresses (ints); returns the status code."""
    return load().fa2_bwd(q, k, v, o, lse, dout, dq, dk, dv, delta, B, H_q, H_kv, N, d, float(scale),
                          int(causal), int(dtype), stream or None)


def fa2_bwd_noalloc_ptr(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N, d, scale, causal, dtype,
                        stream=0) -> int:
    """fa2_bwd_noalloc on raw device addresses (ints): the backward without a
    caller-provided workspace, for callers that cannot allocate device
    memory (at most 2**20 query rows). Returns the status code."""
    return load().fa2_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N, d, float(scale),
                                  int(causal), int(dtype), stream or None)


def fa2_kv4_plan_ptr(seq_lens, new_lens, block_table, free_pages, free_state, seq_lens_out, accepted, slots,
                     free_state_out, B, N, max_pages, page_size, num_pages, stream=0) -> int:
    """fa2_kv4_plan on raw device addresses (ints); returns the status code."""
    return load().fa2_kv4_plan(seq_lens, new_lens, block_table, free_pages, free_state, seq_lens_out, accepted,
                               slots, free_state_out, B, N, max_pages, page_size, num_pages, stream or None)


def fa2_kv4_append_ptr(k, v, slots, cache, k_descale, v_descale, B, H_kv, N, d, k_strides, v_strides, page_size,
                       num_pages, dtype, stream=0) -> int:
    """fa2_kv4_append on raw device addresses (ints), strides (request, head,
    token) in elements; returns the status code."""
    return load().fa2_kv4_append(k, v, slots, cache, k_descale, v_descale, B, H_kv, N, d, *k_strides, *v_strides,
                                 page_size, num_pages, int(dtype), stream or None)


def fa2_kv4_gather_ptr(cache, block_table, seq_lens, starts, k_descale, v_descale, k, v, B, H_kv, N, d, max_pages,
                       page_size, num_pages, dtype, stream=0) -> int:
    """fa2_kv4_gather on raw device addresses (ints; starts may be 0); returns the status code."""
    return load().fa2_kv4_gather(cache, block_table, seq_lens, starts or None, k_descale, v_descale, k, v, B, H_kv,
                                 N, d, max_pages, page_size, num_pages, int(dtype), stream or None)


def fa2_fwd_kv4_ptr(q, cache, block_table, seq_lens, k_descale, v_descale, o, lse, workspace, workspace_bytes, B,
                    H_q, H_kv, N_q, d, max_pages, page_size, num_pages, scale, causal, dtype, stream=0) -> int:
    """fa2_fwd_kv4 on raw device addresses (ints); returns the status code."""
    return load().fa2_fwd_kv4(q, cache, block_table, seq_lens, k_descale, v_descale, o, lse, workspace,
                              workspace_bytes, B, H_q, H_kv, N_q, d, max_pages, page_size, num_pages, float(scale),
                              int(causal), int(dtype), stream or None)


def fa2_fwd_kv4_workspace(B: int, H_q: int, H_kv: int, N_q: int, d: int, max_pages: int, page_size: int) -> int:
    """Bytes of workspace that fa2_fwd_kv4 needs for these sizes, whatever the
    lengths; -1 for sizes that it does not take."""
    return load().fa2_fwd_kv4_workspace(B, H_q, H_kv, N_q, d, max_pages, page_size)


def fa2_check_status(stream=0) -> int:
    return load().fa2_check_status(stream or None)


def fa2_set_wait_limit_ns(limit_ns: int) -> int:
    return load().fa2_set_wait_limit_ns(int(limit_ns))


def fa2_set_debug_flags(flags: int) -> int:
    return load().fa2_set_debug_flags(int(flags))


# bit 0 of fa2_set_tile_config: d = 64, equal lengths, on the 16-bit kernel's d = 64 path
TILE_CFG_D64_SHARED = 1


def fa2_set_tile_config(config: int) -> int:
    """Planner choice for d = 64 with equal lengths (see include/fa2.h);
    returns the previous value, -1 if `config` was rejected."""
    return load().fa2_set_tile_config(int(config))


def fa2_version() -> str:
    return load().fa2_version().decode()


# ------------------------------------------------------------------ torch tensors

def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return FA2_BF16
    if t.dtype == torch.float16:
        return FA2_FP16
    raise TypeError(f"q/k/v must be bf16 or fp16, got {t.dtype}")


def _stream_handle(stream, device) -> int:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def fa2_fwd_gqa(q, k, v, o=None, lse=None, scale=None, stream=None):
    """Attention forward on CUDA tensors q [B,Hq,N,d], k/v [B,Hkv,N,d].

    Allocates o / lse with torch when they are not given (that is device-memory
    plumbing; the library itself allocates nothing). Returns (o, lse).
    """
    import torch

    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, H, N, d]")
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (B, Hkv, N, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, Hkv, N, d] with q's B, N and d")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k and v must share one dtype")
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k and v must be contiguous CUDA tensors")
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    if o.shape != q.shape or o.dtype != q.dtype or not o.is_contiguous():
        raise ValueError("o must be a contiguous tensor like q")
    if tuple(lse.shape) != (B, Hq, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [B, Hq, N]")
    if scale is None:
        scale = d ** -0.5
    rc = fa2_fwd_gqa_ptr(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                         B, Hq, Hkv, N, d, scale, _dtype_code(q), _stream_handle(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_gqa")
    return o, lse


def fa2_fwd_ex(q, k, v, o=None, lse=None, scale=None, causal=False, stream=None):
    """General attention forward: q [B,Hq,Nq,d], k/v [B,Hkv,Nk,d], any Nq, Nk,
    optional causal mask (end-aligned). Returns (o, lse)."""
    import torch

    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, H, N, d]")
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Hkv, Nk, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, Hkv, Nk, d] with q's B and d")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k and v must share one dtype")
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k and v must be contiguous CUDA tensors")
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    if o.shape != q.shape or o.dtype != q.dtype or not o.is_contiguous():
        raise ValueError("o must be a contiguous tensor like q")
    if tuple(lse.shape) != (B, Hq, Nq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [B, Hq, Nq]")
    if scale is None:
        scale = d ** -0.5
    rc = fa2_fwd_ex_ptr(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                        B, Hq, Hkv, Nq, Nk, d, scale, bool(causal), _dtype_code(q),
                        _stream_handle(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_ex")
    return o, lse


def fa2_bwd(q, k, v, o, lse, dout, scale=None, causal=False, dq=None, dk=None, dv=None, delta=None,
            stream=None):
    """Gradients (dq, dk, dv) of the forward for upstream gradient dout.

    q, o, dout: [B, Hq, N, d]; k, v: [B, Hkv, N, d]; lse: fp32 [B, Hq, N]
    from the forward. Outputs and the fp32 workspace `delta` [B, Hq, N] are
    allocated with torch when not given (device-memory plumbing only).
    """
    import torch

    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    for t in (q, k, v, o, dout, lse):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if tuple(k.shape) != (B, Hkv, N, d) or v.shape != k.shape or o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("shape mismatch")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    delta = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if delta is None else delta
    if scale is None:
        scale = d ** -0.5
    rc = fa2_bwd_ptr(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                     dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), delta.data_ptr(), B, Hq, Hkv, N, d, scale,
                     bool(causal), _dtype_code(q), _stream_handle(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_bwd")
    return dq, dk, dv


def _fp8_prepare(q, k, v, q_descale, k_descale, v_descale, o, lse, same_len):
    """Check the FP8 arguments and allocate missing outputs; returns
    (o, lse, B, Hq, Hkv, Nq, Nk, d)."""
    import torch

    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, H, N, d]")
    B, Hq, N, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if same_len and Nk != N:
        raise ValueError("k and v must be [B, Hkv, N, d] with q's B, N and d")
    if tuple(k.shape) != (B, Hkv, Nk, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, Nk, d] with q's B and d")
    for t in (q, k, v):
        if t.element_size() != 1 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k and v must be contiguous one-byte (e4m3) CUDA tensors")
    for t in (q_descale, k_descale, v_descale):
        if t.dtype != torch.float32 or not t.is_cuda or t.numel() != B * Hkv or not t.is_contiguous():
            raise ValueError("descales must be contiguous fp32 CUDA tensors of B*Hkv elements")
    if o is None:
        o = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    if tuple(o.shape) != (B, Hq, N, d) or o.dtype != torch.bfloat16 or not o.is_contiguous():
        raise ValueError("o must be a contiguous bf16 tensor [B, Hq, N, d]")
    if tuple(lse.shape) != (B, Hq, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [B, Hq, N]")
    return o, lse, B, Hq, Hkv, N, Nk, d


def fa2_fwd_fp8(q, k, v, q_descale, k_descale, v_descale, o=None, lse=None, scale=None, stream=None):
    """FP8 attention forward: q [B,Hq,N,d], k/v [B,Hkv,N,d] e4m3 codes as
    uint8 (or torch.float8_e4m3fn) CUDA tensors, descales fp32 [B*Hkv] CUDA
    tensors. Returns (o, lse) with o bf16 [B,Hq,N,d] and lse fp32 [B,Hq,N]."""
    o, lse, B, Hq, Hkv, N, _, d = _fp8_prepare(q, k, v, q_descale, k_descale, v_descale, o, lse, True)
    if scale is None:
        scale = d ** -0.5
    rc = fa2_fwd_fp8_ptr(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_descale.data_ptr(), k_descale.data_ptr(),
                         v_descale.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, N, d, scale,
                         _stream_handle(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_fp8")
    return o, lse


def fa2_fwd_fp8_ex(q, k, v, q_descale, k_descale, v_descale, o=None, lse=None, scale=None, causal=False,
                   stream=None):
    """General FP8 attention forward: q [B,Hq,Nq,d], k/v [B,Hkv,Nk,d] e4m3
    codes, any Nq, Nk, optional causal mask (end-aligned). Returns (o, lse)
    with o bf16 [B,Hq,Nq,d] and lse fp32 [B,Hq,Nq]."""
    o, lse, B, Hq, Hkv, Nq, Nk, d = _fp8_prepare(q, k, v, q_descale, k_descale, v_descale, o, lse, False)
    if scale is None:
        scale = d ** -0.5
    rc = fa2_fwd_fp8_ex_ptr(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_descale.data_ptr(), k_descale.data_ptr(),
                            v_descale.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Nq, Nk, d, scale,
                            bool(causal), _stream_handle(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_fp8_ex")
    return o, lse


def fa2_fwd(q, k, v, o=None, lse=None, scale=None, stream=None):
    """Multi-head attention forward: q, k, v all [B, H, N, d]. Returns (o, lse)."""
    if q.shape[1] != k.shape[1]:
        raise ValueError("fa2_fwd needs equal head counts; use fa2_fwd_gqa")
    return fa2_fwd_gqa(q, k, v, o, lse, scale, stream)


# ------------------------------------------------------------------ the paged 4-bit KV cache

def fa2_kv4_cache_shape(num_pages: int, H_kv: int, page_size: int, d: int) -> tuple:
    """Shape of the uint8 cache tensor (layout: include/fa2.h)."""
    return (num_pages, H_kv, 2, page_size * (d // 2 + d // 16))


# These wrappers run once a layer and decoding step, so each checks its
# arguments in one pass of cheap comparisons; the helpers below find out what
# is wrong once that pass has failed.

def _kv4_call(fn, index, stream, *args):
    """Runs a C entry point with device `index` current (the library launches
    on the current device) on `stream` (None: that device's current stream)."""
    import torch

    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return fn(*args, int(stream))
    return fn(*args, stream)


def _kv4_same_device(index, **tensors):
    for name, t in tensors.items():
        if t.get_device() != index or index < 0:
            raise ValueError(f"all tensors must be on one CUDA device, {name} is on {t.device}")


def _kv4_ints(name, t, shape):
    import torch

    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)}, got {t.dtype} {list(t.shape)}")


def _kv4_refuse_cache(index, cache, k_descale, v_descale, H_kv, d, what):
    """Says what is wrong with a cache or its descales (or, if nothing is,
    with `what`)."""
    import torch

    _kv4_same_device(index, cache=cache, k_descale=k_descale, v_descale=v_descale)
    token = max(1, d // 2 + d // 16)
    if (cache.dtype != torch.uint8 or cache.dim() != 4 or not cache.is_contiguous()
            or cache.shape[1] != H_kv or cache.shape[2] != 2 or cache.shape[3] == 0 or cache.shape[3] % token):
        raise ValueError("cache must be a contiguous uint8 CUDA tensor [num_pages, H_kv, 2, page_size*(d/2+d/16)]")
    for t in (k_descale, v_descale):
        if t.dtype != torch.float32 or t.shape != (H_kv,) or not t.is_contiguous():
            raise ValueError("descales must be contiguous fp32 CUDA tensors [H_kv]")
    raise ValueError(what)


def fa2_kv4_plan(seq_lens, new_lens, block_table, free_pages, free_state, page_size, N, seq_lens_out=None,
                 accepted=None, slots=None, free_state_out=None, stream=None):
    """Pages and slots of one scheduling step (include/fa2.h).

    seq_lens, new_lens [B], block_table [B, max_pages] (updated), free_pages
    [num_pages] (a ring, updated), free_state [2]: int32 CUDA tensors; N: the
    most tokens a request may add. seq_lens_out and free_state_out may be
    seq_lens and free_state themselves. Returns (seq_lens_out [B],
    accepted [B], slots [B, N], free_state_out [2])."""
    import torch

    if seq_lens.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("seq_lens must be [B], block_table [B, max_pages], free_pages [num_pages]")
    B, W = block_table.shape
    dev, index = seq_lens.device, seq_lens.get_device()
    if seq_lens_out is None:
        seq_lens_out = torch.empty_like(seq_lens)
    if accepted is None:
        accepted = torch.empty_like(seq_lens)
    if slots is None:
        slots = torch.empty((B, N), dtype=torch.int32, device=dev)
    if free_state_out is None:
        free_state_out = torch.empty_like(free_state)
    i32, row, two = torch.int32, (B,), (2,)
    for t, shape in ((seq_lens, row), (new_lens, row), (block_table, (B, W)), (free_pages, None), (free_state, two),
                     (seq_lens_out, row), (accepted, row), (slots, (B, N)), (free_state_out, two)):
        if (t.dtype is not i32 or t.get_device() != index or not t.is_contiguous() or index < 0
                or (shape is not None and t.shape != shape)):
            tensors = {"seq_lens": seq_lens, "new_lens": new_lens, "block_table": block_table,
                       "free_pages": free_pages, "free_state": free_state, "seq_lens_out": seq_lens_out,
                       "accepted": accepted, "slots": slots, "free_state_out": free_state_out}
            _kv4_same_device(index, **tensors)
            for name, x in tensors.items():
                _kv4_ints(name, x, {"block_table": (B, W), "free_pages": x.shape, "free_state": two, "slots": (B, N),
                                    "free_state_out": two}.get(name, row))
    rc = _kv4_call(load().fa2_kv4_plan, index, stream, seq_lens.data_ptr(), new_lens.data_ptr(),
                   block_table.data_ptr(), free_pages.data_ptr(), free_state.data_ptr(), seq_lens_out.data_ptr(),
                   accepted.data_ptr(), slots.data_ptr(), free_state_out.data_ptr(), B, N, W, page_size,
                   free_pages.shape[0])
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_kv4_plan")
    return seq_lens_out, accepted, slots, free_state_out


def fa2_kv4_append(k, v, slots, cache, k_descale, v_descale, stream=None):
    """Quantises k, v [B, Hkv, N, d] (any strides that are multiples of 8
    elements, rows of adjacent elements) into the slots [B, N] of the cache;
    negative slots are skipped. Returns the cache."""
    import torch

    if k.dim() != 4 or k.shape != v.shape or cache.dim() != 4:
        raise ValueError("k and v must be 4-D [B, H_kv, N, d] of one shape, cache 4-D")
    B, Hkv, N, d = k.shape
    num_pages, heads, two, size = cache.shape
    index, token = k.get_device(), (d // 2 + d // 16) or 1
    if k.dtype != v.dtype:
        raise TypeError("k and v must share one dtype")
    (kb, kh, kn, ke), (vb, vh, vn, ve) = k.stride(), v.stride()
    if not (index >= 0 and v.get_device() == index and slots.get_device() == index and cache.get_device() == index
            and k_descale.get_device() == index and v_descale.get_device() == index and ke == 1 and ve == 1
            and heads == Hkv and two == 2 and size % token == 0 and cache.dtype is torch.uint8
            and slots.dtype is torch.int32 and k_descale.dtype is torch.float32 and v_descale.dtype is torch.float32
            and slots.shape == (B, N) and k_descale.shape == (Hkv,) and v_descale.shape == (Hkv,)
            and cache.is_contiguous() and slots.is_contiguous() and k_descale.is_contiguous()
            and v_descale.is_contiguous()):
        _kv4_same_device(index, k=k, v=v, slots=slots)
        _kv4_ints("slots", slots, (B, N))
        _kv4_refuse_cache(index, cache, k_descale, v_descale, Hkv, d, "the rows of k and v must be adjacent elements")
    # the stride of an axis of length 1 is never used and may be anything
    if B == 1:
        kb = vb = 0
    if Hkv == 1:
        kh = vh = 0
    if N == 1:
        kn = vn = 0
    rc = _kv4_call(load().fa2_kv4_append, index, stream, k.data_ptr(), v.data_ptr(), slots.data_ptr(),
                   cache.data_ptr(), k_descale.data_ptr(), v_descale.data_ptr(), B, Hkv, N, d, kb, kh, kn, vb, vh, vn,
                   size // token, num_pages, _dtype_code(k))
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_kv4_append")
    return cache


def fa2_kv4_gather(cache, block_table, seq_lens, k_descale, v_descale, N, d, starts=None, dtype=None, k=None, v=None,
                   stream=None):
    """Reads cached tokens back: k, v [B, Hkv, N, d] of `dtype` (bf16 by
    default, or k's), row i of request b its position starts[b] + i (starts
    None: i); rows at or past seq_lens[b] are zeros. Returns (k, v)."""
    import torch

    if block_table.dim() != 2 or cache.dim() != 4:
        raise ValueError("block_table must be [B, max_pages], cache [num_pages, H_kv, 2, page_size*(d/2+d/16)]")
    B, W = block_table.shape
    num_pages, Hkv, two, size = cache.shape
    index, token = cache.get_device(), (d // 2 + d // 16) or 1
    if not (index >= 0 and block_table.get_device() == index and seq_lens.get_device() == index
            and k_descale.get_device() == index and v_descale.get_device() == index and two == 2
            and size % token == 0 and cache.dtype is torch.uint8 and block_table.dtype is torch.int32
            and seq_lens.dtype is torch.int32 and k_descale.dtype is torch.float32
            and v_descale.dtype is torch.float32 and seq_lens.shape == (B,) and k_descale.shape == (Hkv,)
            and v_descale.shape == (Hkv,) and cache.is_contiguous() and block_table.is_contiguous()
            and seq_lens.is_contiguous() and k_descale.is_contiguous() and v_descale.is_contiguous()
            and (starts is None or (starts.get_device() == index and starts.dtype is torch.int32
                                    and starts.shape == (B,) and starts.is_contiguous()))):
        _kv4_same_device(index, block_table=block_table, seq_lens=seq_lens)
        _kv4_ints("block_table", block_table, (B, W))
        _kv4_ints("seq_lens", seq_lens, (B,))
        _kv4_refuse_cache(index, cache, k_descale, v_descale, Hkv, d,
                          "starts must be a contiguous int32 CUDA tensor [B] on the cache's device")
    if dtype is None:
        dtype = torch.bfloat16 if k is None else k.dtype
    shape = (B, Hkv, N, d)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=cache.device)
    elif k.shape != shape or k.dtype != dtype or k.get_device() != index or not k.is_contiguous():
        raise ValueError("k must be a contiguous tensor [B, H_kv, N, d] of `dtype` on the cache's device")
    if v is None:
        v = torch.empty_like(k)
    elif v.shape != shape or v.dtype != dtype or v.get_device() != index or not v.is_contiguous():
        raise ValueError("v must be a contiguous tensor [B, H_kv, N, d] of `dtype` on the cache's device")
    rc = _kv4_call(load().fa2_kv4_gather, index, stream, cache.data_ptr(), block_table.data_ptr(),
                   seq_lens.data_ptr(), None if starts is None else starts.data_ptr(), k_descale.data_ptr(),
                   v_descale.data_ptr(), k.data_ptr(), v.data_ptr(), B, Hkv, N, d, W, size // token, num_pages,
                   _dtype_code(k))
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_kv4_gather")
    return k, v


def fa2_fwd_kv4(q, cache, block_table, seq_lens, k_descale, v_descale, o=None, lse=None, workspace=None, scale=None,
                causal=False, stream=None):
    """Attention of the newest N_q tokens of each request, q [B, Hq, Nq, d],
    over its seq_lens[b] cached tokens. `workspace`: a uint8 CUDA tensor of
    fa2_fwd_kv4_workspace(...) bytes that no other call in flight uses;
    allocated with torch when not given, as o and lse are. Returns
    (o [B, Hq, Nq, d], lse fp32 [B, Hq, Nq])."""
    import torch

    if q.dim() != 4 or cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q must be [B, H_q, N_q, d], cache 4-D and block_table [B, max_pages]")
    B, Hq, Nq, d = q.shape
    num_pages, Hkv, two, size = cache.shape
    rows, W = block_table.shape
    index, token = q.get_device(), (d // 2 + d // 16) or 1
    if not (index >= 0 and cache.get_device() == index and block_table.get_device() == index
            and seq_lens.get_device() == index and k_descale.get_device() == index and v_descale.get_device() == index
            and rows == B and two == 2 and size % token == 0 and cache.dtype is torch.uint8
            and block_table.dtype is torch.int32 and seq_lens.dtype is torch.int32
            and k_descale.dtype is torch.float32 and v_descale.dtype is torch.float32 and seq_lens.shape == (B,)
            and k_descale.shape == (Hkv,) and v_descale.shape == (Hkv,) and q.is_contiguous()
            and cache.is_contiguous() and block_table.is_contiguous() and seq_lens.is_contiguous()
            and k_descale.is_contiguous() and v_descale.is_contiguous()):
        _kv4_same_device(index, q=q, block_table=block_table, seq_lens=seq_lens)
        _kv4_ints("block_table", block_table, (B, W))
        _kv4_ints("seq_lens", seq_lens, (B,))
        _kv4_refuse_cache(index, cache, k_descale, v_descale, Hkv, d, "q must be contiguous")
    page_size = size // token
    if o is None:
        o = torch.empty_like(q)
    elif o.shape != q.shape or o.dtype != q.dtype or o.get_device() != index or not o.is_contiguous():
        raise ValueError("o must be a contiguous tensor like q")
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    elif (lse.shape != (B, Hq, Nq) or lse.dtype != torch.float32 or lse.get_device() != index
          or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 tensor [B, H_q, N_q] on q's device")
    lib = load()
    if workspace is None:
        nbytes = max(lib.fa2_fwd_kv4_workspace(B, Hq, Hkv, Nq, d, W, page_size), 16)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        if stream is not None:   # freed below while `stream` may still use it
            workspace.record_stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    else:
        nbytes = workspace.numel() * workspace.element_size()
    rc = _kv4_call(lib.fa2_fwd_kv4, index, stream, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(),
                   seq_lens.data_ptr(), k_descale.data_ptr(), v_descale.data_ptr(), o.data_ptr(), lse.data_ptr(),
                   workspace.data_ptr(), nbytes, B, Hq, Hkv, Nq, d, W, page_size, num_pages,
                   d ** -0.5 if scale is None else scale, 1 if causal else 0, _dtype_code(q))
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_kv4")
    return o, lse
