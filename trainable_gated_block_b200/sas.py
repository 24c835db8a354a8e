"""ctypes binding of libsas.so (C ABI in include/sas.h).

Argument marshalling only: shapes are read off torch tensors, outputs and
workspaces are allocated with torch on the input's device, and every call
goes straight to the library on torch's current CUDA stream. There is no
fallback: if libsas.so is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsas.so")

SAS_OK, SAS_ERR_INVALID_ARG, SAS_ERR_UNSUPPORTED, SAS_ERR_CUDA, SAS_ERR_TIMEOUT = 0, 1, 2, 3, 4
SAS_F32, SAS_BF16 = 0, 1

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_Z = ctypes.c_size_t
_L = ctypes.c_int64

# name -> (restype, argtypes); must match include/sas.h
SIGNATURES = {
    "sas_last_error": (ctypes.c_char_p, []),
    "sas_kernel_launches": (ctypes.c_uint64, []),
    "sas_get_error_flag": (_I, [_P]),
    "sas_select": (_I, [_P, _I, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P]),
    "sas_select_varlen": (_I, [_P, _I, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P]),
    "sas_attn_fwd": (_I, [_I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _F, _P, _P, _P]),
    "sas_attn_fwd_varlen": (_I, [_I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _F, _P, _P, _P]),
    "sas_attn_bwd_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I]),
    "sas_attn_bwd_varlen_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "sas_attn_bwd": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P,
                          _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P, _Z, _P]),
    "sas_attn_bwd_varlen": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P,
                                 _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P, _Z, _P]),
    "sas_score_select_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "sas_score_select": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "sas_pool_pages": (_I, [_P, _I, _I, _I, _I, _P, _I, _P, _P]),
    "sas_score_select_decode": (_I, [_P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I, _P, _I, _I, _P, _I,
                                     _P, _P, _P, _P, _P]),
    "sas_decode_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "sas_decode_paged": (_I, [_P, _P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                              _P, _P, _P, _F, _P, _P, _P, _Z, _P]),
    "sas_decode_paged_noalloc": (_I, [_P, _P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                                      _P, _P, _P, _F, _P, _P, _P]),
    "sas_decode_q8_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "sas_decode_paged_q8": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                                 _P, _P, _P, _F, _P, _P, _P, _Z, _P]),
    "sas_qk_norm_rope": (_I, [_I, _P, _L, _P, _L, _P, _P, _P, _I, _P, _I, _L, _I, _I, _I, _F, _P, _P, _P]),
    "sas_qk_norm_rope_bwd_workspace_size": (_Z, [_L, _I, _I, _I]),
    "sas_qk_norm_rope_bwd": (_I, [_I, _P, _P, _P, _L, _P, _L, _P, _P, _P, _I, _P, _I, _L, _I, _I, _I, _F,
                                  _P, _P, _P, _P, _P, _Z, _P]),
    "sas_append_paged": (_I, [_P, _L, _P, _L, _P, _L, _P, _P, _P, _I, _P, _I, _I, _L, _P, _P, _I, _I, _I, _I, _I,
                              _I, _F, _P, _P, _P, _P, _P, _P]),
    "sas_append_paged_q8": (_I, [_P, _L, _P, _L, _P, _L, _P, _P, _P, _I, _P, _I, _I, _L, _P, _P, _I, _I, _I, _I, _I,
                                 _I, _F, _P, _P, _P, _P, _P, _P, _P, _P]),
    "sas_selftest_bounded_wait": (_I, [_P]),
}


class SasError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libsas status {code}: {msg}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load libsas.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m trainable_gated_block_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


def _check(code: int):
    if code != SAS_OK:
        raise SasError(code, lib().sas_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SAS_BF16
    if t.dtype == torch.float32:
        return SAS_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def kernel_launches() -> int:
    """Kernels libsas.so has enqueued in this process so far."""
    return int(lib().sas_kernel_launches())


def get_error_flag(stream=None):
    """Synchronise the stream and raise if a kernel flagged bad data or a timeout."""
    _check(lib().sas_get_error_flag(_stream(stream)))


def selftest_bounded_wait(stream=None):
    """Enqueue the library's bounded-wait fault injection: a kernel whose wait can never
    complete gives up after its budget (about 2 s) and the next get_error_flag raises
    SasError with SAS_ERR_TIMEOUT."""
    _check(lib().sas_selftest_bounded_wait(_stream(stream)))


def select(s, K: int, kv_len=None, block_size: int = 64):
    """Top-K + log-gates. Prefill: s [B,Hkv,NQB,ld]. Decode: s [N,Hkv,ld], kv_len [N].

    Returns idx, cnt, log_gate, lse_s shaped [B,Hkv,R,K], [B,Hkv,R], [B,Hkv,R,K],
    [B,Hkv,R] (decode: R dimension dropped).
    """
    decode = kv_len is not None
    s4 = s[:, :, None, :] if decode else s
    _contig(s4, kv_len)
    B, H, R, ld = s4.shape
    dev = s.device
    idx = torch.empty((B, H, R, K), dtype=torch.int32, device=dev)
    cnt = torch.empty((B, H, R), dtype=torch.int32, device=dev)
    lg = torch.empty((B, H, R, K), dtype=torch.float32, device=dev)
    lse_s = torch.empty((B, H, R), dtype=torch.float32, device=dev)
    _check(lib().sas_select(_ptr(s4), B, H, R, ld, _ptr(kv_len), block_size, K,
                            _ptr(idx), _ptr(cnt), _ptr(lg), _ptr(lse_s), _stream()))
    if decode:
        return idx[:, :, 0], cnt[:, :, 0], lg[:, :, 0], lse_s[:, :, 0]
    return idx, cnt, lg, lse_s


def select_varlen(s, K: int, cu_seqlens, block_size: int = 64):
    """Top-K + log-gates for a packed batch: s [B,Hkv,R,ld] (R >= blocks of the longest
    sequence), cu_seqlens int32 [B+1] on the device. Padding rows come back empty."""
    _contig(s, cu_seqlens)
    B, H, R, ld = s.shape
    dev = s.device
    idx = torch.empty((B, H, R, K), dtype=torch.int32, device=dev)
    cnt = torch.empty((B, H, R), dtype=torch.int32, device=dev)
    lg = torch.empty((B, H, R, K), dtype=torch.float32, device=dev)
    lse_s = torch.empty((B, H, R), dtype=torch.float32, device=dev)
    _check(lib().sas_select_varlen(_ptr(s), B, H, R, ld, _ptr(cu_seqlens), block_size, K,
                                   _ptr(idx), _ptr(cnt), _ptr(lg), _ptr(lse_s), _stream()))
    return idx, cnt, lg, lse_s


def score_select(q, k, K: int, noise=None, block_size: int = 64, workspace=None, s_out=None):
    """Stand-in selector scores (block-pooled q . k / sqrt(D) + noise), then Top-K and
    log-gates, in one call. q [B,S,Hq,D], k [B,S,Hkv,D] bf16; noise [B,Hkv,NQB,ld] fp32 or None.
    Returns s [B,Hkv,NQB,NQB] (entries j >= i are whatever s_out held, zero when it is
    allocated here), idx, cnt, log_gate, lse_s."""
    _contig(q, k, noise)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    NQB = S // block_size
    dev = q.device
    if s_out is None:
        s_out = torch.zeros((B, Hkv, NQB, NQB), dtype=torch.float32, device=dev)
    need = int(lib().sas_score_select_workspace_size(B, S, Hq, Hkv, D))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    idx = torch.empty((B, Hkv, NQB, K), dtype=torch.int32, device=dev)
    cnt = torch.empty((B, Hkv, NQB), dtype=torch.int32, device=dev)
    lg = torch.empty((B, Hkv, NQB, K), dtype=torch.float32, device=dev)
    lse_s = torch.empty((B, Hkv, NQB), dtype=torch.float32, device=dev)
    ld_noise = 0 if noise is None else noise.shape[-1]
    _check(lib().sas_score_select(_ptr(q), _ptr(k), _ptr(noise), ld_noise, B, S, Hq, Hkv, D, block_size, K,
                                  _ptr(s_out), s_out.shape[-1], _ptr(idx), _ptr(cnt), _ptr(lg), _ptr(lse_s),
                                  _ptr(workspace), workspace.numel(), _stream()))
    return s_out, idx, cnt, lg, lse_s


def attn_fwd(q, k, v, idx, cnt, log_gate, sm_scale=None, block_size: int = 64):
    """Gated block-sparse causal attention forward. Returns o [B,S,Hq,D], lse [B,Hq,S]."""
    _contig(q, k, v, idx, cnt, log_gate)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    K = idx.shape[-1]
    sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    _check(lib().sas_attn_fwd(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), B, S, Hq, Hkv, D, block_size, K,
                              _ptr(idx), _ptr(cnt), _ptr(log_gate), sm_scale, _ptr(o), _ptr(lse), _stream()))
    return o, lse


def attn_fwd_varlen(q, k, v, cu_seqlens, max_seqlen: int, idx, cnt, log_gate, sm_scale=None,
                    block_size: int = 64):
    """Forward for a packed batch: q [T,Hq,D], k/v [T,Hkv,D]. Returns o [T,Hq,D] and
    lse [B,Hq,max_seqlen] (entries past a sequence's end are left unwritten)."""
    _contig(q, k, v, cu_seqlens, idx, cnt, log_gate)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.shape[0] - 1
    K = idx.shape[-1]
    sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, max_seqlen), dtype=torch.float32, device=q.device)
    _check(lib().sas_attn_fwd_varlen(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), B, max_seqlen,
                                     T, Hq, Hkv, D, block_size, K, _ptr(idx), _ptr(cnt), _ptr(log_gate),
                                     sm_scale, _ptr(o), _ptr(lse), _stream()))
    return o, lse


def bwd_workspace_bytes(q, k, K: int) -> int:
    B, S, Hq, D = q.shape
    return int(lib().sas_attn_bwd_workspace_size(_dtype_code(q), B, S, Hq, k.shape[2], D, K))


def attn_bwd(q, k, v, o, do, lse, s, lse_s, idx, cnt, log_gate, sm_scale=None, block_size: int = 64,
             workspace=None):
    """Backward. Returns dq, dk, dv (input dtype) and ds fp32 [B,Hkv,NQB,ld_s]."""
    _contig(q, k, v, o, do, lse, s, lse_s, idx, cnt, log_gate)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    K = idx.shape[-1]
    ld_s = s.shape[-1]
    sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    need = bwd_workspace_bytes(q, k, K)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    ds = torch.empty(s.shape, dtype=torch.float32, device=q.device)
    _check(lib().sas_attn_bwd(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                              _ptr(s), ld_s, _ptr(lse_s), _ptr(idx), _ptr(cnt), _ptr(log_gate),
                              B, S, Hq, Hkv, D, block_size, K, sm_scale,
                              _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ds), _ptr(workspace), workspace.numel(),
                              _stream()))
    return dq, dk, dv, ds


def attn_bwd_varlen(q, k, v, o, do, lse, s, lse_s, idx, cnt, log_gate, cu_seqlens, max_seqlen: int,
                    sm_scale=None, block_size: int = 64, workspace=None):
    """Backward for a packed batch. Returns dq [T,Hq,D], dk, dv [T,Hkv,D] (rows of no
    sequence left unwritten) and ds fp32 shaped like s (padding rows zero)."""
    _contig(q, k, v, o, do, lse, s, lse_s, idx, cnt, log_gate, cu_seqlens)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.shape[0] - 1
    K = idx.shape[-1]
    ld_s = s.shape[-1]
    sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    need = int(lib().sas_attn_bwd_varlen_workspace_size(_dtype_code(q), B, max_seqlen, T, Hq, Hkv, D, K))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    ds = torch.empty(s.shape, dtype=torch.float32, device=q.device)
    _check(lib().sas_attn_bwd_varlen(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                                     _ptr(s), ld_s, _ptr(lse_s), _ptr(idx), _ptr(cnt), _ptr(log_gate),
                                     _ptr(cu_seqlens), B, max_seqlen, T, Hq, Hkv, D, block_size, K, sm_scale,
                                     _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ds), _ptr(workspace), workspace.numel(),
                                     _stream()))
    return dq, dk, dv, ds


def pool_pages(k_cache, pages=None, kpool=None, page_size: int = 64):
    """Pooled-key cache kpool [P,Hkv,D] fp32: the mean key of each (page, KV head) of
    k_cache [P,Hkv,64,D]; only `pages` (int32 ids) when given."""
    _contig(k_cache, pages, kpool)
    P, Hkv, _, D = k_cache.shape
    if kpool is None:
        kpool = torch.zeros((P, Hkv, D), dtype=torch.float32, device=k_cache.device)
    n = 0 if pages is None else pages.numel()
    _check(lib().sas_pool_pages(_ptr(k_cache), P, Hkv, D, page_size, _ptr(pages), n, _ptr(kpool), _stream()))
    return kpool


def score_select_decode(q, kpool, page_table, kv_len, K: int, ld_s: int, noise=None, page_size: int = 64):
    """Decode stand-in scores from the pooled-key cache, then Top-K + log-gates.
    Returns s [N,Hkv,ld_s], idx [N,Hkv,K], cnt [N,Hkv], log_gate [N,Hkv,K], lse_s [N,Hkv]."""
    _contig(q, kpool, page_table, kv_len, noise)
    N, Hq, D = q.shape
    P, Hkv = kpool.shape[0], kpool.shape[1]
    dev = q.device
    s = torch.zeros((N, Hkv, ld_s), dtype=torch.float32, device=dev)
    idx = torch.empty((N, Hkv, K), dtype=torch.int32, device=dev)
    cnt = torch.empty((N, Hkv), dtype=torch.int32, device=dev)
    lg = torch.empty((N, Hkv, K), dtype=torch.float32, device=dev)
    lse_s = torch.empty((N, Hkv), dtype=torch.float32, device=dev)
    ld_noise = 0 if noise is None else noise.shape[-1]
    _check(lib().sas_score_select_decode(_ptr(q), _ptr(kpool), P, _ptr(page_table), page_table.shape[1],
                                         _ptr(kv_len), N, Hq, Hkv, D, page_size, _ptr(noise), ld_noise, K,
                                         _ptr(s), ld_s, _ptr(idx), _ptr(cnt), _ptr(lg), _ptr(lse_s), _stream()))
    return s, idx, cnt, lg, lse_s


def decode_workspace_bytes(N: int, Hq: int, Hkv: int, D: int, K: int) -> int:
    return int(lib().sas_decode_workspace_size(N, Hq, Hkv, D, K))


def decode_paged(q, k_cache, v_cache, page_table, kv_len, idx, cnt, log_gate, sm_scale=None,
                 page_size: int = 64, workspace=None, with_lse: bool = True):
    """Paged decode. q [N,Hq,D]; caches [P,Hkv,64,D]; kv_len 0 is a padding entry (o 0, lse -inf).
    Returns o [N,Hq,D] and lse [N,Hq] (or None)."""
    _contig(q, k_cache, v_cache, page_table, kv_len, idx, cnt, log_gate)
    N, Hq, D = q.shape
    P, Hkv = k_cache.shape[0], k_cache.shape[1]
    K = idx.shape[-1]
    sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    need = decode_workspace_bytes(N, Hq, Hkv, D, K)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((N, Hq), dtype=torch.float32, device=q.device) if with_lse else None
    _check(lib().sas_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), P, _ptr(page_table),
                                  page_table.shape[1], _ptr(kv_len), N, Hq, Hkv, D, page_size, K,
                                  _ptr(idx), _ptr(cnt), _ptr(log_gate), sm_scale, _ptr(o), _ptr(lse),
                                  _ptr(workspace), workspace.numel(), _stream()))
    return o, lse


def decode_q8_workspace_bytes(N: int, Hq: int, Hkv: int, D: int, K: int) -> int:
    """Workspace of decode_paged_q8 for exactly these sizes (fewer sequences may need more than many)."""
    return int(lib().sas_decode_q8_workspace_size(N, Hq, Hkv, D, K))


_BF16, _F32T, _I32, _F8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _raw_stream(dev: int) -> int:
    """torch's current stream on a device, without building a Stream object around it."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _expect(name, t, dtype, shape, dev) -> int:
    """Address of a contiguous tensor of this dtype, shape and device; raises on any other."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on the device of the other tensors")


def _expect_rows(name, t, dtype, shape, dev) -> int:
    """Token stride of [T,H,D] or [B,S,H,D] rows whose heads are contiguous within a token."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors")
    return _token_stride(name, t, shape)


def _token_stride(name, t, shape) -> int:
    if len(shape) == 3:
        T, H, D = shape
        st, head, one = t.stride()
        ld = st if T > 1 else H * D
    else:
        B, S, H, D = shape
        seq, st, head, one = t.stride()
        if B > 1 and S > 1 and seq != S * st:
            raise ValueError(f"{name}: token rows must lie at one stride")
        ld = st if S > 1 else seq if B > 1 else H * D
    if one != 1 or (H > 1 and head != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return ld


def _expect_current(dev: int):
    """The tensors' device must be the current CUDA device, whose stream the call goes to."""
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    if dev != torch._C._cuda_getDevice():
        raise ValueError("tensors must be on the current CUDA device")


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(call: str, dev: int, *sizes) -> int:
    """A call's workspace size: a function of the device and the sizes (asking the library takes 0.7 us)."""
    return int(getattr(lib(), call)(*sizes))


_NO_WORKSPACE = 256         # a size that stands for none (the C calls want an address all the same)


@functools.lru_cache(maxsize=None)
def _placeholder(dev: int):
    """What stands in for a workspace that nothing is kept in."""
    return torch.empty(_NO_WORKSPACE, dtype=torch.uint8, device=f"cuda:{dev}")


def _dense_like(t):
    """An uninitialised contiguous tensor of t's shape, dtype and device (the cheapest way torch has)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _workspace(workspace, need: int, dev: int, like):
    """Address and bytes of the caller's workspace, or of a new one (third, to be kept until the launch)."""
    if workspace is None:
        workspace = like.new_empty(max(need, 256), dtype=torch.uint8)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the device of the other tensors")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def decode_paged_q8(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, idx, cnt, log_gate, sm_scale=None,
                    page_size: int = 64, workspace=None, with_lse: bool = True):
    """Paged decode over 8-bit pages: caches [P,Hkv,64,D] float8_e4m3fn, scales [P,Hkv] fp32 (a key is
    k_scale * code). Other arguments as in decode_paged. Returns o [N,Hq,D] and lse [N,Hq] (or None)."""
    N, Hq, D = q.shape
    P, Hkv = k_cache.shape[:2]
    K = idx.shape[-1]
    max_pages = page_table.shape[-1]
    dev = q.get_device()
    pages = (P, Hkv, page_size, D)
    ptrs = (_expect("q", q, _BF16, (N, Hq, D), dev), _expect("k_cache", k_cache, _F8, pages, dev),
            _expect("v_cache", v_cache, _F8, pages, dev), _expect("k_scale", k_scale, _F32T, (P, Hkv), dev),
            _expect("v_scale", v_scale, _F32T, (P, Hkv), dev))
    pt = _expect("page_table", page_table, _I32, (N, max_pages), dev)
    kv = _expect("kv_len", kv_len, _I32, (N,), dev)
    sel = (_expect("idx", idx, _I32, (N, Hkv, K), dev), _expect("cnt", cnt, _I32, (N, Hkv), dev),
           _expect("log_gate", log_gate, _F32T, (N, Hkv, K), dev))
    _expect_current(dev)
    sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    o = torch.empty_like(q)
    lse = q.new_empty(N, Hq, dtype=_F32T) if with_lse else None
    if N == 0:
        return o, lse
    need = _workspace_bytes("sas_decode_q8_workspace_size", dev, N, Hq, Hkv, D, K)
    if workspace is None and need == _NO_WORKSPACE:
        workspace = _placeholder(dev)
    ws, ws_bytes, workspace = _workspace(workspace, need, dev, q)
    code = lib().sas_decode_paged_q8(*ptrs, P, pt, max_pages, kv, N, Hq, Hkv, D, page_size, K, *sel, sm_scale, o.data_ptr(),
                                 lse.data_ptr() if with_lse else None, ws, ws_bytes, _raw_stream(dev))
    if code:
        _check(code)
    return o, lse


def rope_table(max_pos: int, D: int, base: float = 1e6, device="cuda"):
    """Rotation table [max_pos, D] fp32 for the calls below: D/2 cosines, then D/2 sines, of the angles
    p * base^(-2i/D), taken in 64 bits. Any other table of this layout (scaled frequencies) serves too."""
    inv = base ** (-torch.arange(0, D, 2, dtype=torch.float64, device=device) / D)
    ang = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((ang.cos(), ang.sin()), dim=1).float()


def _weight_ptrs(q_weight, k_weight, dtype, D, dev):
    if q_weight is None and k_weight is None:
        return None, None
    if q_weight is None or k_weight is None:
        raise ValueError("q_weight and k_weight go together")
    return _expect("q_weight", q_weight, dtype, (D,), dev), _expect("k_weight", k_weight, dtype, (D,), dev)


def _qk_args(q, k, table, q_weight, k_weight, positions, eps):
    """Checks shared by qk_norm_rope and its gradient: the C calls' arguments from the dtype (first) and from
    q on, and T, Hq, Hkv, D and the device."""
    qs, ks = q.shape, k.shape
    n = len(qs)
    if n == 3 and len(ks) == 3:
        (S, Hq, D), (Sk, Hkv, Dk) = qs, ks
        T, same = S, Sk == S and Dk == D
    elif n == 4 and len(ks) == 4:
        (B, S, Hq, D), (Bk, Sk, Hkv, Dk) = qs, ks
        T, same = B * S, Bk == B and Sk == S and Dk == D
    else:
        same = False
    if not same:
        raise ValueError(f"q and k must be [T,H,D] or [B,S,H,D] with the same tokens, got {tuple(qs)}, {tuple(ks)}")
    dtype, dev = q.dtype, q.get_device()
    max_pos = table.shape[0]
    ld_q, ld_k = _token_stride("q", q, qs), _expect_rows("k", k, dtype, ks, dev)
    tab = _expect("table", table, _F32T, (max_pos, D), dev)
    w = _weight_ptrs(q_weight, k_weight, dtype, D, dev)
    pos = None
    if positions is not None:
        pos = _expect("positions", positions, _I32, qs[:-2], dev)
    elif S > max_pos:
        raise ValueError(f"{S} positions, the table has {max_pos}")
    code = _dtype_code(q)
    _expect_current(dev)
    return code, (q.data_ptr(), ld_q, k.data_ptr(), ld_k, *w, tab, max_pos, pos, S, T, Hq, Hkv, D, eps), (T, Hq, Hkv, D, dev)


def qk_norm_rope(q, k, table, q_weight=None, k_weight=None, positions=None, eps: float = 1e-6):
    """Per-head RMS norm and rotary position embedding of queries and keys in one pass.

    q [B,S,Hq,D] or [T,Hq,D], k likewise, bf16 or fp32; token rows may be strided (parts of a fused
    projection's output). Weights [D] of the same dtype (both None: rotation only); table from rope_table;
    positions int32 of the token shape, or None: 0..S-1 in each sequence (3-D: one sequence).
    Returns contiguous q and k, as attn_fwd takes them."""
    code, args, (*_, dev) = _qk_args(q, k, table, q_weight, k_weight, positions, eps)
    q_out, k_out = _dense_like(q), _dense_like(k)
    code = lib().sas_qk_norm_rope(code, *args, q_out.data_ptr(), k_out.data_ptr(), _raw_stream(dev))
    if code:
        _check(code)
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, table, q_weight=None, k_weight=None, positions=None, eps: float = 1e-6,
                     workspace=None):
    """Gradients of qk_norm_rope: dq_out, dk_out (contiguous) are those of its outputs, the other arguments
    its inputs. Returns dq, dk (input dtype, contiguous) and the weights' gradients in fp32 (None without)."""
    code, args, (T, Hq, Hkv, D, dev) = _qk_args(q, k, table, q_weight, k_weight, positions, eps)
    up = (_expect("dq_out", dq_out, q.dtype, q.shape, dev), _expect("dk_out", dk_out, q.dtype, k.shape, dev))
    dq, dk = torch.empty_like(dq_out), torch.empty_like(dk_out)
    dwq = dwk = None
    if q_weight is not None:
        dwq, dwk = torch.empty_like(q_weight, dtype=_F32T), torch.empty_like(k_weight, dtype=_F32T)
    need = _workspace_bytes("sas_qk_norm_rope_bwd_workspace_size", dev, T, Hq, Hkv, D)
    ws, ws_bytes, workspace = _workspace(workspace, need, dev, q)
    code = lib().sas_qk_norm_rope_bwd(code, *up, *args, dq.data_ptr(), dk.data_ptr(), _addr(dwq), _addr(dwk), ws, ws_bytes,
                                  _raw_stream(dev))
    if code:
        _check(code)
    return dq, dk, dwq, dwk


def _addr(t):
    return None if t is None else t.data_ptr()


def _append(q8, q, k, v, table, k_cache, v_cache, scales, page_table, kv_len, q_weight, k_weight, cu_new, max_new, eps,
            kpool, with_k, page_size):
    T, Hq, D = q.shape
    Hkv, P, N = k.shape[1], k_cache.shape[0], kv_len.shape[0]
    max_pos, max_pages = table.shape[0], page_table.shape[-1]
    dev = q.get_device()
    dt = _F8 if q8 else _BF16
    pages = (P, Hkv, page_size, D)
    if q.dtype is not _BF16:
        raise TypeError(f"q must be {_BF16}, got {q.dtype}")
    ld_q = _token_stride("q", q, (T, Hq, D))
    ld_k = _expect_rows("k", k, _BF16, (T, Hkv, D), dev)
    ld_v = _expect_rows("v", v, _BF16, (T, Hkv, D), dev)
    tab = _expect("table", table, _F32T, (max_pos, D), dev)
    store = [_expect("k_cache", k_cache, dt, pages, dev), _expect("v_cache", v_cache, dt, pages, dev)]
    if q8:
        store += [_expect("k_scale", scales[0], _F32T, (P, Hkv), dev), _expect("v_scale", scales[1], _F32T, (P, Hkv), dev)]
    pt = _expect("page_table", page_table, _I32, (N, max_pages), dev)
    kv = _expect("kv_len", kv_len, _I32, (N,), dev)
    w = _weight_ptrs(q_weight, k_weight, _BF16, D, dev)
    cu = None if cu_new is None else _expect("cu_new", cu_new, _I32, (N + 1,), dev)
    pool = None if kpool is None else _expect("kpool", kpool, _F32T, (P, Hkv, D), dev)
    _expect_current(dev)
    q_out = _dense_like(q)
    k_out = _dense_like(k) if with_k else None
    fn = lib().sas_append_paged_q8 if q8 else lib().sas_append_paged
    code = fn(q.data_ptr(), ld_q, k.data_ptr(), ld_k, v.data_ptr(), ld_v, *w, tab, max_pos, cu, N, max_new, T, kv, pt,
              max_pages, P, Hq, Hkv, D, page_size, eps, q_out.data_ptr(), _addr(k_out), *store, pool, _raw_stream(dev))
    if code:
        _check(code)
    return (q_out, k_out) if with_k else q_out


def append_paged(q, k, v, table, k_cache, v_cache, page_table, kv_len, q_weight=None, k_weight=None, cu_new=None,
                 max_new: int = 1, eps: float = 1e-6, kpool=None, with_k: bool = False, page_size: int = 64):
    """New tokens into a paged KV cache [P,Hkv,64,D], with the norm and rotation of qk_norm_rope on the way.

    q [T,Hq,D], k, v [T,Hkv,D] bf16 (token rows may be strided). kv_len [N] counts the new tokens. One token
    for each sequence (T = N; kv_len 0: a padding entry), or with cu_new int32 [N+1] the rows
    cu_new[n]..cu_new[n+1]-1 of each, at most max_new. kpool [P,Hkv,D]: filled pages get their mean key.
    Returns the rotated q [T,Hq,D]; with_k: q and the rotated k [T,Hkv,D], as attn_fwd_varlen takes them for
    whole prompts. (Pieces behind cached tokens are stored, but no call attends from them to the cache.)"""
    return _append(False, q, k, v, table, k_cache, v_cache, (), page_table, kv_len, q_weight, k_weight, cu_new,
                   max_new, eps, kpool, with_k, page_size)


def append_paged_q8(q, k, v, table, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, q_weight=None,
                    k_weight=None, cu_new=None, max_new: int = 1, eps: float = 1e-6, kpool=None, with_k: bool = False,
                    page_size: int = 64):
    """append_paged into 8-bit pages: caches float8_e4m3fn, k_scale, v_scale [P,Hkv] fp32 (set by a page's
    first row, grown where later rows need it)."""
    return _append(True, q, k, v, table, k_cache, v_cache, (k_scale, v_scale), page_table, kv_len, q_weight,
                   k_weight, cu_new, max_new, eps, kpool, with_k, page_size)
