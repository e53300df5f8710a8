"""Thin ctypes binding of libzp.so (include/zp.h).  Argument marshalling only:
every step of compression and decode attention runs in the library's CUDA
kernels.  There is no fallback: if the library is missing or fails to load,
every call raises.

The functions keep the C names (``zp_cache_create``, ``zp_cache_create_fp8``, ``zp_compress``,
``zp_paged_decode_attn``, ``zp_append_slots``, ``zp_append_kv``,
``zp_compress_prefill``, ``zp_compress_prefill_workspace_size``, ``zp_global_redundancy``,
``zp_global_redundancy_gram``,
``zp_alloc_rows``, ``zp_release_rows``, ``zp_fork_rows``,
``zp_append_kv_chunk``, ``zp_paged_chunk_attn``, ``zp_verify_draft``,
``zp_sample``, ``zp_token_probs``,
``zp_cache_status``, ``zp_cache_destroy``, ``zp_status_string``) and take raw integers (device pointers, a cudaStream_t
as an int).  ``Cache`` wraps them for torch tensors: it reads ``data_ptr()``
and the current stream, and keeps the pool tensors alive.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_OUT_OF_BLOCKS = -3
ERR_DEVICE_CHECK = -4
ERR_CUDA = -5
ERR_TIMEOUT = -6

DTYPE_F32 = 0
DTYPE_BF16 = 1

P = ctypes.c_void_p
I64 = ctypes.c_int64
I32 = ctypes.c_int32


class zp_cache_desc(ctypes.Structure):
    _fields_ = [
        ("num_layers", I32), ("num_kv_heads", I32), ("num_q_heads", I32), ("head_dim", I32),
        ("block_size", I32), ("num_blocks", I32), ("max_requests", I32),
        ("max_blocks_per_req", I32), ("k_pools", ctypes.POINTER(P)),
        ("v_pools", ctypes.POINTER(P)),
    ]


class zp_block_pool(ctypes.Structure):
    _fields_ = [("free_ids", P), ("free_count", P), ("refcount", P), ("capacity", I32)]


class ZpError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None


def library_path() -> str:
    return _build.LIB


def lib():
    """The loaded libzp.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it first "
                              "(python -m compressed_paged_kv_gb300._build)")
        L = ctypes.CDLL(path)
        L.zp_cache_create.argtypes = [ctypes.POINTER(zp_cache_desc), ctypes.POINTER(P)]
        L.zp_cache_create.restype = I32
        L.zp_cache_create_fp8.argtypes = [ctypes.POINTER(zp_cache_desc), ctypes.POINTER(P),
                                          ctypes.POINTER(P), ctypes.POINTER(P)]
        L.zp_cache_create_fp8.restype = I32
        L.zp_cache_destroy.argtypes = [P]
        L.zp_cache_destroy.restype = None
        L.zp_compress.argtypes = [P, P, I32, I32, P, P, I32, P, I32, I32, ctypes.c_float,
                                  ctypes.POINTER(zp_block_pool), P, P, P]
        L.zp_compress.restype = I32
        L.zp_paged_decode_attn.argtypes = [P, I32, P, P, I32, I32, P, P, I32, ctypes.c_float, P,
                                           P]
        L.zp_paged_decode_attn.restype = I32
        L.zp_paged_decode_attn_noalloc.argtypes = [P, P, I32, I32, I32, I32, P, P, I32, I32, P,
                                                   P, I32, ctypes.c_float, P, P, P]
        L.zp_paged_decode_attn_noalloc.restype = I32
        L.zp_append_slots.argtypes = [P, P, I32, I32, P, P, I32, I32,
                                      ctypes.POINTER(zp_block_pool), P, P, P]
        L.zp_append_slots.restype = I32
        L.zp_append_kv.argtypes = [P, I32, P, P, P, I32, I32, P, P, I32, P]
        L.zp_append_kv.restype = I32
        L.zp_compress_prefill_workspace_size.argtypes = [P, I32, I32,
                                                         ctypes.POINTER(ctypes.c_size_t)]
        L.zp_compress_prefill_workspace_size.restype = I32
        L.zp_compress_prefill.argtypes = [P, P, I32, I32, P, P, I32, P, I32, I32, ctypes.c_float,
                                          ctypes.POINTER(zp_block_pool), P, ctypes.c_size_t, P,
                                          P, P]
        L.zp_compress_prefill.restype = I32
        L.zp_alloc_rows.argtypes = [P, P, I32, I32, P, P, I32, P, ctypes.POINTER(zp_block_pool), P]
        L.zp_alloc_rows.restype = I32
        L.zp_release_rows.argtypes = [P, P, I32, I32, P, P, I32, ctypes.POINTER(zp_block_pool), P]
        L.zp_release_rows.restype = I32
        L.zp_fork_rows.argtypes = [P, P, I32, I32, P, P, P, I32, P, P]
        L.zp_fork_rows.restype = I32
        L.zp_append_kv_chunk.argtypes = [P, I32, P, I64, P, I64, P, I32, P, I32, I32, P, P, I32, P]
        L.zp_append_kv_chunk.restype = I32
        L.zp_paged_chunk_attn.argtypes = [P, I32, P, I64, P, I32, P, I32, I32, P, P, I32,
                                          ctypes.c_float, P, P]
        L.zp_paged_chunk_attn.restype = I32
        L.zp_verify_draft.argtypes = [P, P, P, I32, P, P, I32, I32, I64, P, P, P, I32, P, I32, P,
                                      P, P]
        L.zp_verify_draft.restype = I32
        L.zp_sample.argtypes = [P, P, I32, I32, I64, P, P, P, P, I32, P, P, I32, P, P]
        L.zp_sample.restype = I32
        L.zp_token_probs.argtypes = [P, P, I32, I32, I64, P, P, P, P, I32, P, I32, P, I32, I64, P]
        L.zp_token_probs.restype = I32
        L.zp_global_redundancy.argtypes = [P, P, I32, I32, P, P, I32, P, P]
        L.zp_global_redundancy.restype = I32
        L.zp_global_redundancy_gram.argtypes = [P, P, I32, I32, P, P, I32, P, P]
        L.zp_global_redundancy_gram.restype = I32
        L.zp_cache_status.argtypes = [P, P, ctypes.POINTER(I32)]
        L.zp_cache_status.restype = I32
        L.zp_status_string.argtypes = [I32]
        L.zp_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


# ------------------------------------------------------------- raw C names

def status_string(status: int) -> str:
    return lib().zp_status_string(int(status)).decode()


zp_status_string = status_string


def zp_cache_create(desc: zp_cache_desc) -> int:
    """Returns the handle (an int) or raises ZpError."""
    h = P()
    st = lib().zp_cache_create(ctypes.byref(desc), ctypes.byref(h))
    if st != OK:
        raise ZpError(st, "zp_cache_create")
    return h.value


def zp_cache_create_fp8(desc: zp_cache_desc, k_scales, v_scales) -> int:
    """``k_scales``, ``v_scales``: ctypes arrays of the layers' scale pointers.
    Returns the handle (an int) or raises ZpError."""
    h = P()
    st = lib().zp_cache_create_fp8(ctypes.byref(desc), k_scales, v_scales, ctypes.byref(h))
    if st != OK:
        raise ZpError(st, "zp_cache_create_fp8")
    return h.value


def zp_cache_destroy(handle: int) -> None:
    lib().zp_cache_destroy(P(handle))


def zp_compress(handle, block_tables, bt_stride, num_rows, lengths, req_idx, R, window_q,
                n_max, window, lam, pool: zp_block_pool, stream, scores_out=0,
                kept_out=0) -> int:
    return lib().zp_compress(P(handle), P(block_tables), bt_stride, num_rows, P(lengths),
                             P(req_idx or None), R, P(window_q), n_max, window, float(lam),
                             ctypes.byref(pool), P(stream or None), P(scores_out or None),
                             P(kept_out or None))


def zp_compress_prefill_workspace_size(handle, R, bt_stride) -> int:
    n = ctypes.c_size_t(0)
    st = lib().zp_compress_prefill_workspace_size(P(handle), R, bt_stride, ctypes.byref(n))
    if st != OK:
        raise ZpError(st, "zp_compress_prefill_workspace_size")
    return n.value


def zp_compress_prefill(handle, block_tables, bt_stride, num_rows, lengths, req_idx, R, window_q,
                        n_max, window, lam, pool: zp_block_pool, workspace, workspace_bytes,
                        stream, scores_out=0, kept_out=0) -> int:
    return lib().zp_compress_prefill(P(handle), P(block_tables), bt_stride, num_rows,
                                     P(lengths), P(req_idx or None), R, P(window_q), n_max,
                                     window, float(lam), ctypes.byref(pool), P(workspace or None),
                                     workspace_bytes, P(stream or None), P(scores_out or None),
                                     P(kept_out or None))


def zp_paged_decode_attn(handle, layer, q, block_tables, bt_stride, num_rows, lengths, req_idx,
                         R, scale, out, stream) -> int:
    return lib().zp_paged_decode_attn(P(handle), layer, P(q), P(block_tables), bt_stride,
                                      num_rows, P(lengths), P(req_idx or None), R, float(scale),
                                      P(out), P(stream or None))


def zp_paged_decode_attn_noalloc(k_pool, v_pool, num_blocks, num_kv_heads, num_q_heads, head_dim,
                                 q, block_tables, bt_stride, num_rows, lengths, req_idx, R, scale,
                                 out, status, stream) -> int:
    """Decode attention without a handle and without any allocation (for
    callers that cannot call cudaMalloc); see include/zp.h."""
    return lib().zp_paged_decode_attn_noalloc(
        P(k_pool), P(v_pool), num_blocks, num_kv_heads, num_q_heads, head_dim, P(q),
        P(block_tables), bt_stride, num_rows, P(lengths), P(req_idx or None), R, float(scale),
        P(out), P(status or None), P(stream or None))


def zp_append_slots(handle, block_tables, bt_stride, num_rows, lengths, req_idx, R, n_max,
                    pool: zp_block_pool, stream, trigger_rows=0, trigger_count=0) -> int:
    return lib().zp_append_slots(P(handle), P(block_tables), bt_stride, num_rows, P(lengths),
                                 P(req_idx or None), R, n_max, ctypes.byref(pool),
                                 P(stream or None), P(trigger_rows or None),
                                 P(trigger_count or None))


def zp_append_kv(handle, layer, k_new, v_new, block_tables, bt_stride, num_rows, lengths,
                 req_idx, R, stream) -> int:
    return lib().zp_append_kv(P(handle), layer, P(k_new), P(v_new), P(block_tables), bt_stride,
                              num_rows, P(lengths), P(req_idx or None), R, P(stream or None))


def zp_alloc_rows(handle, block_tables, bt_stride, num_rows, lengths, req_idx, R, counts,
                  pool: zp_block_pool, stream) -> int:
    return lib().zp_alloc_rows(P(handle), P(block_tables), bt_stride, num_rows, P(lengths),
                               P(req_idx or None), R, P(counts), ctypes.byref(pool),
                               P(stream or None))


def zp_release_rows(handle, block_tables, bt_stride, num_rows, lengths, req_idx, R,
                    pool: zp_block_pool, stream) -> int:
    return lib().zp_release_rows(P(handle), P(block_tables), bt_stride, num_rows, P(lengths),
                                 P(req_idx or None), R, ctypes.byref(pool), P(stream or None))


def zp_fork_rows(handle, block_tables, bt_stride, num_rows, lengths, src_rows, dst_rows, n,
                 refcount, stream) -> int:
    return lib().zp_fork_rows(P(handle), P(block_tables), bt_stride, num_rows, P(lengths),
                              P(src_rows), P(dst_rows), n, P(refcount), P(stream or None))


def zp_append_kv_chunk(handle, layer, k_new, k_stride, v_new, v_stride, starts, total,
                       block_tables, bt_stride, num_rows, lengths, req_idx, R, stream) -> int:
    # plain integers: their pointer arguments are declared, so ctypes converts them
    return lib().zp_append_kv_chunk(handle, layer, k_new, k_stride, v_new, v_stride, starts, total,
                                    block_tables, bt_stride, num_rows, lengths, req_idx, R, stream)


def zp_paged_chunk_attn(handle, layer, q, q_stride, starts, total, block_tables, bt_stride,
                        num_rows, lengths, req_idx, R, scale, out, stream) -> int:
    return lib().zp_paged_chunk_attn(handle, layer, q, q_stride, starts, total, block_tables,
                                     bt_stride, num_rows, lengths, req_idx, R, scale, out, stream)


def zp_verify_draft(handle, tokens, starts, total, target_probs, draft_probs, prob_dtype, vocab,
                    prob_stride, accept_u, sample_u, lengths, num_rows, req_idx, R, accepted,
                    next_tokens, stream) -> int:
    return lib().zp_verify_draft(handle, tokens, starts, total, target_probs, draft_probs,
                                 prob_dtype, vocab, prob_stride, accept_u, sample_u, lengths,
                                 num_rows, req_idx, R, accepted, next_tokens, stream)


def zp_sample(handle, logits, logit_dtype, vocab, logit_stride, temperature, top_k, top_p, min_p,
              num_rows, req_idx, u, R, tokens, stream) -> int:
    return lib().zp_sample(handle, logits, logit_dtype, vocab, logit_stride, temperature, top_k,
                           top_p, min_p, num_rows, req_idx, u, R, tokens, stream)


def zp_token_probs(handle, logits, logit_dtype, vocab, logit_stride, temperature, top_k, top_p,
                   min_p, num_rows, req_idx, R, probs, prob_dtype, prob_stride, stream) -> int:
    return lib().zp_token_probs(handle, logits, logit_dtype, vocab, logit_stride, temperature,
                                top_k, top_p, min_p, num_rows, req_idx, R, probs, prob_dtype,
                                prob_stride, stream)


def zp_global_redundancy(handle, block_tables, bt_stride, num_rows, lengths, req_idx, R, red_out,
                         stream) -> int:
    return lib().zp_global_redundancy(P(handle), P(block_tables), bt_stride, num_rows,
                                      P(lengths), P(req_idx or None), R, P(red_out),
                                      P(stream or None))


def zp_global_redundancy_gram(handle, block_tables, bt_stride, num_rows, lengths, req_idx, R,
                              red_out, stream) -> int:
    return lib().zp_global_redundancy_gram(P(handle), P(block_tables), bt_stride, num_rows,
                                           P(lengths), P(req_idx or None), R, P(red_out),
                                           P(stream or None))


def zp_cache_status(handle, stream) -> tuple[int, int]:
    """(call status, device status) after synchronising the stream."""
    v = I32(0)
    st = lib().zp_cache_status(P(handle), P(stream or None), ctypes.byref(v))
    return st, v.value


# ------------------------------------------------------------ torch wrapper

def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    import torch
    # the handle of the current stream without building a Stream object (3 us
    # less a call), where torch has it
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _row_stride(t, what, inner, dtype):
    """Elements between the rows of a packed tensor [total, *inner] whose rows
    are each contiguous."""
    shape, strides = t.shape, t.stride()
    n = 1
    ok = len(shape) == 1 + len(inner) and t.dtype == dtype and t.is_cuda
    for dim in range(len(inner), 0, -1):
        if not ok:
            break
        size = inner[dim - 1]
        ok = shape[dim] == size and (strides[dim] == n or size <= 1)
        n *= size
    if not ok:
        raise ValueError(f"{what} must be a {dtype} CUDA tensor [total, "
                         f"{', '.join(map(str, inner))}] with contiguous rows, got {t.dtype} "
                         f"{tuple(shape)} strides {strides}")
    return strides[0] if shape[0] > 1 else n


def _flat(t, what, n, dtype):
    if t.dtype != dtype or t.numel() < n or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{what} must be a contiguous {dtype} CUDA tensor of {n} elements")


class Cache:
    """A zp_cache over per-layer torch pools ([num_blocks][Hkv][16][d] bf16), or with
    ``k_scales`` and ``v_scales`` ([num_blocks][Hkv] fp32 a layer) an 8-bit one
    over float8_e4m3fn pools."""

    def __init__(self, k_pools, v_pools, num_q_heads, max_requests, max_blocks_per_req,
                 k_scales=None, v_scales=None):
        import torch
        assert len(k_pools) == len(v_pools) >= 1
        fp8 = k_scales is not None
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        for t in list(k_pools) + list(v_pools):
            if not (t.is_cuda and t.dtype == dtype and t.is_contiguous() and t.dim() == 4):
                raise ValueError(f"pools must be contiguous 4-D {dtype} CUDA tensors")
            if fp8 and t.shape != k_pools[0].shape:
                raise ValueError("pools must have one shape")
        nb, hkv, b, d = k_pools[0].shape
        if fp8 != (v_scales is not None) or (
                fp8 and not len(k_scales) == len(v_scales) == len(k_pools)):
            raise ValueError("k_scales and v_scales must hold one tensor a layer, or both be None")
        for t in (list(k_scales) + list(v_scales)) if fp8 else []:
            if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()
                    and t.shape == (nb, hkv)):
                raise ValueError("scales must be contiguous [num_blocks, Hkv] float32 CUDA tensors")
        self.k_scales, self.v_scales = (list(k_scales), list(v_scales)) if fp8 else (None, None)
        self.k_pools, self.v_pools = list(k_pools), list(v_pools)
        self.dtype, self.int32, self.float32 = torch.bfloat16, torch.int32, torch.float32
        self.L, self.Hkv, self.Hq, self.d, self.b, self.num_blocks = (
            len(k_pools), hkv, num_q_heads, d, b, nb)
        kp = (P * self.L)(*[t.data_ptr() for t in k_pools])
        vp = (P * self.L)(*[t.data_ptr() for t in v_pools])
        desc = zp_cache_desc(self.L, hkv, num_q_heads, d, b, nb, max_requests,
                             max_blocks_per_req, kp, vp)
        if fp8:
            ks = (P * self.L)(*[t.data_ptr() for t in k_scales])
            vs = (P * self.L)(*[t.data_ptr() for t in v_scales])
            self.handle = zp_cache_create_fp8(desc, ks, vs)
        else:
            self.handle = zp_cache_create(desc)

    def close(self):
        if getattr(self, "handle", None):
            zp_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def compress(self, block_tables, lengths, window_q, n_max, window, lam, free_ids,
                 free_count, refcount, req_idx=None, scores_out=None, kept_out=None,
                 stream=None, check=True):
        pool = zp_block_pool(free_ids.data_ptr(), free_count.data_ptr(), refcount.data_ptr(),
                             free_ids.numel())
        R = window_q.shape[1]
        st = zp_compress(self.handle, block_tables.data_ptr(), block_tables.shape[1],
                         block_tables.shape[0], lengths.data_ptr(), _ptr(req_idx), R,
                         window_q.data_ptr(), n_max, window, lam, pool, _stream(stream),
                         _ptr(scores_out), _ptr(kept_out))
        if check and st != OK:
            raise ZpError(st, "zp_compress")
        return st

    def compress_prefill(self, block_tables, lengths, window_q, n_max, window, lam, free_ids,
                         free_count, refcount, workspace, req_idx=None, scores_out=None,
                         kept_out=None, stream=None, check=True):
        """``workspace``: a uint8 CUDA tensor of at least
        ``prefill_workspace_bytes(R, block_tables.shape[1])`` bytes."""
        pool = zp_block_pool(free_ids.data_ptr(), free_count.data_ptr(), refcount.data_ptr(),
                             free_ids.numel())
        R = window_q.shape[1]
        st = zp_compress_prefill(self.handle, block_tables.data_ptr(), block_tables.shape[1],
                                 block_tables.shape[0], lengths.data_ptr(), _ptr(req_idx), R,
                                 window_q.data_ptr(), n_max, window, lam, pool,
                                 workspace.data_ptr(), workspace.numel(), _stream(stream),
                                 _ptr(scores_out), _ptr(kept_out))
        if check and st != OK:
            raise ZpError(st, "zp_compress_prefill")
        return st

    def prefill_workspace_bytes(self, R, bt_stride) -> int:
        return zp_compress_prefill_workspace_size(self.handle, R, bt_stride)

    def decode(self, layer, q, block_tables, lengths, scale, out, req_idx=None, stream=None,
               check=True):
        st = zp_paged_decode_attn(self.handle, layer, q.data_ptr(), block_tables.data_ptr(),
                                  block_tables.shape[1], block_tables.shape[0],
                                  lengths.data_ptr(), _ptr(req_idx), q.shape[0], scale,
                                  out.data_ptr(), _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_paged_decode_attn")
        return st

    def append_slots(self, block_tables, lengths, n_max, free_ids, free_count, refcount,
                     req_idx=None, R=None, trigger_rows=None, trigger_count=None, stream=None,
                     check=True):
        pool = zp_block_pool(free_ids.data_ptr(), free_count.data_ptr(), refcount.data_ptr(),
                             free_ids.numel())
        if R is None:
            R = req_idx.numel() if req_idx is not None else block_tables.shape[0]
        st = zp_append_slots(self.handle, block_tables.data_ptr(), block_tables.shape[1],
                             block_tables.shape[0], lengths.data_ptr(), _ptr(req_idx), R, n_max,
                             pool, _stream(stream), _ptr(trigger_rows), _ptr(trigger_count))
        if check and st != OK:
            raise ZpError(st, "zp_append_slots")
        return st

    def append_kv(self, layer, k_new, v_new, block_tables, lengths, req_idx=None, stream=None,
                  check=True):
        st = zp_append_kv(self.handle, layer, k_new.data_ptr(), v_new.data_ptr(),
                          block_tables.data_ptr(), block_tables.shape[1], block_tables.shape[0],
                          lengths.data_ptr(), _ptr(req_idx), k_new.shape[0], _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_append_kv")
        return st

    def append_kv_chunk(self, layer, k_new, v_new, starts, block_tables, lengths, req_idx=None,
                        stream=None, check=True):
        """k_new, v_new: [total, Hkv, d] bf16, each token's row contiguous (a
        slice of a packed projection output is passed as it is)."""
        row = (self.Hkv, self.d)
        ks = _row_stride(k_new, "k_new", row, self.dtype)
        vs = _row_stride(v_new, "v_new", row, self.dtype)
        total = k_new.shape[0]
        if v_new.shape[0] != total:
            raise ValueError("k_new and v_new must hold the same tokens")
        R, rows = self._chunk_ints(starts, block_tables, lengths, req_idx)
        st = zp_append_kv_chunk(self.handle, layer, k_new.data_ptr(), ks, v_new.data_ptr(), vs,
                                starts.data_ptr(), total, block_tables.data_ptr(),
                                block_tables.shape[1], rows, lengths.data_ptr(), _ptr(req_idx), R,
                                _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_append_kv_chunk")
        return st

    def chunk_attn(self, layer, q, starts, block_tables, lengths, scale, out, req_idx=None,
                   stream=None, check=True):
        """q: [total, Hq, d] bf16, each token's row contiguous; out: the same
        shape, contiguous."""
        qs = _row_stride(q, "q", (self.Hq, self.d), self.dtype)
        _flat(out, "out", q.numel(), self.dtype)
        R, rows = self._chunk_ints(starts, block_tables, lengths, req_idx)
        st = zp_paged_chunk_attn(self.handle, layer, q.data_ptr(), qs, starts.data_ptr(),
                                 q.shape[0], block_tables.data_ptr(), block_tables.shape[1], rows,
                                 lengths.data_ptr(), _ptr(req_idx), R, scale, out.data_ptr(),
                                 _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_paged_chunk_attn")
        return st

    def _chunk_ints(self, starts, block_tables, lengths, req_idx):
        """Checks the index tensors of a chunk call: (chunks, table rows)."""
        i32 = self.int32
        R = starts.shape[0] - 1
        rows = block_tables.shape[0]
        _flat(starts, "starts", 1, i32)
        _flat(block_tables, "block_tables", 1, i32)
        _flat(lengths, "lengths", rows, i32)
        if req_idx is not None:
            _flat(req_idx, "req_idx", R, i32)
        elif R > rows:
            raise ValueError(f"{R} chunks for {rows} table rows")
        return R, rows

    def verify_draft(self, tokens, starts, target_probs, accept_u, sample_u, accepted,
                     next_tokens, draft_probs=None, lengths=None, req_idx=None, stream=None,
                     check=True):
        """target_probs, draft_probs: [total, vocab] fp32 or bf16 with the same
        row stride."""
        i32, f32, dtype = self.int32, self.float32, target_probs.dtype
        if target_probs.dim() != 2 or dtype not in (f32, self.dtype):
            raise ValueError("target_probs must be [total, vocab], float32 or bfloat16")
        total, vocab = target_probs.shape
        ps = _row_stride(target_probs, "target_probs", (vocab,), dtype)
        if draft_probs is not None:
            ds = _row_stride(draft_probs, "draft_probs", (vocab,), dtype)
            if draft_probs.shape[0] != total or ds != ps:
                raise ValueError("draft_probs must have target_probs' rows and row stride")
        R = starts.shape[0] - 1
        _flat(starts, "starts", 1, i32)
        _flat(tokens, "tokens", total, i32)
        _flat(accept_u, "accept_u", total, f32)
        _flat(sample_u, "sample_u", R, f32)
        _flat(accepted, "accepted", R, i32)
        _flat(next_tokens, "next_tokens", R, i32)
        rows = 0
        if lengths is not None:
            rows = lengths.shape[0]
            _flat(lengths, "lengths", R if req_idx is None else 1, i32)
            if req_idx is not None:
                _flat(req_idx, "req_idx", R, i32)
        st = zp_verify_draft(self.handle, tokens.data_ptr(), starts.data_ptr(), total,
                             target_probs.data_ptr(), _ptr(draft_probs),
                             DTYPE_F32 if dtype == f32 else DTYPE_BF16, vocab, ps,
                             accept_u.data_ptr(), sample_u.data_ptr(), _ptr(lengths), rows,
                             _ptr(req_idx), R, accepted.data_ptr(), next_tokens.data_ptr(),
                             _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_verify_draft")
        return st

    def sample(self, logits, u, tokens, temperature=None, top_k=None, top_p=None, min_p=None,
               req_idx=None, stream=None, check=True):
        """logits: [R, vocab] fp32 or bf16 with contiguous rows; the filters one entry a
        request ([rows], row i uses entry req_idx[i] or i), each optional."""
        dtype, vocab, ls, R, rows = self._logit_rows(logits, temperature, top_k, top_p, min_p,
                                                     req_idx)
        _flat(u, "u", R, self.float32)
        _flat(tokens, "tokens", R, self.int32)
        st = zp_sample(self.handle, logits.data_ptr(), dtype, vocab, ls, _ptr(temperature),
                       _ptr(top_k), _ptr(top_p), _ptr(min_p), rows, _ptr(req_idx), u.data_ptr(), R,
                       tokens.data_ptr(), _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_sample")
        return st

    def token_probs(self, logits, probs, temperature=None, top_k=None, top_p=None, min_p=None,
                    req_idx=None, stream=None, check=True):
        """logits and the filters as in ``sample``; probs: [R, vocab] fp32 or bf16 with
        contiguous rows."""
        dtype, vocab, ls, R, rows = self._logit_rows(logits, temperature, top_k, top_p, min_p,
                                                     req_idx)
        if probs.dtype not in (self.float32, self.dtype):
            raise ValueError("probs must be [R, vocab], float32 or bfloat16")
        ps = _row_stride(probs, "probs", (vocab,), probs.dtype)
        if probs.shape[0] != R:
            raise ValueError("probs must have a row for each row of logits")
        st = zp_token_probs(self.handle, logits.data_ptr(), dtype, vocab, ls, _ptr(temperature),
                            _ptr(top_k), _ptr(top_p), _ptr(min_p), rows, _ptr(req_idx), R,
                            probs.data_ptr(),
                            DTYPE_F32 if probs.dtype == self.float32 else DTYPE_BF16, ps,
                            _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_token_probs")
        return st

    def _logit_rows(self, logits, temperature, top_k, top_p, min_p, req_idx):
        """Checks the rows of logits and their filters: (type, vocabulary, row stride, rows,
        entries of the filters)."""
        if logits.dim() != 2 or logits.dtype not in (self.float32, self.dtype):
            raise ValueError("logits must be [R, vocab], float32 or bfloat16")
        R, vocab = logits.shape
        stride = _row_stride(logits, "logits", (vocab,), logits.dtype)
        rows = None
        for t, what, dtype in ((temperature, "temperature", self.float32),
                               (top_k, "top_k", self.int32), (top_p, "top_p", self.float32),
                               (min_p, "min_p", self.float32)):
            if t is None:
                continue
            if rows is None:
                rows = t.numel()
            _flat(t, what, rows, dtype)
            if t.numel() != rows:
                raise ValueError("the filters must have as many entries as each other")
        if req_idx is not None:
            _flat(req_idx, "req_idx", R, self.int32)
            if rows is None:  # no filters: any entry will do
                rows = 0x7fffffff
        elif rows is None:
            rows = max(R, 1)
        elif rows < R:
            raise ValueError(f"{R} rows for {rows} entries of the filters")
        return (DTYPE_F32 if logits.dtype == self.float32 else DTYPE_BF16, vocab, stride, R, rows)

    def alloc_rows(self, block_tables, lengths, counts, free_ids, free_count, refcount,
                   req_idx=None, stream=None, check=True):
        pool = zp_block_pool(free_ids.data_ptr(), free_count.data_ptr(), refcount.data_ptr(),
                             free_ids.numel())
        st = zp_alloc_rows(self.handle, block_tables.data_ptr(), block_tables.shape[1],
                           block_tables.shape[0], lengths.data_ptr(), _ptr(req_idx),
                           counts.numel(), counts.data_ptr(), pool, _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_alloc_rows")
        return st

    def release_rows(self, block_tables, lengths, free_ids, free_count, refcount, req_idx=None,
                     R=None, stream=None, check=True):
        pool = zp_block_pool(free_ids.data_ptr(), free_count.data_ptr(), refcount.data_ptr(),
                             free_ids.numel())
        if R is None:
            R = req_idx.numel() if req_idx is not None else block_tables.shape[0]
        st = zp_release_rows(self.handle, block_tables.data_ptr(), block_tables.shape[1],
                             block_tables.shape[0], lengths.data_ptr(), _ptr(req_idx), R, pool,
                             _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_release_rows")
        return st

    def fork_rows(self, block_tables, lengths, refcount, src_rows, dst_rows, stream=None,
                  check=True):
        st = zp_fork_rows(self.handle, block_tables.data_ptr(), block_tables.shape[1],
                          block_tables.shape[0], lengths.data_ptr(), src_rows.data_ptr(),
                          dst_rows.data_ptr(), src_rows.numel(), refcount.data_ptr(),
                          _stream(stream))
        if check and st != OK:
            raise ZpError(st, "zp_fork_rows")
        return st

    def global_redundancy(self, block_tables, lengths, red_out, req_idx=None, R=None,
                          stream=None, check=True, gram=False):
        """gram=False: zp_global_redundancy (O(T d)); gram=True:
        zp_global_redundancy_gram (the dense Gram on the tensor cores)."""
        if R is None:
            R = req_idx.numel() if req_idx is not None else block_tables.shape[0]
        fn = zp_global_redundancy_gram if gram else zp_global_redundancy
        st = fn(self.handle, block_tables.data_ptr(), block_tables.shape[1],
                block_tables.shape[0], lengths.data_ptr(), _ptr(req_idx), R,
                red_out.data_ptr(), _stream(stream))
        if check and st != OK:
            raise ZpError(st, fn.__name__)
        return st

    def status(self, stream=None) -> int:
        st, dev = zp_cache_status(self.handle, _stream(stream))
        if st != OK:
            raise ZpError(st, "zp_cache_status")
        return dev
