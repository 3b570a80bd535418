"""paged_kv_cache_171_gb300 -- paged GQA attention for GB300 (sm_103a).

A thin ctypes binding over libpa.so, whose C ABI is include/pa.h.  The
functions named like the C entry points (``pa_decode``, ``pa_append_kv``,
``pa_prefill_paged``, ``pa_merge_partials``, ...) only marshal arguments:
torch tensors become device pointers, the stream becomes a cudaStream_t,
and a nonzero status raises :class:`PAError`.  Every step of the attention
runs in libpa's CUDA kernels; there is no CPU or PyTorch fallback, and using
any of these functions without a built libpa.so raises.

Build the library with ``python -m paged_kv_cache_171_gb300.build`` (or
``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "PAError", "BF16", "F16", "lib", "dtype_code", "pa_decode", "pa_decode_append",
    "decode_append",
    "pa_decode_partition_tokens", "pa_decode_workspace_size",
    "pa_decode_static_workspace",
    "pa_merge_partials", "pa_append_kv", "pa_prefill_paged",
    "pa_prefill_paged_split", "pa_prefill_partition_tokens", "pa_prefill_workspace_size",
    "pa_decode_window", "pa_decode_window_workspace_size", "decode_window",
    "pa_pool_create", "pa_pool_destroy", "pa_pool_free_pages", "pa_pool_refcount",
    "pa_pool_alloc", "pa_pool_share", "pa_pool_release", "pa_pool_prepare_append",
    "pa_copy_pages", "pa_topm_retain", "pa_topm_workspace_size", "topm_retain",
    "pa_last_device_error", "pa_selftest_wait_timeout", "pa_strerror", "decode", "prefill",
    "prefill_split", "pa_decode_cascade", "pa_decode_cascade_workspace_size",
    "decode_cascade",
    "append_kv",
    "pa_append_kv_rope", "pa_append_kv_rope_at", "append_kv_rope", "rope_table",
    "pa_kv4_block_bytes", "kv4_cache", "pa_append_kv4", "append_kv4", "pa_read_kv4", "read_kv4",
    "pa_copy_pages_kv4", "copy_pages_kv4", "pa_decode_kv4", "pa_decode_kv4_workspace_size",
    "decode_kv4", "pa_prefill_kv4", "pa_prefill_kv4_workspace_size", "prefill_kv4",
    "weight_pool", "pa_decode_weighted", "pa_decode_weighted_workspace_size", "decode_weighted",
    "pa_prefill_weights", "pa_prefill_weights_workspace_size", "prefill_weights",
    "pa_evict_kv", "pa_evict_kv_workspace_size", "evict_kv", "pa_compact_kv", "compact_kv",
    "pa_prefill_tree", "pa_prefill_tree_workspace_size", "prefill_tree", "pa_tree_mask",
    "tree_mask",
]

BF16 = 0
F16 = 1

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libpa.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "pa.h")

_lib = None


class PAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {pa_strerror(status)} ({status})")


def lib():
    """The loaded libpa.so (ctypes.CDLL); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"libpa.so not built ({LIB_PATH}); run "
                "`python -m paged_kv_cache_171_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.pa_strerror.argtypes = [I]
        L.pa_strerror.restype = ctypes.c_char_p
        L.pa_decode.argtypes = [P, P, P, P, P, P, F] + [I] * 8 + [I, P, Z, P]
        L.pa_decode.restype = I
        L.pa_decode_append.argtypes = [P] * 8 + [F] + [I] * 8 + [I, P, Z, P]
        L.pa_decode_append.restype = I
        L.pa_decode_partition_tokens.argtypes = [I] * 7
        L.pa_decode_partition_tokens.restype = I
        L.pa_decode_workspace_size.argtypes = [I] * 7
        L.pa_decode_workspace_size.restype = Z
        L.pa_merge_partials.argtypes = [P, P, P, I, I, I, I, I, P]
        L.pa_merge_partials.restype = I
        L.pa_append_kv.argtypes = [P] * 7 + [I] * 8 + [P]
        L.pa_append_kv.restype = I
        L.pa_prefill_paged.argtypes = [P, P, P, P, P, I, P, F] + [I] * 8 + [P]
        L.pa_prefill_paged.restype = I
        L.pa_prefill_paged_split.argtypes = [P, P, P, P, P, I, P, F] + [I] * 9 + [P, Z, P]
        L.pa_prefill_paged_split.restype = I
        L.pa_prefill_partition_tokens.argtypes = [I] * 8
        L.pa_prefill_partition_tokens.restype = I
        L.pa_prefill_workspace_size.argtypes = [I] * 8
        L.pa_prefill_workspace_size.restype = Z
        L.pa_decode_window.argtypes = [P, P, P, P, P, P, F] + [I] * 11 + [P, Z, P]
        L.pa_decode_window.restype = I
        L.pa_decode_window_workspace_size.argtypes = [I] * 9
        L.pa_decode_window_workspace_size.restype = Z
        L.pa_pool_create.argtypes = [I]
        L.pa_pool_create.restype = P
        L.pa_pool_destroy.argtypes = [P]
        L.pa_pool_destroy.restype = None
        L.pa_pool_free_pages.argtypes = [P]
        L.pa_pool_free_pages.restype = I
        L.pa_pool_refcount.argtypes = [P, I]
        L.pa_pool_refcount.restype = I
        for f in ("pa_pool_alloc", "pa_pool_share", "pa_pool_release"):
            getattr(L, f).argtypes = [P, I, P] if f == "pa_pool_alloc" else [P, P, I]
            getattr(L, f).restype = I
        L.pa_pool_prepare_append.argtypes = [P, P, I, I, I, P, P]
        L.pa_pool_prepare_append.restype = I
        L.pa_copy_pages.argtypes = [P, P, P, P] + [I] * 6 + [P]
        L.pa_copy_pages.restype = I
        L.pa_topm_workspace_size.argtypes = [I, I, I]
        L.pa_topm_workspace_size.restype = Z
        L.pa_topm_retain.argtypes = [P, I, I, I, I, ctypes.c_longlong, P, P, P, Z, P]
        L.pa_topm_retain.restype = I
        L.pa_decode_cascade.argtypes = [P, P, P, P, I, I, P, P, P, F] + [I] * 9 + [P, Z, P]
        L.pa_decode_cascade.restype = I
        L.pa_decode_cascade_workspace_size.argtypes = [I] * 8
        L.pa_decode_cascade_workspace_size.restype = Z
        L.pa_decode_static_workspace.argtypes = [P, P, P, P, P, P, F] + [I] * 9 + [P]
        L.pa_decode_static_workspace.restype = I
        J = ctypes.c_int64
        L.pa_append_kv_rope.argtypes = [P] * 10 + [I, J, J, J] + [I] * 11 + [P]
        L.pa_append_kv_rope.restype = I
        L.pa_append_kv_rope_at.argtypes = [P] * 11 + [I, J, J, J] + [I] * 11 + [P]
        L.pa_append_kv_rope_at.restype = I
        L.pa_kv4_block_bytes.argtypes = [I]
        L.pa_kv4_block_bytes.restype = Z
        L.pa_append_kv4.argtypes = [P] * 9 + [I, J, J, J] + [I] * 11 + [P]
        L.pa_append_kv4.restype = I
        L.pa_read_kv4.argtypes = [P] * 6 + [I] * 8 + [P]
        L.pa_read_kv4.restype = I
        L.pa_copy_pages_kv4.argtypes = [P] * 3 + [I] * 5 + [P]
        L.pa_copy_pages_kv4.restype = I
        L.pa_decode_kv4.argtypes = [P] * 5 + [F] + [I] * 8 + [P, Z, P]
        L.pa_decode_kv4.restype = I
        L.pa_decode_kv4_workspace_size.argtypes = [I]
        L.pa_decode_kv4_workspace_size.restype = Z
        L.pa_prefill_kv4.argtypes = [P] * 4 + [I, P, F] + [I] * 8 + [P, Z, P]
        L.pa_prefill_kv4.restype = I
        L.pa_prefill_kv4_workspace_size.argtypes = [I] * 7
        L.pa_prefill_kv4_workspace_size.restype = Z
        L.pa_decode_weighted.argtypes = [P] * 7 + [F] + [I] * 9 + [P, Z, P]
        L.pa_decode_weighted.restype = I
        L.pa_decode_weighted_workspace_size.argtypes = [I] * 6
        L.pa_decode_weighted_workspace_size.restype = Z
        L.pa_prefill_weights.argtypes = [P] * 5 + [I, F, I, J, J] + [I] * 8 + [P, Z, P]
        L.pa_prefill_weights.restype = I
        L.pa_prefill_weights_workspace_size.argtypes = [I] * 7
        L.pa_prefill_weights_workspace_size.restype = Z
        L.pa_evict_kv.argtypes = [P] * 7 + [I] * 11 + [P, Z, P]
        L.pa_evict_kv.restype = I
        L.pa_evict_kv_workspace_size.argtypes = [I] * 6
        L.pa_evict_kv_workspace_size.restype = Z
        L.pa_compact_kv.argtypes = [P] * 7 + [I, P] + [I] * 7 + [P]
        L.pa_compact_kv.restype = I
        L.pa_prefill_tree.argtypes = [P] * 6 + [I, P, F] + [I] * 8 + [P, Z, P]
        L.pa_prefill_tree.restype = I
        L.pa_prefill_tree_workspace_size.argtypes = [I] * 7
        L.pa_prefill_tree_workspace_size.restype = Z
        L.pa_tree_mask.argtypes = [P] * 3 + [I, I, P]
        L.pa_tree_mask.restype = I
        L.pa_last_device_error.argtypes = [P]
        L.pa_last_device_error.restype = I
        L.pa_selftest_wait_timeout.argtypes = [P]
        L.pa_selftest_wait_timeout.restype = I
        _lib = L
    return _lib


def pa_strerror(status: int) -> str:
    try:
        return lib().pa_strerror(int(status)).decode()
    except ImportError:
        return f"status {status}"


def dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return F16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str) -> int:
    if rc != 0:
        raise PAError(rc, where)
    return rc


# --- the C entry points, same names and argument order ------------------------

def pa_decode(q, k_cache, v_cache, block_table, ctx_lens, out, scale, n_q_heads,
              n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
              num_pages, dtype, partition_tokens=0, workspace=None,
              workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                         _ptr(ctx_lens), _ptr(out), float(scale), n_q_heads,
                         n_kv_heads, head_dim, page_size, batch,
                         max_blocks_per_seq, num_pages, dtype, partition_tokens,
                         _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "pa_decode")


def pa_decode_append(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, out, scale,
                     n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                     num_pages, dtype, partition_tokens=0, workspace=None, workspace_bytes=0,
                     stream=None) -> int:
    rc = lib().pa_decode_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), _ptr(out),
                                float(scale), n_q_heads, n_kv_heads, head_dim, page_size,
                                batch, max_blocks_per_seq, num_pages, dtype, partition_tokens,
                                _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "pa_decode_append")


def pa_decode_static_workspace(q, k_cache, v_cache, block_table, ctx_lens, out,
                               scale, n_q_heads, n_kv_heads, head_dim, page_size,
                               batch, max_blocks_per_seq, num_pages, dtype,
                               partition_tokens=0, stream=None) -> int:
    """pa_decode with its split-K scratch in the library's fixed 16 MiB
    device array: for callers that cannot allocate device memory."""
    rc = lib().pa_decode_static_workspace(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens),
        _ptr(out), float(scale), n_q_heads, n_kv_heads, head_dim, page_size, batch,
        max_blocks_per_seq, num_pages, dtype, partition_tokens, _stream(stream))
    return _check(rc, "pa_decode_static_workspace")


def pa_decode_partition_tokens(batch, n_q_heads, n_kv_heads, head_dim, page_size,
                               max_blocks_per_seq, partition_tokens=0) -> int:
    rc = lib().pa_decode_partition_tokens(batch, n_q_heads, n_kv_heads, head_dim,
                                          page_size, max_blocks_per_seq,
                                          partition_tokens)
    if rc < 0:
        raise PAError(rc, "pa_decode_partition_tokens")
    return rc


def pa_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, page_size,
                             max_blocks_per_seq, partition_tokens=0) -> int:
    return lib().pa_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim,
                                          page_size, max_blocks_per_seq,
                                          partition_tokens)


def pa_merge_partials(partials, ctx_lens, out, batch, n_q_heads, head_dim,
                      n_parts, partition_tokens, stream=None) -> int:
    rc = lib().pa_merge_partials(_ptr(partials), _ptr(ctx_lens), _ptr(out), batch,
                                 n_q_heads, head_dim, n_parts, partition_tokens,
                                 _stream(stream))
    return _check(rc, "pa_merge_partials")


def pa_append_kv(k_new, v_new, k_cache, v_cache, block_table, seq_idx, pos, n_tok,
                 n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                 num_pages, dtype, stream=None) -> int:
    rc = lib().pa_append_kv(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                            _ptr(block_table), _ptr(seq_idx), _ptr(pos), n_tok,
                            n_kv_heads, head_dim, page_size, batch,
                            max_blocks_per_seq, num_pages, dtype, _stream(stream))
    return _check(rc, "pa_append_kv")


def pa_prefill_paged(q, k_cache, v_cache, block_table, ctx_lens, n_new, out, scale,
                     n_q_heads, n_kv_heads, head_dim, page_size, batch,
                     max_blocks_per_seq, num_pages, dtype, stream=None) -> int:
    rc = lib().pa_prefill_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                _ptr(block_table), _ptr(ctx_lens), n_new, _ptr(out),
                                float(scale), n_q_heads, n_kv_heads, head_dim,
                                page_size, batch, max_blocks_per_seq, num_pages,
                                dtype, _stream(stream))
    return _check(rc, "pa_prefill_paged")


def pa_prefill_paged_split(q, k_cache, v_cache, block_table, ctx_lens, n_new, out,
                           scale, n_q_heads, n_kv_heads, head_dim, page_size, batch,
                           max_blocks_per_seq, num_pages, dtype, partition_tokens=0,
                           workspace=None, workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_prefill_paged_split(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), n_new,
        _ptr(out), float(scale), n_q_heads, n_kv_heads, head_dim, page_size, batch,
        max_blocks_per_seq, num_pages, dtype, partition_tokens, _ptr(workspace),
        workspace_bytes, _stream(stream))
    return _check(rc, "pa_prefill_paged_split")


def pa_prefill_partition_tokens(batch, n_new, n_q_heads, n_kv_heads, head_dim, page_size,
                                max_blocks_per_seq, partition_tokens=0) -> int:
    rc = lib().pa_prefill_partition_tokens(batch, n_new, n_q_heads, n_kv_heads, head_dim,
                                           page_size, max_blocks_per_seq, partition_tokens)
    if rc < 0:
        raise PAError(rc, "pa_prefill_partition_tokens")
    return rc


def pa_prefill_workspace_size(batch, n_new, n_q_heads, n_kv_heads, head_dim, page_size,
                              max_blocks_per_seq, partition_tokens=0) -> int:
    return lib().pa_prefill_workspace_size(batch, n_new, n_q_heads, n_kv_heads, head_dim,
                                           page_size, max_blocks_per_seq, partition_tokens)


def pa_decode_cascade(q, k_cache, v_cache, prefix_table, prefix_len, prefix_blocks,
                      block_table, ctx_lens, out, scale, n_q_heads, n_kv_heads, head_dim,
                      page_size, batch, max_blocks_per_seq, num_pages, dtype, partition_tokens,
                      workspace, workspace_bytes, stream=None):
    rc = lib().pa_decode_cascade(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(prefix_table), prefix_len, prefix_blocks,
        _ptr(block_table), _ptr(ctx_lens), _ptr(out), float(scale), n_q_heads, n_kv_heads,
        head_dim, page_size, batch, max_blocks_per_seq, num_pages, dtype, partition_tokens,
        _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "pa_decode_cascade")


def pa_decode_cascade_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, page_size,
                                     prefix_blocks, prefix_len, partition_tokens=0) -> int:
    return lib().pa_decode_cascade_workspace_size(batch, n_q_heads, n_kv_heads, head_dim,
                                                  page_size, prefix_blocks, prefix_len,
                                                  partition_tokens)


def pa_decode_window(q, k_cache, v_cache, block_table, ctx_lens, out, scale, n_q_heads,
                     n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, num_pages,
                     dtype, sink_tokens, window_tokens, partition_tokens=0, workspace=None,
                     workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_decode_window(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), _ptr(out),
        float(scale), n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
        num_pages, dtype, sink_tokens, window_tokens, partition_tokens, _ptr(workspace),
        workspace_bytes, _stream(stream))
    return _check(rc, "pa_decode_window")


def pa_decode_window_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, page_size,
                                    max_blocks_per_seq, sink_tokens, window_tokens,
                                    partition_tokens=0) -> int:
    return lib().pa_decode_window_workspace_size(batch, n_q_heads, n_kv_heads, head_dim,
                                                 page_size, max_blocks_per_seq, sink_tokens,
                                                 window_tokens, partition_tokens)


def _i32_host(a):
    """A C-contiguous host int32 numpy array (tables and page lists)."""
    import numpy as np
    a = np.ascontiguousarray(a, dtype=np.int32)
    return a, a.ctypes.data


def pa_pool_create(num_pages) -> int:
    """A page pool handle (an opaque pointer as int); raises on failure."""
    h = lib().pa_pool_create(int(num_pages))
    if not h:
        raise PAError(-5, "pa_pool_create")
    return h


def pa_pool_destroy(pool) -> None:
    lib().pa_pool_destroy(pool)


def pa_pool_free_pages(pool) -> int:
    return lib().pa_pool_free_pages(pool)


def pa_pool_refcount(pool, page) -> int:
    rc = lib().pa_pool_refcount(pool, int(page))
    if rc < 0:
        raise PAError(rc, "pa_pool_refcount")
    return rc


def pa_pool_alloc(pool, n):
    """n fresh pages as an int32 numpy array."""
    import numpy as np
    out = np.empty(int(n), dtype=np.int32)
    _check(lib().pa_pool_alloc(pool, int(n), out.ctypes.data if n else None), "pa_pool_alloc")
    return out


def pa_pool_share(pool, pages) -> int:
    a, ptr = _i32_host(pages)
    return _check(lib().pa_pool_share(pool, ptr if a.size else None, a.size), "pa_pool_share")


def pa_pool_release(pool, pages) -> int:
    a, ptr = _i32_host(pages)
    return _check(lib().pa_pool_release(pool, ptr if a.size else None, a.size),
                  "pa_pool_release")


def pa_pool_prepare_append(pool, table_row, page_size, pos):
    """table_row: host int32 numpy array, updated in place.  Returns
    (copy_src, copy_dst): a page pair for pa_copy_pages, or (-1, -1)."""
    import numpy as np
    assert isinstance(table_row, np.ndarray) and table_row.dtype == np.int32 \
        and table_row.flags.c_contiguous
    src, dst = ctypes.c_int32(-1), ctypes.c_int32(-1)
    rc = lib().pa_pool_prepare_append(pool, table_row.ctypes.data, table_row.size,
                                      int(page_size), int(pos), ctypes.addressof(src),
                                      ctypes.addressof(dst))
    if rc < 0:
        raise PAError(rc, "pa_pool_prepare_append")
    return src.value, dst.value


def pa_copy_pages(k_cache, v_cache, src, dst, n, n_kv_heads, head_dim, page_size, num_pages,
                  dtype, stream=None) -> int:
    rc = lib().pa_copy_pages(_ptr(k_cache), _ptr(v_cache), _ptr(src), _ptr(dst), n,
                             n_kv_heads, head_dim, page_size, num_pages, dtype,
                             _stream(stream))
    return _check(rc, "pa_copy_pages")


def pa_topm_workspace_size(n_layers, n_heads, n_tokens) -> int:
    return lib().pa_topm_workspace_size(n_layers, n_heads, n_tokens)


def pa_topm_retain(scores, n_layers, n_heads, n_tokens, current, budget, keep,
                   kept_per_head=None, workspace=None, workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_topm_retain(_ptr(scores), n_layers, n_heads, n_tokens, current, int(budget),
                              _ptr(keep), _ptr(kept_per_head), _ptr(workspace),
                              workspace_bytes, _stream(stream))
    return _check(rc, "pa_topm_retain")


def pa_append_kv_rope(k_new, v_new, q, k_cache, v_cache, q_out, block_table, seq_idx, pos,
                      cos_sin, n_tok, k_stride, v_stride, q_stride, n_q_heads, n_kv_heads,
                      head_dim, page_size, batch, max_blocks_per_seq, num_pages, max_pos,
                      rot_dim, interleaved, dtype, stream=None) -> int:
    rc = lib().pa_append_kv_rope(
        _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(q_out),
        _ptr(block_table), _ptr(seq_idx), _ptr(pos), _ptr(cos_sin), n_tok, k_stride, v_stride,
        q_stride, n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
        num_pages, max_pos, rot_dim, int(interleaved), dtype, _stream(stream))
    return _check(rc, "pa_append_kv_rope")


def pa_append_kv_rope_at(k_new, v_new, q, k_cache, v_cache, q_out, block_table, seq_idx, pos,
                         rope_pos, cos_sin, n_tok, k_stride, v_stride, q_stride, n_q_heads,
                         n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, num_pages,
                         max_pos, rot_dim, interleaved, dtype, stream=None) -> int:
    rc = lib().pa_append_kv_rope_at(
        _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(q_out),
        _ptr(block_table), _ptr(seq_idx), _ptr(pos), _ptr(rope_pos), _ptr(cos_sin), n_tok,
        k_stride, v_stride, q_stride, n_q_heads, n_kv_heads, head_dim, page_size, batch,
        max_blocks_per_seq, num_pages, max_pos, rot_dim, int(interleaved), dtype,
        _stream(stream))
    return _check(rc, "pa_append_kv_rope_at")


def pa_kv4_block_bytes(head_dim) -> int:
    return lib().pa_kv4_block_bytes(head_dim)


def pa_append_kv4(k_new, v_new, q, kv_cache, q_out, block_table, seq_idx, pos, cos_sin, n_tok,
                  k_stride, v_stride, q_stride, n_q_heads, n_kv_heads, head_dim, page_size,
                  batch, max_blocks_per_seq, num_pages, max_pos, rot_dim, interleaved, dtype,
                  stream=None) -> int:
    rc = lib().pa_append_kv4(
        _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(kv_cache), _ptr(q_out), _ptr(block_table),
        _ptr(seq_idx), _ptr(pos), _ptr(cos_sin), n_tok, k_stride, v_stride, q_stride, n_q_heads,
        n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, num_pages, max_pos, rot_dim,
        int(interleaved), dtype, _stream(stream))
    return _check(rc, "pa_append_kv4")


def pa_read_kv4(kv_cache, block_table, seq_idx, pos, k_out, v_out, n_tok, n_kv_heads, head_dim,
                page_size, batch, max_blocks_per_seq, num_pages, dtype, stream=None) -> int:
    rc = lib().pa_read_kv4(
        _ptr(kv_cache), _ptr(block_table), _ptr(seq_idx), _ptr(pos), _ptr(k_out), _ptr(v_out),
        n_tok, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, num_pages, dtype,
        _stream(stream))
    return _check(rc, "pa_read_kv4")


def pa_copy_pages_kv4(kv_cache, src, dst, n, n_kv_heads, head_dim, page_size, num_pages,
                      stream=None) -> int:
    rc = lib().pa_copy_pages_kv4(_ptr(kv_cache), _ptr(src), _ptr(dst), n, n_kv_heads, head_dim,
                                 page_size, num_pages, _stream(stream))
    return _check(rc, "pa_copy_pages_kv4")


def pa_decode_kv4(q, kv_cache, block_table, ctx_lens, out, scale, n_q_heads, n_kv_heads,
                  head_dim, page_size, batch, max_blocks_per_seq, num_pages, dtype,
                  workspace=None, workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_decode_kv4(
        _ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(ctx_lens), _ptr(out), float(scale),
        n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, num_pages, dtype,
        _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "pa_decode_kv4")


def pa_decode_kv4_workspace_size(head_dim) -> int:
    return lib().pa_decode_kv4_workspace_size(head_dim)


def pa_prefill_kv4(q, kv_cache, block_table, ctx_lens, n_new, out, scale, n_q_heads, n_kv_heads,
                   head_dim, page_size, batch, max_blocks_per_seq, num_pages, dtype,
                   workspace=None, workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_prefill_kv4(
        _ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(ctx_lens), n_new, _ptr(out),
        float(scale), n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
        num_pages, dtype, _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "pa_prefill_kv4")


def pa_prefill_kv4_workspace_size(batch, n_new, n_q_heads, n_kv_heads, head_dim, page_size,
                                  max_blocks_per_seq) -> int:
    return lib().pa_prefill_kv4_workspace_size(batch, n_new, n_q_heads, n_kv_heads, head_dim,
                                               page_size, max_blocks_per_seq)


def pa_decode_weighted(q, k_cache, v_cache, weights, block_table, ctx_lens, out, scale, fresh,
                       n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                       num_pages, dtype, workspace=None, workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_decode_weighted(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(weights), _ptr(block_table), _ptr(ctx_lens),
        _ptr(out), float(scale), fresh, n_q_heads, n_kv_heads, head_dim, page_size, batch,
        max_blocks_per_seq, num_pages, dtype, _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "pa_decode_weighted")


def pa_decode_weighted_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, page_size,
                                      max_blocks_per_seq) -> int:
    return lib().pa_decode_weighted_workspace_size(batch, n_q_heads, n_kv_heads, head_dim,
                                                   page_size, max_blocks_per_seq)


def pa_prefill_weights(q, k_cache, weights, block_table, ctx_lens, n_new, scale, fresh,
                       q_batch_stride, q_token_stride, n_q_heads, n_kv_heads, head_dim, page_size,
                       batch, max_blocks_per_seq, num_pages, dtype, workspace=None,
                       workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_prefill_weights(
        _ptr(q), _ptr(k_cache), _ptr(weights), _ptr(block_table), _ptr(ctx_lens), n_new,
        float(scale), fresh, q_batch_stride, q_token_stride, n_q_heads, n_kv_heads, head_dim,
        page_size, batch, max_blocks_per_seq, num_pages, dtype, _ptr(workspace), workspace_bytes,
        _stream(stream))
    return _check(rc, "pa_prefill_weights")


def pa_prefill_weights_workspace_size(batch, n_new, n_q_heads, n_kv_heads, head_dim, page_size,
                                      max_blocks_per_seq) -> int:
    return lib().pa_prefill_weights_workspace_size(batch, n_new, n_q_heads, n_kv_heads, head_dim,
                                                   page_size, max_blocks_per_seq)


def pa_evict_kv(k_cache, v_cache, weights, block_table, ctx_lens, dst_table, new_lens, budget,
                sink_tokens, recent_tokens, n_kv_heads, head_dim, page_size, batch,
                max_blocks_per_seq, dst_blocks_per_seq, num_pages, dtype, workspace=None,
                workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_evict_kv(
        _ptr(k_cache), _ptr(v_cache), _ptr(weights), _ptr(block_table), _ptr(ctx_lens),
        _ptr(dst_table), _ptr(new_lens), budget, sink_tokens, recent_tokens, n_kv_heads, head_dim,
        page_size, batch, max_blocks_per_seq, dst_blocks_per_seq, num_pages, dtype,
        _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "pa_evict_kv")


def pa_evict_kv_workspace_size(batch, n_kv_heads, head_dim, page_size, max_blocks_per_seq,
                               budget) -> int:
    return lib().pa_evict_kv_workspace_size(batch, n_kv_heads, head_dim, page_size,
                                            max_blocks_per_seq, budget)


def pa_compact_kv(k_cache, v_cache, weights, block_table, ctx_lens, keep, n_keep, max_keep,
                  new_lens, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, num_pages,
                  dtype, stream=None) -> int:
    rc = lib().pa_compact_kv(
        _ptr(k_cache), _ptr(v_cache), _ptr(weights), _ptr(block_table), _ptr(ctx_lens),
        _ptr(keep), _ptr(n_keep), max_keep, _ptr(new_lens), n_kv_heads, head_dim, page_size,
        batch, max_blocks_per_seq, num_pages, dtype, _stream(stream))
    return _check(rc, "pa_compact_kv")


def pa_prefill_tree(q, k_cache, v_cache, block_table, ctx_lens, mask, n_new, out, scale,
                    n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                    num_pages, dtype, workspace=None, workspace_bytes=0, stream=None) -> int:
    rc = lib().pa_prefill_tree(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), _ptr(mask),
        n_new, _ptr(out), float(scale), n_q_heads, n_kv_heads, head_dim, page_size, batch,
        max_blocks_per_seq, num_pages, dtype, _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "pa_prefill_tree")


def pa_prefill_tree_workspace_size(batch, n_new, n_q_heads, n_kv_heads, head_dim, page_size,
                                   max_blocks_per_seq) -> int:
    return lib().pa_prefill_tree_workspace_size(batch, n_new, n_q_heads, n_kv_heads, head_dim,
                                                page_size, max_blocks_per_seq)


def pa_tree_mask(parents, mask, depth, batch, n_new, stream=None) -> int:
    rc = lib().pa_tree_mask(_ptr(parents), _ptr(mask), _ptr(depth), batch, n_new, _stream(stream))
    return _check(rc, "pa_tree_mask")


def pa_last_device_error(stream=None) -> int:
    """Synchronises the stream; returns and clears the device status word."""
    return lib().pa_last_device_error(_stream(stream))


def pa_selftest_wait_timeout(stream=None):
    """One warp waits on a barrier phase nothing completes; the bounded wait
    gives up after 2 s and records PA_ERR_TIMEOUT."""
    return _check(lib().pa_selftest_wait_timeout(_stream(stream)), "pa_selftest_wait_timeout")


# --- tensor-shaped conveniences (allocation by torch, compute by libpa) ------

def decode(q, k_cache, v_cache, block_table, ctx_lens, scale, partition_tokens=0,
           out=None, workspace=None, stream=None):
    """q [B, h_q, D]; caches [pages, h_kv, 16, D]; block_table int32 [B, max_blocks];
    ctx_lens int32 [B].  Returns fp32 [B, h_q, D]."""
    import torch
    B, hq, D = q.shape
    pages, hkv, P, D2 = k_cache.shape
    assert D2 == D and block_table.shape[0] == B
    mb = block_table.shape[1]
    if out is None:
        out = torch.empty((B, hq, D), dtype=torch.float32, device=q.device)
    ws_bytes = pa_decode_workspace_size(B, hq, hkv, D, P, mb, partition_tokens)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes // 4, dtype=torch.float32, device=q.device)
    pa_decode(q, k_cache, v_cache, block_table, ctx_lens, out, scale, hq, hkv, D, P,
              B, mb, pages, dtype_code(q), partition_tokens, workspace,
              ws_bytes, stream)
    return out


def decode_append(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, scale,
                  partition_tokens=0, out=None, workspace=None, stream=None):
    """pa_decode_append on tensors: q [B, h_q, D]; k_new, v_new [B, h_kv, D], the
    step's token of each sequence, stored at position ctx_lens[b] - 1 (the
    caches are written in place); ctx_lens counts that token.  Returns fp32
    [B, h_q, D]."""
    import torch
    B, hq, D = q.shape
    pages, hkv, P, D2 = k_cache.shape
    assert D2 == D and block_table.shape[0] == B and tuple(k_new.shape) == (B, hkv, D)
    mb = block_table.shape[1]
    if out is None:
        out = torch.empty((B, hq, D), dtype=torch.float32, device=q.device)
    ws_bytes = pa_decode_workspace_size(B, hq, hkv, D, P, mb, partition_tokens)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes // 4, dtype=torch.float32, device=q.device)
    pa_decode_append(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, out, scale, hq,
                     hkv, D, P, B, mb, pages, dtype_code(q), partition_tokens, workspace,
                     ws_bytes, stream)
    return out


def append_kv(k_new, v_new, k_cache, v_cache, block_table, seq_idx, pos, stream=None):
    n_tok, hkv, D = k_new.shape
    pages, _, P, _ = k_cache.shape
    B, mb = block_table.shape
    pa_append_kv(k_new, v_new, k_cache, v_cache, block_table, seq_idx, pos, n_tok,
                 hkv, D, P, B, mb, pages, dtype_code(k_new), stream)


def prefill(q, k_cache, v_cache, block_table, ctx_lens, scale, out=None, stream=None):
    """q [B, n_new, h_q, D]; ctx_lens = cached tokens before the chunk."""
    import torch
    B, n_new, hq, D = q.shape
    pages, hkv, P, _ = k_cache.shape
    mb = block_table.shape[1]
    if out is None:
        out = torch.empty((B, n_new, hq, D), dtype=torch.float32, device=q.device)
    pa_prefill_paged(q, k_cache, v_cache, block_table, ctx_lens, n_new, out, scale,
                     hq, hkv, D, P, B, mb, pages, dtype_code(q), stream)
    return out


def prefill_split(q, k_cache, v_cache, block_table, ctx_lens, scale, partition_tokens=0,
                  out=None, workspace=None, stream=None):
    """pa_prefill_paged_split on tensors: q [B, n_new, h_q, D] (e.g. the gamma
    drafted tokens of a speculative-decoding verify step); ctx_lens = cached
    tokens before the chunk.  Returns fp32 [B, n_new, h_q, D]."""
    import torch
    B, n_new, hq, D = q.shape
    pages, hkv, P, _ = k_cache.shape
    mb = block_table.shape[1]
    if out is None:
        out = torch.empty((B, n_new, hq, D), dtype=torch.float32, device=q.device)
    ws_bytes = pa_prefill_workspace_size(B, n_new, hq, hkv, D, P, mb, partition_tokens)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes // 4, dtype=torch.float32, device=q.device)
    pa_prefill_paged_split(q, k_cache, v_cache, block_table, ctx_lens, n_new, out, scale,
                           hq, hkv, D, P, B, mb, pages, dtype_code(q), partition_tokens,
                           workspace, ws_bytes, stream)
    return out


def decode_cascade(q, k_cache, v_cache, prefix_table, prefix_len, block_table, ctx_lens,
                   scale, partition_tokens=0, out=None, workspace=None, stream=None):
    """pa_decode_cascade on tensors: q [B, h_q, D], one query per fork of a
    shared prefix of prefix_len tokens (pages prefix_table, int32 [n]);
    block_table [B, max_blocks] and ctx_lens [B] hold each fork's own tokens
    after the prefix.  Returns fp32 [B, h_q, D]."""
    import torch
    B, hq, D = q.shape
    pages, hkv, P, _ = k_cache.shape
    mb = block_table.shape[1]
    n_pref = prefix_table.shape[0]
    if out is None:
        out = torch.empty((B, hq, D), dtype=torch.float32, device=q.device)
    ws_bytes = pa_decode_cascade_workspace_size(B, hq, hkv, D, P, n_pref, prefix_len,
                                                partition_tokens)
    if workspace is None:
        workspace = torch.empty(max(1, ws_bytes // 4), dtype=torch.float32, device=q.device)
    pa_decode_cascade(q, k_cache, v_cache, prefix_table, prefix_len, n_pref, block_table,
                      ctx_lens, out, scale, hq, hkv, D, P, B, mb, pages, dtype_code(q),
                      partition_tokens, workspace, ws_bytes, stream)
    return out


def decode_window(q, k_cache, v_cache, block_table, ctx_lens, scale, sink_tokens,
                  window_tokens, partition_tokens=0, out=None, workspace=None, stream=None):
    """pa_decode_window on tensors (shapes as decode()): attends keys t < sink_tokens
    and t >= T - window_tokens of each sequence.  Returns fp32 [B, h_q, D]."""
    import torch
    B, hq, D = q.shape
    pages, hkv, P, _ = k_cache.shape
    mb = block_table.shape[1]
    if out is None:
        out = torch.empty((B, hq, D), dtype=torch.float32, device=q.device)
    ws_bytes = pa_decode_window_workspace_size(B, hq, hkv, D, P, mb, sink_tokens,
                                               window_tokens, partition_tokens)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes // 4, dtype=torch.float32, device=q.device)
    pa_decode_window(q, k_cache, v_cache, block_table, ctx_lens, out, scale, hq, hkv, D, P,
                     B, mb, pages, dtype_code(q), sink_tokens, window_tokens,
                     partition_tokens, workspace, ws_bytes, stream)
    return out


def topm_retain(scores, current, budget, keep=None, kept_per_head=None, workspace=None,
                stream=None):
    """pa_topm_retain on tensors: scores float32 [L, H, N] on the device.
    Returns (keep uint8 [L, H, N], kept_per_head int32 [L, H])."""
    import torch
    L, H, N = scores.shape
    if keep is None:
        keep = torch.empty((L, H, N), dtype=torch.uint8, device=scores.device)
    if kept_per_head is None:
        kept_per_head = torch.empty((L, H), dtype=torch.int32, device=scores.device)
    ws_bytes = pa_topm_workspace_size(L, H, N)
    if workspace is None:
        workspace = torch.empty(max(1, ws_bytes // 4), dtype=torch.int32, device=scores.device)
    pa_topm_retain(scores, L, H, N, current, budget, keep, kept_per_head, workspace, ws_bytes,
                   stream)
    return keep, kept_per_head


# --- rotated appends and the 4-bit cache --------------------------------------
# A decode step makes these calls once a layer, so their checks are kept cheap: a
# tensor that is as it should be costs four attribute reads.

def _bad(t, name, dtype, shape, index):
    return ValueError(
        f"{name}: want a contiguous {dtype} tensor of shape "
        f"{tuple('*' if w is None else w for w in shape)} on cuda:{index}, got {t.dtype} "
        f"{tuple(t.shape)} with strides {tuple(t.stride())} on {t.device}")


def _want(t, name, dtype, shape, index):
    """t is a contiguous tensor of this type and shape on CUDA device `index`."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or \
            t.get_device() != index:
        raise _bad(t, name, dtype, shape, index)


def _want_2d(t, name, dtype, rows, index):
    """As _want, of any number of columns; returns (rows, columns)."""
    if t.dtype is not dtype or t.dim() != 2 or not t.is_contiguous() or \
            t.get_device() != index or (rows is not None and t.shape[0] != rows):
        raise _bad(t, name, dtype, (rows, None), index)
    return t.shape


def _token_stride(t, name, dtype, index, n_tok, heads, D):
    """Elements from one token's rows [heads, D] to the next one's."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != (n_tok, heads, D):
        raise ValueError(f"{name}: want {dtype} [{n_tok}, {heads}, {D}] on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    token, head, one = t.stride()
    if one != 1 or (heads > 1 and head != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous rows (strides "
                         f"{(token, head, one)}); call .contiguous()")
    return token if n_tok > 1 else heads * D


def _device_index(t):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"tensors must be on a CUDA device, got {t.device}")
    return index


# What an empty tensor, which has no address, is passed on as: the library wants every
# pointer, and checks the other arguments, of calls with nothing to do too.
_NOTHING = 16


class _On:
    """Makes device `index` current, and `stream` (a torch stream or a handle, if
    given) the current stream there, so that what a call allocates belongs to the
    stream it runs on.  Yields the stream's handle."""

    def __init__(self, index, stream):
        self.index, self.stream, self.guards = index, stream, []

    def __enter__(self):
        import torch
        stream = self.stream
        if stream is not None and not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(stream, device=self.index)
        if stream is not None and stream.device_index != self.index:
            raise ValueError(f"stream of cuda:{stream.device_index} for tensors on "
                             f"cuda:{self.index}")
        self.guards.append(torch.cuda.device(self.index))
        if stream is not None:
            self.guards.append(torch.cuda.stream(stream))
        for g in self.guards:
            g.__enter__()
        return (stream or torch.cuda.current_stream()).cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _elsewhere(index, stream):
    """True unless the call is for the current device and its current stream (the
    usual case, found out cheaply); then it is made again under _On."""
    import torch
    return stream is not None or torch._C._cuda_getDevice() != index


def rope_table(max_pos, rot_dim, base=10000.0, device="cuda"):
    """cos_sin of the rotated appends, float32 [max_pos, rot_dim]: the cosines of
    position * base^(-2 i / rot_dim) for i < rot_dim / 2, then the sines (angles
    in float64, so far positions keep their digits)."""
    import torch
    inv = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    ang = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((ang.cos(), ang.sin()), -1).float()


_KV4_HEAD_DIM = {16 * d + 128: d for d in (64, 128)}  # block bytes -> head_dim


def kv4_cache(num_pages, n_kv_heads, head_dim, device="cuda"):
    """An empty 4-bit cache: uint8 [num_pages, n_kv_heads, block bytes]."""
    import torch
    block = pa_kv4_block_bytes(head_dim)
    if not block:
        raise PAError(-3, "kv4_cache")
    return torch.zeros((num_pages, n_kv_heads, block), dtype=torch.uint8, device=device)


def _kv4_dims(kv_cache, index):
    """num_pages, n_kv_heads and head_dim of a 4-bit cache tensor on device `index`."""
    import torch
    shape = kv_cache.shape
    D = _KV4_HEAD_DIM.get(shape[2]) if len(shape) == 3 else None
    if D is None or kv_cache.dtype is not torch.uint8 or not kv_cache.is_contiguous() or \
            kv_cache.get_device() != index:
        raise ValueError("kv_cache: want contiguous uint8 [num_pages, n_kv_heads, "
                         f"pa_kv4_block_bytes(head_dim)] on cuda:{index}, got {kv_cache.dtype} "
                         f"{tuple(shape)} on {kv_cache.device}")
    return shape[0], shape[1], D


def _append(entry, where, k_new, v_new, q, q_out, caches, num_pages, page_size, hkv_cache, D_cache,
            block_table, seq_idx, pos, cos_sin, interleaved, index, rope_pos=None):
    """The common part of the two rotated appends, on the current stream of device
    `index`: `entry` with `caches` (pointers)."""
    import torch
    if k_new.dim() != 3:
        raise ValueError(f"k_new: want [n_tok, n_kv_heads, head_dim], got {tuple(k_new.shape)}")
    n_tok, hkv, D = k_new.shape
    if hkv != hkv_cache or D != D_cache:
        raise ValueError(f"the cache holds {hkv_cache} heads of head_dim {D_cache}, k_new has "
                         f"{hkv} of {D}")
    dtype, i32 = k_new.dtype, torch.int32
    ks = _token_stride(k_new, "k_new", dtype, index, n_tok, hkv, D)
    vs = _token_stride(v_new, "v_new", dtype, index, n_tok, hkv, D)
    batch, max_blocks = _want_2d(block_table, "block_table", i32, None, index)
    _want(seq_idx, "seq_idx", i32, (n_tok,), index)
    _want(pos, "pos", i32, (n_tok,), index)
    max_pos = rot = hq = qs = 0
    table = q_in = q_to = None
    if cos_sin is not None:
        max_pos, rot = _want_2d(cos_sin, "cos_sin", torch.float32, None, index)
        table = cos_sin.data_ptr() or _NOTHING
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q: want [n_tok, n_q_heads, head_dim], got {tuple(q.shape)}")
        hq = q.shape[1]
        qs = _token_stride(q, "q", dtype, index, n_tok, hq, D)
        if q_out is None:
            q_out = torch.empty((n_tok, hq, D), dtype=dtype, device=q.device)
        else:
            _want(q_out, "q_out", dtype, (n_tok, hq, D), index)
        q_in, q_to = q.data_ptr() or _NOTHING, q_out.data_ptr() or _NOTHING
    elif q_out is not None:
        raise ValueError("q_out without q")
    k, v, seqs, at = k_new.data_ptr(), v_new.data_ptr(), seq_idx.data_ptr(), pos.data_ptr()
    if n_tok == 0:
        k = v = seqs = at = _NOTHING
    turn = ()
    if rope_pos is not None:
        _want(rope_pos, "rope_pos", i32, (n_tok,), index)
        turn = (rope_pos.data_ptr() or _NOTHING,)
    rc = entry(k, v, q_in, *caches, q_to, block_table.data_ptr(), seqs, at, *turn, table, n_tok,
               ks, vs, qs, hq, hkv, D, page_size, batch, max_blocks, num_pages, max_pos, rot,
               bool(interleaved), dtype_code(k_new), torch._C._cuda_getCurrentRawStream(index))
    if rc:
        raise PAError(rc, where)
    return q_out


def append_kv_rope(k_new, v_new, k_cache, v_cache, block_table, seq_idx, pos, cos_sin, q=None,
                   q_out=None, interleaved=False, stream=None, rope_pos=None):
    """pa_append_kv_rope on tensors: k_new, v_new [n_tok, h_kv, D] and q
    [n_tok, h_q, D] may be views with any token stride (a fused projection's
    output); cos_sin float32 [max_pos, rot_dim] (rope_table).  Writes the caches
    [pages, h_kv, 16, D]; returns the rotated q ([n_tok, h_q, D], q_out if
    given), or None without q.  rope_pos int32 [n_tok]: positions to rotate by, where
    they are not pos (pa_append_kv_rope_at: the tokens of a drafted tree)."""
    index = _device_index(k_new)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return append_kv_rope(k_new, v_new, k_cache, v_cache, block_table, seq_idx, pos,
                                  cos_sin, q, q_out, interleaved, rope_pos=rope_pos)
    if cos_sin is None or k_cache.dim() != 4:
        raise ValueError("append_kv_rope wants cos_sin and caches [pages, h_kv, 16, D]")
    pages, hkv, P, D = shape = k_cache.shape
    _want(k_cache, "k_cache", k_new.dtype, shape, index)
    _want(v_cache, "v_cache", k_new.dtype, shape, index)
    where = "pa_append_kv_rope" if rope_pos is None else "pa_append_kv_rope_at"
    return _append(getattr(lib(), where), where, k_new, v_new, q, q_out,
                   (k_cache.data_ptr(), v_cache.data_ptr()), pages, P, hkv, D, block_table,
                   seq_idx, pos, cos_sin, interleaved, index, rope_pos)


def append_kv4(k_new, v_new, kv_cache, block_table, seq_idx, pos, cos_sin=None, q=None,
               q_out=None, interleaved=False, stream=None):
    """pa_append_kv4 on tensors: as append_kv_rope, into a 4-bit cache (kv4_cache);
    without cos_sin nothing is rotated.  The dtype of k_new is that of the cache's
    scales and zeros: keep to one for a cache.  Returns the rotated q, or None."""
    index = _device_index(k_new)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return append_kv4(k_new, v_new, kv_cache, block_table, seq_idx, pos, cos_sin, q,
                              q_out, interleaved)
    pages, hkv, D = _kv4_dims(kv_cache, index)
    return _append(lib().pa_append_kv4, "pa_append_kv4", k_new, v_new, q, q_out,
                   (kv_cache.data_ptr(),), pages, 16, hkv, D, block_table, seq_idx, pos, cos_sin,
                   interleaved, index)


def read_kv4(kv_cache, block_table, seq_idx, pos, dtype=None, k_out=None, v_out=None,
             stream=None):
    """pa_read_kv4 on tensors: the K and V rows of tokens (seq_idx[j], pos[j]) as
    values, each [n_tok, h_kv, D] of dtype (torch.bfloat16 or torch.float16, the
    type the cache was written with; k_out's if given)."""
    import torch
    index = _device_index(kv_cache)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return read_kv4(kv_cache, block_table, seq_idx, pos, dtype, k_out, v_out)
    pages, hkv, D = _kv4_dims(kv_cache, index)
    batch, max_blocks = _want_2d(block_table, "block_table", torch.int32, None, index)
    n_tok = seq_idx.numel()
    _want(seq_idx, "seq_idx", torch.int32, (n_tok,), index)
    _want(pos, "pos", torch.int32, (n_tok,), index)
    if dtype is None:
        if k_out is None and v_out is None:
            raise ValueError("read_kv4 wants dtype, k_out or v_out")
        dtype = (k_out if k_out is not None else v_out).dtype
    shape = (n_tok, hkv, D)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=kv_cache.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=kv_cache.device)
    _want(k_out, "k_out", dtype, shape, index)
    _want(v_out, "v_out", dtype, shape, index)
    ptrs = (_NOTHING,) * 4 if n_tok == 0 else (seq_idx.data_ptr(), pos.data_ptr(),
                                               k_out.data_ptr(), v_out.data_ptr())
    rc = lib().pa_read_kv4(kv_cache.data_ptr(), block_table.data_ptr(), *ptrs, n_tok, hkv, D, 16,
                           batch, max_blocks, pages, dtype_code(k_out),
                           torch._C._cuda_getCurrentRawStream(index))
    if rc:
        raise PAError(rc, "pa_read_kv4")
    return k_out, v_out


def copy_pages_kv4(kv_cache, src, dst, stream=None):
    """pa_copy_pages_kv4 on tensors: page src[i] to page dst[i] (int32, on the device)."""
    import torch
    index = _device_index(kv_cache)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return copy_pages_kv4(kv_cache, src, dst)
    pages, hkv, D = _kv4_dims(kv_cache, index)
    n = src.numel()
    _want(src, "src", torch.int32, (n,), index)
    _want(dst, "dst", torch.int32, (n,), index)
    _check(lib().pa_copy_pages_kv4(kv_cache.data_ptr(), src.data_ptr() or _NOTHING,
                                   dst.data_ptr() or _NOTHING, n, hkv, D, 16, pages,
                                   torch._C._cuda_getCurrentRawStream(index)),
           "pa_copy_pages_kv4")


def _attention_args(q, kv_cache, block_table, ctx_lens, out, out_dtype, workspace, index):
    """What decode_kv4 and prefill_kv4 have in common: the checks, and (B, h_q, D,
    pages, h_kv, max_blocks, out)."""
    import torch
    shape = q.shape
    B, hq, D = shape[0], shape[-2], shape[-1]
    pages, hkv, D4 = _kv4_dims(kv_cache, index)
    if D4 != D:
        raise ValueError(f"kv_cache holds head_dim {D4}, q has {D}")
    if not q.is_contiguous():
        raise ValueError(f"q: want a contiguous tensor, got strides {tuple(q.stride())}")
    _, mb = _want_2d(block_table, "block_table", torch.int32, B, index)
    _want(ctx_lens, "ctx_lens", torch.int32, (B,), index)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=q.device)
    else:
        _want(out, "out", out_dtype, shape, index)
    if workspace is not None and (workspace.get_device() != index or
                                  not workspace.is_contiguous()):
        raise ValueError(f"workspace: want a contiguous tensor on cuda:{index}")
    return B, hq, D, pages, hkv, mb, out


def decode_kv4(q, kv_cache, block_table, ctx_lens, scale, out=None, workspace=None, stream=None):
    """pa_decode_kv4 on tensors: q [B, h_q, D]; kv_cache uint8 [pages, h_kv, block]
    (kv4_cache), written by append_kv4 with q's dtype; block_table int32
    [B, max_blocks]; ctx_lens int32 [B].  Returns fp32 [B, h_q, D].  workspace:
    any tensor of pa_decode_kv4_workspace_size(D) bytes, not shared with a call
    that may run at the same time."""
    import torch
    index = _device_index(q)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return decode_kv4(q, kv_cache, block_table, ctx_lens, scale, out, workspace)
    if q.dim() != 3:
        raise ValueError(f"q: want [B, h_q, D], got {tuple(q.shape)}")
    B, hq, D, pages, hkv, mb, out = _attention_args(q, kv_cache, block_table, ctx_lens, out,
                                                    torch.float32, workspace, index)
    if workspace is None:
        workspace = torch.empty(pa_decode_kv4_workspace_size(D), dtype=torch.uint8,
                                device=q.device)
    rc = lib().pa_decode_kv4(q.data_ptr(), kv_cache.data_ptr(), block_table.data_ptr(),
                             ctx_lens.data_ptr(), out.data_ptr(), scale, hq, hkv, D, 16, B, mb,
                             pages, dtype_code(q), workspace.data_ptr(), workspace.nbytes,
                             torch._C._cuda_getCurrentRawStream(index))
    if rc:
        raise PAError(rc, "pa_decode_kv4")
    return out


def prefill_kv4(q, kv_cache, block_table, ctx_lens, scale, out=None, workspace=None,
                stream=None):
    """pa_prefill_kv4 on tensors: q [B, n_new, h_q, D], the chunk's queries, whose
    K/V rows append_kv4 has stored at positions ctx_lens[b] ..; ctx_lens = tokens
    cached before the chunk.  Returns [B, n_new, h_q, D] in q's dtype.  workspace:
    any tensor of pa_prefill_kv4_workspace_size(...) bytes, as in decode_kv4."""
    import torch
    index = _device_index(q)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return prefill_kv4(q, kv_cache, block_table, ctx_lens, scale, out, workspace)
    if q.dim() != 4:
        raise ValueError(f"q: want [B, n_new, h_q, D], got {tuple(q.shape)}")
    n_new = q.shape[1]
    B, hq, D, pages, hkv, mb, out = _attention_args(q, kv_cache, block_table, ctx_lens, out,
                                                    q.dtype, workspace, index)
    if workspace is None:
        workspace = torch.empty(pa_prefill_kv4_workspace_size(B, n_new, hq, hkv, D, 16, mb),
                                dtype=torch.uint8, device=q.device)
    q_in, q_to = (q.data_ptr(), out.data_ptr()) if n_new else (_NOTHING, _NOTHING)
    rc = lib().pa_prefill_kv4(q_in, kv_cache.data_ptr(), block_table.data_ptr(),
                              ctx_lens.data_ptr(), n_new, q_to, scale, hq, hkv, D, 16,
                              B, mb, pages, dtype_code(q), workspace.data_ptr(), workspace.nbytes,
                              torch._C._cuda_getCurrentRawStream(index))
    if rc:
        raise PAError(rc, "pa_prefill_kv4")
    return out


# --- eviction by gathered attention weight, and trees of drafted tokens --------

def weight_pool(num_pages, n_kv_heads, device="cuda"):
    """A pool of gathered attention weights beside a 16-bit cache: float32
    [num_pages, n_kv_heads, 16]."""
    import torch
    return torch.zeros((num_pages, n_kv_heads, 16), dtype=torch.float32, device=device)


def _cache_dims(k_cache, v_cache, dtype, index):
    """num_pages, n_kv_heads and head_dim of 16-bit caches on device `index`; v_cache may
    be None."""
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError(f"k_cache: want [pages, h_kv, 16, D], got {tuple(shape)}")
    _want(k_cache, "k_cache", dtype, shape, index)
    if v_cache is not None:
        _want(v_cache, "v_cache", dtype, shape, index)
    if shape[2] != 16:
        raise PAError(-4, "caches")
    return shape[0], shape[1], shape[3]


def _scratch(workspace, need, device, index):
    """(pointer, bytes) of the caller's workspace, or of one allocated for the call (the
    tensor too: it has to live until the launch)."""
    import torch
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace: want a contiguous tensor on cuda:{index}")
    return workspace, workspace.data_ptr(), workspace.nbytes


def decode_weighted(q, k_cache, v_cache, weights, block_table, ctx_lens, scale, fresh=1, out=None,
                    workspace=None, stream=None):
    """pa_decode_weighted on tensors: decode()'s attention, and the weight each cached token
    got from the step's queries gathered in weights float32 [pages, h_kv, 16] (weight_pool):
    added, but set for the last `fresh` tokens of a sequence.  Returns fp32 [B, h_q, D].
    workspace: any tensor of pa_decode_weighted_workspace_size(...) bytes, not shared with a
    call that may run at the same time."""
    import torch
    index = _device_index(q)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return decode_weighted(q, k_cache, v_cache, weights, block_table, ctx_lens, scale,
                                   fresh, out, workspace)
    if q.dim() != 3:
        raise ValueError(f"q: want [B, h_q, D], got {tuple(q.shape)}")
    B, hq, D = q.shape
    _want(q, "q", q.dtype, q.shape, index)
    pages, hkv, D_cache = _cache_dims(k_cache, v_cache, q.dtype, index)
    if D_cache != D:
        raise ValueError(f"the cache holds head_dim {D_cache}, q has {D}")
    _want(weights, "weights", torch.float32, (pages, hkv, 16), index)
    _, mb = _want_2d(block_table, "block_table", torch.int32, B, index)
    _want(ctx_lens, "ctx_lens", torch.int32, (B,), index)
    if out is None:
        out = torch.empty((B, hq, D), dtype=torch.float32, device=q.device)
    else:
        _want(out, "out", torch.float32, (B, hq, D), index)
    L = lib()
    need = 0 if workspace is not None else \
        L.pa_decode_weighted_workspace_size(B, hq, hkv, D, 16, mb)
    workspace, ws, ws_bytes = _scratch(workspace, need, q.device, index)
    rc = L.pa_decode_weighted(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                              weights.data_ptr(), block_table.data_ptr(), ctx_lens.data_ptr(),
                              out.data_ptr(), scale, fresh, hq, hkv, D, 16, B, mb, pages,
                              dtype_code(q), ws, ws_bytes,
                              torch._C._cuda_getCurrentRawStream(index))
    if rc:
        raise PAError(rc, "pa_decode_weighted")
    return out


def prefill_weights(q, k_cache, weights, block_table, ctx_lens, scale, fresh=None, workspace=None,
                    stream=None):
    """pa_prefill_weights on tensors: the weight that the chunk's queries q [B, n_new, h_q, D]
    (or a view of its last ones: the heads of a token must be contiguous) give each cached
    token, gathered in weights [pages, h_kv, 16]; ctx_lens = tokens before these queries.
    fresh: how many of a sequence's last tokens are set, not added to (None: n_new, the
    queries' own).  Returns weights.  workspace: any tensor of
    pa_prefill_weights_workspace_size(...) bytes, as in decode_weighted."""
    import torch
    index = _device_index(q)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return prefill_weights(q, k_cache, weights, block_table, ctx_lens, scale, fresh,
                                   workspace)
    if q.dim() != 4:
        raise ValueError(f"q: want [B, n_new, h_q, D], got {tuple(q.shape)}")
    B, n_new, hq, D = q.shape
    sb, st, sh, one = q.stride()
    if n_new == 1:
        st = hq * D
    if B == 1:
        sb = max(n_new, 1) * st
    if one != 1 or (hq > 1 and sh != D):
        raise ValueError(f"q: the heads of a token must be contiguous rows (strides "
                         f"{tuple(q.stride())}); call .contiguous()")
    pages, hkv, D_cache = _cache_dims(k_cache, None, q.dtype, index)
    if D_cache != D:
        raise ValueError(f"the cache holds head_dim {D_cache}, q has {D}")
    _want(weights, "weights", torch.float32, (pages, hkv, 16), index)
    _, mb = _want_2d(block_table, "block_table", torch.int32, B, index)
    _want(ctx_lens, "ctx_lens", torch.int32, (B,), index)
    if fresh is None:
        fresh = n_new
    L = lib()
    need = 0 if workspace is not None else \
        L.pa_prefill_weights_workspace_size(B, n_new, hq, hkv, D, 16, mb)
    workspace, ws, ws_bytes = _scratch(workspace, need, q.device, index)
    rc = L.pa_prefill_weights(q.data_ptr() or _NOTHING, k_cache.data_ptr(), weights.data_ptr(),
                              block_table.data_ptr(), ctx_lens.data_ptr(), n_new, scale, fresh,
                              sb if n_new else hq * D, st, hq, hkv, D, 16, B, mb, pages,
                              dtype_code(q), ws, ws_bytes,
                              torch._C._cuda_getCurrentRawStream(index))
    if rc:
        raise PAError(rc, "pa_prefill_weights")
    return weights


def evict_kv(k_cache, v_cache, weights, block_table, ctx_lens, budget, sink=0, recent=0,
             dst_table=None, new_lens=None, workspace=None, stream=None):
    """pa_evict_kv on tensors: every sequence of more than `budget` tokens keeps, for each kv
    head, its first `sink`, its last `recent` and the heaviest others by weights
    [pages, h_kv, 16]; K, V and weights move to positions 0 .. in place, or to the pages of
    dst_table int32 [B, blocks].  Returns the new lengths, int32 [B] (new_lens if given;
    apart from the call's other tensors).  workspace: any tensor of
    pa_evict_kv_workspace_size(...) bytes, as in decode_weighted."""
    import torch
    index = _device_index(k_cache)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return evict_kv(k_cache, v_cache, weights, block_table, ctx_lens, budget, sink,
                            recent, dst_table, new_lens, workspace)
    pages, hkv, D = _cache_dims(k_cache, v_cache, k_cache.dtype, index)
    _want(weights, "weights", torch.float32, (pages, hkv, 16), index)
    B, mb = _want_2d(block_table, "block_table", torch.int32, None, index)
    _want(ctx_lens, "ctx_lens", torch.int32, (B,), index)
    if dst_table is None:
        dst_table = block_table
    _, db = _want_2d(dst_table, "dst_table", torch.int32, B, index)
    if new_lens is None:
        new_lens = torch.empty((B,), dtype=torch.int32, device=k_cache.device)
    else:
        _want(new_lens, "new_lens", torch.int32, (B,), index)
    L = lib()
    need = 0 if workspace is not None else \
        L.pa_evict_kv_workspace_size(B, hkv, D, 16, mb, budget)
    workspace, ws, ws_bytes = _scratch(workspace, need, k_cache.device, index)
    rc = L.pa_evict_kv(k_cache.data_ptr(), v_cache.data_ptr(), weights.data_ptr(),
                       block_table.data_ptr(), ctx_lens.data_ptr(), dst_table.data_ptr(),
                       new_lens.data_ptr(), budget, sink, recent, hkv, D, 16, B, mb, db, pages,
                       dtype_code(k_cache), ws, ws_bytes,
                       torch._C._cuda_getCurrentRawStream(index))
    if rc:
        raise PAError(rc, "pa_evict_kv")
    return new_lens


def compact_kv(k_cache, v_cache, block_table, ctx_lens, keep, n_keep, weights=None, new_lens=None,
               stream=None):
    """pa_compact_kv on tensors: rows ctx_lens[b] + keep[b, j], j < n_keep[b], of K, V and (if
    given) weights move up to positions ctx_lens[b] + j, in place: the accepted branch of a
    tree of drafted tokens, or (ctx_lens 0) a sequence cut to the listed tokens.  keep int32
    [B, max_keep], ascending in each row; n_keep int32 [B].  Returns the new lengths, int32
    [B] (new_lens if given; apart from the call's other tensors)."""
    import torch
    index = _device_index(k_cache)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return compact_kv(k_cache, v_cache, block_table, ctx_lens, keep, n_keep, weights,
                              new_lens)
    pages, hkv, D = _cache_dims(k_cache, v_cache, k_cache.dtype, index)
    if weights is not None:
        _want(weights, "weights", torch.float32, (pages, hkv, 16), index)
    B, mb = _want_2d(block_table, "block_table", torch.int32, None, index)
    _want(ctx_lens, "ctx_lens", torch.int32, (B,), index)
    _, most = _want_2d(keep, "keep", torch.int32, B, index)
    _want(n_keep, "n_keep", torch.int32, (B,), index)
    if new_lens is None:
        new_lens = torch.empty((B,), dtype=torch.int32, device=k_cache.device)
    else:
        _want(new_lens, "new_lens", torch.int32, (B,), index)
    rc = lib().pa_compact_kv(k_cache.data_ptr(), v_cache.data_ptr(),
                             weights.data_ptr() if weights is not None else None,
                             block_table.data_ptr(), ctx_lens.data_ptr(),
                             keep.data_ptr() or _NOTHING, n_keep.data_ptr(), most,
                             new_lens.data_ptr(), hkv, D, 16, B, mb, pages, dtype_code(k_cache),
                             torch._C._cuda_getCurrentRawStream(index))
    if rc:
        raise PAError(rc, "pa_compact_kv")
    return new_lens


def tree_mask(parents, mask=None, depth=None, stream=None):
    """pa_tree_mask on tensors: parents int32 [B, n] of the drafted tokens (-1: the last
    cached token; a parent comes before its children).  Returns (mask int32
    [B, n, ceil(n / 32)], depth int32 [B, n]): which drafted tokens each one sees, and how
    many come before it on its branch (its position is the context's length plus that)."""
    import torch
    index = _device_index(parents)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return tree_mask(parents, mask, depth)
    B, n = _want_2d(parents, "parents", torch.int32, None, index)
    words = -(-n // 32)
    if mask is None:
        mask = torch.empty((B, n, words), dtype=torch.int32, device=parents.device)
    else:
        _want(mask, "mask", torch.int32, (B, n, words), index)
    if depth is None:
        depth = torch.empty((B, n), dtype=torch.int32, device=parents.device)
    else:
        _want(depth, "depth", torch.int32, (B, n), index)
    _check(lib().pa_tree_mask(parents.data_ptr() or _NOTHING, mask.data_ptr() or _NOTHING,
                              depth.data_ptr() or _NOTHING, B, n,
                              torch._C._cuda_getCurrentRawStream(index)), "pa_tree_mask")
    return mask, depth


def prefill_tree(q, k_cache, v_cache, block_table, ctx_lens, mask, scale, out=None, workspace=None,
                 stream=None):
    """pa_prefill_tree on tensors: q [B, n, h_q, D], the queries of n drafted tokens a sequence,
    whose K/V rows are cached at positions ctx_lens[b] .. ctx_lens[b] + n - 1; mask int32
    [B, n, ceil(n / 32)] (tree_mask): bit j of row i lets token i see drafted token j.  Returns
    [B, n, h_q, D] in q's dtype.  workspace: any tensor of
    pa_prefill_tree_workspace_size(...) bytes, as in decode_weighted."""
    import torch
    index = _device_index(q)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return prefill_tree(q, k_cache, v_cache, block_table, ctx_lens, mask, scale, out,
                                workspace)
    if q.dim() != 4:
        raise ValueError(f"q: want [B, n, h_q, D], got {tuple(q.shape)}")
    B, n, hq, D = shape = q.shape
    _want(q, "q", q.dtype, shape, index)
    pages, hkv, D_cache = _cache_dims(k_cache, v_cache, q.dtype, index)
    if D_cache != D:
        raise ValueError(f"the cache holds head_dim {D_cache}, q has {D}")
    _, mb = _want_2d(block_table, "block_table", torch.int32, B, index)
    _want(ctx_lens, "ctx_lens", torch.int32, (B,), index)
    _want(mask, "mask", torch.int32, (B, n, -(-n // 32)), index)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    else:
        _want(out, "out", q.dtype, shape, index)
    L = lib()
    need = 0 if workspace is not None else \
        L.pa_prefill_tree_workspace_size(B, n, hq, hkv, D, 16, mb)
    workspace, ws, ws_bytes = _scratch(workspace, need, q.device, index)
    ptrs = (q.data_ptr(), mask.data_ptr(), out.data_ptr()) if n else (_NOTHING,) * 3
    rc = L.pa_prefill_tree(ptrs[0], k_cache.data_ptr(), v_cache.data_ptr(),
                           block_table.data_ptr(), ctx_lens.data_ptr(), ptrs[1], n, ptrs[2],
                           scale, hq, hkv, D, 16, B, mb, pages, dtype_code(q), ws, ws_bytes,
                           torch._C._cuda_getCurrentRawStream(index))
    if rc:
        raise PAError(rc, "pa_prefill_tree")
    return out
