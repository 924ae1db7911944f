"""ctypes binding of libpkv.so: the same calls, taking torch tensors.

This module only marshals arguments (pointers, sizes, the current CUDA stream)
and turns status codes into exceptions; every step of the computation runs in
the library's CUDA kernels.  There is no fallback: when the library is missing
the calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from .build import LIB_PATH

_lock = threading.Lock()
_lib = None

OK, EINVAL, EUNSUPPORTED, ECUDA = 0, 1, 2, 3
DEV_BAD_SLOT, DEV_BAD_PAGE, DEV_BAD_SEQLEN, DEV_BAD_CUSEQ, DEV_TIMEOUT = 1, 2, 4, 8, 16
DEV_BAD_WORKSPACE, DEV_BAD_SHARED, DEV_BAD_POS, DEV_BAD_ROW = 32, 64, 128, 256

_P = ctypes.c_void_p
_I32, _I64, _F32, _SZ = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t

SIGNATURES = {
    "pkv_status_string": ([_I32], ctypes.c_char_p),
    "pkv_version": ([], _I32),
    "pkv_kv_store": ([_P, _P, _P, _I64, _P, _P, _I64, _I32, _I32, _I32, _P, _P], _I32),
    "pkv_decode_workspace_size": ([_I32, _I32, _I32, _I32], _SZ),
    "pkv_paged_decode_attn": ([_P, _P, _P, _P, _I64, _P, _I32, _I32, _I32, _I32, _I32, _I64,
                               _F32, _P, _SZ, _P, _P, _P], _I32),
    "pkv_paged_decode_attn_store": ([_P, _P, _P, _P, _P, _P, _P, _I64, _P, _I32, _I32, _I32,
                                     _I32, _I32, _I64, _F32, _P, _SZ, _P, _P, _P], _I32),
    "pkv_paged_prefill_attn": ([_P, _P, _P, _P, _P, _I64, _P, _I32, _I64, _I32, _I32, _I32,
                                _I32, _I32, _I64, _F32, _P, _SZ, _P, _P, _P], _I32),
    "pkv_prefill_workspace_size": ([], _SZ),
    "pkv_paged_prefill_attn_shared": ([_P, _P, _P, _P, _P, _I64, _P, _I32, _I64, _I32, _I32, _I32,
                                       _I32, _I32, _I64, _F32, _P, _P, _I32, _I32, _P, _SZ, _P, _P,
                                       _P], _I32),
    "pkv_paged_decode_attn_noalloc": ([_P, _P, _P, _P, _I64, _P, _I32, _I32, _I32, _I32, _I32,
                                       _I64, _F32, _P, _P, _P], _I32),
    "pkv_qk_norm_rope_store": ([_P, _I64, _P, _I64, _P, _I64, _P, _P, _F32, _P, _P, _I64, _I32, _I32,
                                _P, _I64, _I32, _I32, _I32, _P, _P, _I64, _I32, _P, _P, _P], _I32),
    "pkv_decode_weights_workspace_size": ([_I32, _I32, _I32, _I32, _I32], _SZ),
    "pkv_paged_decode_attn_weights": ([_P, _P, _P, _P, _I64, _P, _I32, _I32, _I32, _I32, _I32, _I64,
                                       _F32, _P, _P, _I64, _I64, _I32, _P, _SZ, _P, _P, _P], _I32),
    "pkv_kv_evict": ([_P, _P, _P, _I64, _P, _I64, _P, _P, _I32, _I32, _I32, _I32, _I64, _I32, _I32,
                      _P, _P, _P, _I64, _I64, _P, _I64, _P, _P, _P], _I32),
}


class PkvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = load_library().pkv_status_string(status).decode()
        super().__init__(f"{fn} returned {status} ({msg})")
        self.status = status


def load_library(path: str | None = None):
    """Load libpkv.so (built by ``paged_kv_cache_out_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"the CUDA library {p} is not built: run "
                                   "paged_kv_cache_out_gb300.build.build() first")
            lib = ctypes.CDLL(p)
            for name, (args, res) in SIGNATURES.items():
                f = getattr(lib, name)
                f.argtypes, f.restype = args, res
            _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, status):
    if status != OK:
        raise PkvError(fn, status)


def _bf16(t, name):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor")


def _i32(t, name):
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor")


def kv_store(k_new, v_new, out_loc, k_cache, v_cache, dev_status=None, stream=None):
    """Copy new K/V rows [T, Hkv, d] into pool slots out_loc (pool [P, ps, Hkv, d])."""
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _bf16(t, n)
    _i32(out_loc, "out_loc")
    P, ps, Hkv, d = k_cache.shape
    T = out_loc.shape[0]
    if k_new.shape != (T, Hkv, d) or v_new.shape != (T, Hkv, d) or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch")
    st = load_library().pkv_kv_store(_ptr(k_new), _ptr(v_new), _ptr(out_loc), T, _ptr(k_cache),
                                     _ptr(v_cache), P, ps, Hkv, d, _ptr(dev_status), _stream(stream))
    _check("pkv_kv_store", st)


def decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim) -> int:
    return int(load_library().pkv_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim))


def decode_workspace(batch, num_q_heads, num_kv_heads, head_dim, device=None):
    n = decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def paged_decode_attn(q, k_cache, v_cache, page_table, seq_lens, softmax_scale, workspace=None,
                      dev_status=None, out=None, stream=None):
    """Decode attention: q [B, Hq, d] over the pool through page_table [B, stride]."""
    _bf16(q, "q"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache")
    _i32(seq_lens, "seq_lens")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be a 2-D int32 tensor with unit column stride")
    B, Hq, d = q.shape
    P, ps, Hkv, d2 = k_cache.shape
    if d2 != d or v_cache.shape != k_cache.shape or seq_lens.shape[0] != B:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = decode_workspace(B, Hq, Hkv, d, q.device)
    st = load_library().pkv_paged_decode_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), page_table.stride(0),
        _ptr(seq_lens), B, Hq, Hkv, d, ps, P, float(softmax_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _ptr(out), _stream(stream))
    _check("pkv_paged_decode_attn", st)
    return out


def paged_decode_attn_store(q, k_new, v_new, out_loc, k_cache, v_cache, page_table, seq_lens,
                            softmax_scale, workspace=None, dev_status=None, out=None, stream=None):
    """kv_store of the decode rows k_new/v_new [B, Hkv, d] at out_loc [B] fused
    into decode attention (same results as kv_store followed by paged_decode_attn)."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"),
                 (v_cache, "v_cache")):
        _bf16(t, n)
    _i32(seq_lens, "seq_lens"), _i32(out_loc, "out_loc")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be a 2-D int32 tensor with unit column stride")
    B, Hq, d = q.shape
    P, ps, Hkv, d2 = k_cache.shape
    if (d2 != d or v_cache.shape != k_cache.shape or seq_lens.shape[0] != B
            or out_loc.shape[0] != B or k_new.shape != (B, Hkv, d) or v_new.shape != (B, Hkv, d)):
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = decode_workspace(B, Hq, Hkv, d, q.device)
    st = load_library().pkv_paged_decode_attn_store(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out_loc), _ptr(k_cache), _ptr(v_cache),
        _ptr(page_table), page_table.stride(0), _ptr(seq_lens), B, Hq, Hkv, d, ps, P,
        float(softmax_scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_status), _ptr(out), _stream(stream))
    _check("pkv_paged_decode_attn_store", st)
    return out


def prefill_workspace(device=None):
    """A zero-filled prefill workspace (the queue counters must start at zero;
    every call leaves them at zero)."""
    n = int(load_library().pkv_prefill_workspace_size())
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def paged_prefill_attn(q, cu_seqlens_q, k_cache, v_cache, page_table, seq_lens, softmax_scale,
                       max_q_len, workspace=None, dev_status=None, out=None, stream=None):
    """Ragged causal prefill: q [Tq, Hq, d] with offsets cu_seqlens_q [B+1].

    workspace: from prefill_workspace(); calls that may overlap on the GPU
    need separate workspaces.  Without one, a fresh zeroed one is made."""
    _bf16(q, "q"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache")
    _i32(seq_lens, "seq_lens"), _i32(cu_seqlens_q, "cu_seqlens_q")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be a 2-D int32 tensor with unit column stride")
    Tq, Hq, d = q.shape
    P, ps, Hkv, d2 = k_cache.shape
    B = seq_lens.shape[0]
    if d2 != d or v_cache.shape != k_cache.shape or cu_seqlens_q.shape[0] != B + 1:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = prefill_workspace(q.device)
    st = load_library().pkv_paged_prefill_attn(
        _ptr(q), _ptr(cu_seqlens_q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
        page_table.stride(0), _ptr(seq_lens), B, Tq, int(max_q_len), Hq, Hkv, d, ps, P,
        float(softmax_scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_status), _ptr(out), _stream(stream))
    _check("pkv_paged_prefill_attn", st)
    return out


def paged_prefill_attn_shared(q, cu_seqlens_q, k_cache, v_cache, page_table, seq_lens,
                              softmax_scale, max_q_len, prefix_group_start, prefix_len,
                              max_group_tokens, workspace=None, dev_status=None, out=None,
                              stream=None):
    """Ragged causal prefill for requests that share cached prefixes.

    prefix_group_start [n_groups + 1] int32: group g is requests
    prefix_group_start[g] .. prefix_group_start[g+1]-1 (the groups partition
    the batch in order); prefix_len [n_groups] int32: the keys they share
    (whole pages, listed first in every member's page-table row; 0 for a
    request that shares nothing).  max_group_tokens bounds the new tokens of
    any group.  The result equals paged_prefill_attn on the same arguments.
    workspace: from prefill_workspace()."""
    _bf16(q, "q"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache")
    _i32(seq_lens, "seq_lens"), _i32(cu_seqlens_q, "cu_seqlens_q")
    _i32(prefix_group_start, "prefix_group_start"), _i32(prefix_len, "prefix_len")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be a 2-D int32 tensor with unit column stride")
    Tq, Hq, d = q.shape
    P, ps, Hkv, d2 = k_cache.shape
    B = seq_lens.shape[0]
    n_groups = prefix_len.shape[0]
    if (d2 != d or v_cache.shape != k_cache.shape or cu_seqlens_q.shape[0] != B + 1
            or prefix_group_start.shape[0] != n_groups + 1):
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = prefill_workspace(q.device)
    st = load_library().pkv_paged_prefill_attn_shared(
        _ptr(q), _ptr(cu_seqlens_q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
        page_table.stride(0), _ptr(seq_lens), B, Tq, int(max_q_len), Hq, Hkv, d, ps, P,
        float(softmax_scale), _ptr(prefix_group_start), _ptr(prefix_len), n_groups,
        int(max_group_tokens), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_status), _ptr(out), _stream(stream))
    _check("pkv_paged_prefill_attn_shared", st)
    return out


# The calls below check that every tensor is on the current device (the library
# launches there), pass addresses as plain integers, and allocate what the caller
# did not give on the stream that uses it.

def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _tensor(t, name, dtype, device, shape=None):
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on the current CUDA device")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _status(t, device):
    if t is not None and (t.dtype is not torch.int32 or t.get_device() != device or t.numel() < 1):
        raise ValueError("dev_status must be an int32 tensor on the current CUDA device")


def _heads(t, name, device, tokens, head_dim):
    """A [tokens, heads, head_dim] bf16 tensor whose heads are dense; returns the
    elements from token to token."""
    if t.dtype is not torch.bfloat16 or t.get_device() != device or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D bfloat16 tensor on the current CUDA device")
    T, H, d = t.shape
    step, head, one = t.stride()
    if T != tokens or d != head_dim:
        raise ValueError(f"{name} must have shape ({tokens}, heads, {head_dim}), not {tuple(t.shape)}")
    if one != 1 or (head != d and H > 1):
        raise ValueError(f"the heads of each token of {name} must be dense")
    return step if T > 1 else H * d


def _pages(t, name, device, batch):
    """Row width of a page table; every row lies inside the tensor's storage."""
    if (t.dtype is not torch.int32 or t.get_device() != device or t.dim() != 2 or t.shape[0] < batch
            or t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D int32 tensor on the current CUDA device with a row per "
                         "sequence and unit column stride")
    width = t.stride(0)
    if width != t.shape[1]:  # columns of a wider table
        if t.shape[0] == 1:
            return t.shape[1]
        room = t.untyped_storage().nbytes() // 4 - t.storage_offset()
        if width < t.shape[1] or (t.shape[0] - 1) * width + width > room:
            raise ValueError(f"the last row of {name} must be as wide as the others in memory")
    return width


def _on(stream):
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def qk_norm_rope_store(q, k, v, positions, cos_sin, out_loc, k_cache, v_cache, q_weight=None,
                       k_weight=None, eps=1e-6, interleaved=False, dev_status=None, out=None,
                       stream=None):
    """RMS norm (with q_weight / k_weight [d]) and rotation of each head of q [T, Hq, d] and
    k [T, Hkv, d], and kv_store of k and v [T, Hkv, d] at out_loc [T]: returns the queries.

    cos_sin [positions, rot_dim] fp32: cosines of the rot_dim / 2 pairs, then their sines;
    positions [T] int32 names each token's row.  None for both: no rotation.  q, k and v may be
    column ranges of one buffer (a token's heads dense).  out may be q when q is contiguous."""
    dev = torch.cuda.current_device()
    P, ps, Hkv, d = k_cache.shape
    T, Hq = q.shape[0], q.shape[1]
    qs, ks, vs = _heads(q, "q", dev, T, d), _heads(k, "k", dev, T, d), _heads(v, "v", dev, T, d)
    if k.shape[1] != Hkv or v.shape[1] != Hkv:
        raise ValueError("k, v and the caches must have the same number of heads")
    _tensor(k_cache, "k_cache", torch.bfloat16, dev)
    _tensor(v_cache, "v_cache", torch.bfloat16, dev, k_cache.shape)
    _tensor(out_loc, "out_loc", torch.int32, dev, (T,))
    if q_weight is not None:
        _tensor(q_weight, "q_weight", torch.bfloat16, dev, (d,))
    if k_weight is not None:
        _tensor(k_weight, "k_weight", torch.bfloat16, dev, (d,))
    if (positions is None) != (cos_sin is None):
        raise ValueError("positions and cos_sin come together")
    rows, rot = 0, 0
    if cos_sin is not None:
        _tensor(positions, "positions", torch.int32, dev, (T,))
        _tensor(cos_sin, "cos_sin", torch.float32, dev)
        rows, rot = cos_sin.shape
    _status(dev_status, dev)
    if out is None:
        with _on(stream):
            out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=q.device)
    else:
        _tensor(out, "out", torch.bfloat16, dev, q.shape)
    st = load_library().pkv_qk_norm_rope_store(
        q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, _addr(q_weight), _addr(k_weight), eps,
        _addr(positions), _addr(cos_sin), rows, rot, interleaved, out_loc.data_ptr(), T, Hq, Hkv, d,
        k_cache.data_ptr(), v_cache.data_ptr(), P, ps, out.data_ptr(), _addr(dev_status),
        _raw_stream(stream, dev))
    if st:
        raise PkvError("pkv_qk_norm_rope_store", st)
    return out


def decode_weights_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len) -> int:
    return int(load_library().pkv_decode_weights_workspace_size(batch, num_q_heads, num_kv_heads,
                                                                head_dim, max_seq_len))


def decode_weights_workspace(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, device=None):
    n = decode_weights_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def paged_decode_attn_weights(q, k_cache, v_cache, page_table, seq_lens, softmax_scale, acc,
                              max_seq_len, acc_rows=None, workspace=None, dev_status=None, out=None,
                              stream=None):
    """paged_decode_attn that adds every key's softmax weight, summed over the query heads of its
    KV head, to acc[acc_rows[b], kv head, position] (acc [rows, Hkv, positions] fp32).  The newest
    key's sum starts with this call.  max_seq_len bounds seq_lens.

    workspace: from decode_weights_workspace(); calls that may overlap on the GPU need separate
    ones."""
    dev = torch.cuda.current_device()
    B, Hq, d = q.shape
    P, ps, Hkv, d2 = k_cache.shape
    if d2 != d:
        raise ValueError("q and the caches must have the same head size")
    _tensor(q, "q", torch.bfloat16, dev)
    _tensor(k_cache, "k_cache", torch.bfloat16, dev)
    _tensor(v_cache, "v_cache", torch.bfloat16, dev, k_cache.shape)
    _tensor(seq_lens, "seq_lens", torch.int32, dev, (B,))
    _tensor(acc, "acc", torch.float32, dev)
    rows, heads, positions = acc.shape
    if heads != Hkv:
        raise ValueError("acc must have a row for each KV head")
    if acc_rows is not None:
        _tensor(acc_rows, "acc_rows", torch.int32, dev, (B,))
    width = _pages(page_table, "page_table", dev, B)
    _status(dev_status, dev)
    if out is None or workspace is None:
        with _on(stream):
            if out is None:
                out = torch.empty_like(q)
            if workspace is None:
                workspace = decode_weights_workspace(B, Hq, Hkv, d, max_seq_len, q.device)
    _tensor(out, "out", torch.bfloat16, dev, q.shape)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the current CUDA device")
    st = load_library().pkv_paged_decode_attn_weights(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), width,
        seq_lens.data_ptr(), B, Hq, Hkv, d, ps, P, softmax_scale, acc.data_ptr(), _addr(acc_rows), rows,
        positions, max_seq_len, workspace.data_ptr(), workspace.nbytes, _addr(dev_status),
        out.data_ptr(), _raw_stream(stream, dev))
    if st:
        raise PkvError("pkv_paged_decode_attn_weights", st)
    return out


def kv_evict(k_cache, v_cache, page_table, seq_lens, keep_lens, acc, num_first, num_recent,
             acc_rows=None, page_table_out=None, acc_out=None, kept=None, new_seq_lens=None,
             max_keep=None, dev_status=None, stream=None):
    """Keep keep_lens[b] keys of every sequence and KV head: the first num_first, the last
    num_recent and the heaviest of the rest by acc; their K/V rows and sums move to positions
    0 .. n - 1.  Returns (kept [B, Hkv, max_keep] int32: the kept positions, rising, at
    0 .. n - 1; new_seq_lens [B]).

    page_table_out: where the rows go (default page_table: in place); acc_out: where the sums go
    (default acc).  max_keep sizes kept when it is not given (default: all positions of acc)."""
    dev = torch.cuda.current_device()
    P, ps, Hkv, d = k_cache.shape
    B = seq_lens.shape[0]
    _tensor(k_cache, "k_cache", torch.bfloat16, dev)
    _tensor(v_cache, "v_cache", torch.bfloat16, dev, k_cache.shape)
    _tensor(seq_lens, "seq_lens", torch.int32, dev, (B,))
    _tensor(keep_lens, "keep_lens", torch.int32, dev, (B,))
    _tensor(acc, "acc", torch.float32, dev)
    rows, heads, positions = acc.shape
    if heads != Hkv:
        raise ValueError("acc must have a row for each KV head")
    if acc_rows is not None:
        _tensor(acc_rows, "acc_rows", torch.int32, dev, (B,))
    if acc_out is None:
        acc_out = acc
    else:
        _tensor(acc_out, "acc_out", torch.float32, dev, acc.shape)
    width = _pages(page_table, "page_table", dev, B)
    if page_table_out is None:
        page_table_out, width_out = page_table, width
    else:
        width_out = _pages(page_table_out, "page_table_out", dev, B)
    _status(dev_status, dev)
    if kept is None or new_seq_lens is None:
        with _on(stream):
            if kept is None:
                kept = torch.empty((B, Hkv, positions if max_keep is None else max_keep),
                                   dtype=torch.int32, device=acc.device)
            if new_seq_lens is None:
                new_seq_lens = torch.empty_like(seq_lens)
    _tensor(kept, "kept", torch.int32, dev)
    if kept.dim() != 3 or kept.shape[0] != B or kept.shape[1] != Hkv:
        raise ValueError("kept must have shape (batch, KV heads, max_keep)")
    _tensor(new_seq_lens, "new_seq_lens", torch.int32, dev, (B,))
    st = load_library().pkv_kv_evict(
        k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), width, page_table_out.data_ptr(),
        width_out, seq_lens.data_ptr(), keep_lens.data_ptr(), B, Hkv, d, ps, P, num_first, num_recent,
        acc.data_ptr(), acc_out.data_ptr(), _addr(acc_rows), rows, positions, kept.data_ptr(),
        kept.shape[2], new_seq_lens.data_ptr(), _addr(dev_status), _raw_stream(stream, dev))
    if st:
        raise PkvError("pkv_kv_evict", st)
    return kept, new_seq_lens
