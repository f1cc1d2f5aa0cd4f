"""Tensor-level convenience over the C ABI (marshalling and output allocation).

Callers that hold torch tensors use these; every step of the computation runs
in ``libpkv.so``.  Outputs (and the decode workspace, unless one is passed)
are allocated with torch on the inputs' device.

The cache in 8 bits (``append_q8``, ``copy_pages_q8``, ``paged_q8``) holds its
codes in int8 or float8_e4m3fn pages and one float32 scale for each block of
tokens and kv head; ``paged_weights`` and ``evict`` keep a cache within a budget
of tokens.  These five check their tensors, raise ValueError or TypeError for
ones that do not fit together, and run on the tensors' device whichever device
is current.

With ``stream`` None a call runs on the current stream (these five: of the
tensors' device).  Another stream the caller orders against the producers of the
tensors that are passed and the consumers of the results.  What a call allocates
it takes from its own stream's memory, which no other stream's earlier work can
still be using; results may be dropped on the stream that is current at the call,
and elsewhere by torch's rules (``record_stream``).
"""

from __future__ import annotations

import contextlib
import functools

import torch

from . import binding as B

_DT = {torch.bfloat16: B.PKV_BF16, torch.float32: B.PKV_F32}


_HERE = contextlib.nullcontext()


def _torch_stream(stream, device):
    return stream if isinstance(stream, torch.cuda.Stream) else \
        torch.cuda.ExternalStream(B._stream(stream), device=device)


def _allocating(stream, device):
    """A context whose torch allocations come from `stream`'s memory (None: the current stream's)."""
    return _HERE if stream is None else torch.cuda.stream(_torch_stream(stream, device))


def _used_on(stream, passed=(), made=()):
    """Keep tensors from being reused before work that their own stream does not know of has run: the call's for
    those that were passed, the caller's for those that the call made."""
    if stream is None:
        return
    for t in passed:
        if t is not None:
            t.record_stream(_torch_stream(stream, t.device))
    for t in made:
        if t is not None:
            t.record_stream(torch.cuda.current_stream(t.device))


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def prefill(Q, K, V, causal: bool, scale: float, out=None, stream=None) -> torch.Tensor:
    """Contiguous attention, Q/K/V [B, H, N, d] on one CUDA device."""
    Bn, H, N, d = Q.shape
    for t in (Q, K, V):
        assert t.is_contiguous() and t.shape == Q.shape and t.dtype == Q.dtype
    O = out
    if O is None:
        with _allocating(stream, Q.device):
            O = torch.empty_like(Q)
        _used_on(stream, made=(O,))
    B.attn_prefill(Q, K, V, O, Bn, H, N, d, causal, scale, _dtype(Q), stream)
    return O


def workspace_for(num_seqs: int, H: int, d: int, max_seq_len: int, page_size: int,
                  device) -> torch.Tensor | None:
    n = B.paged_attn_workspace_size(num_seqs, H, d, max_seq_len, page_size)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device)


def paged(q, k_pages, v_pages, block_table, seq_lens, page_size: int, causal: bool,
          scale: float, max_seq_len: int, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Paged attention: q [S, H, q_len, d]; pages [P, page_size, H_kv, d]."""
    S, H, q_len, d = q.shape
    P, ps, H_kv, d2 = k_pages.shape
    assert ps == page_size and d2 == d and v_pages.shape == k_pages.shape
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32
    assert block_table.is_contiguous() and q.is_contiguous() and k_pages.is_contiguous()
    o, ws = out, workspace
    if o is None:
        with _allocating(stream, q.device):
            o = torch.empty_like(q)
        _used_on(stream, made=(o,))
    if ws is None and q_len == 1:
        with _allocating(stream, q.device):
            ws = workspace_for(S, H, d, max_seq_len, page_size, q.device)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    B.paged_attn(q, k_pages, v_pages, block_table, seq_lens, page_size, S, q_len, H, H_kv, d,
                 P, block_table.shape[1], max_seq_len, causal, scale, _dtype(q), o, ws,
                 ws_bytes, stream)
    return o


# ------------------------------------------------ 8-bit cache, weights, eviction --

_Q8 = {torch.int8: B.PKV_I8, torch.float8_e4m3fn: B.PKV_E4M3}


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _on_device(*tensors):
    """A context in which the tensors' device is current (nothing to do if it is)."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev or dev < 0:
            raise ValueError("every tensor must be on one CUDA device")
        if not t.is_contiguous():
            raise ValueError("every tensor must be contiguous")
    return _HERE if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream_of(stream, t):
    """The stream's address: None means the current stream of the tensor's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else B._stream(stream)


def _pools(k_pages, v_pages, k_scales, v_scales):
    """(cache dtype, tokens a block) of a pool of pages and its scales."""
    shape, dtype = k_pages.shape, k_pages.dtype
    _need(len(shape) == 4 and v_pages.shape == shape and v_pages.dtype == dtype,
          "k_pages and v_pages must be [pages, page_size, H_kv, d] of one type")
    if dtype in _DT:
        _need(k_scales is None and v_scales is None, "only an 8-bit cache has scales")
        return _DT[dtype], 0
    if dtype not in _Q8:
        raise TypeError(f"unsupported cache dtype {dtype}")
    _need(k_scales is not None and v_scales is not None, "an 8-bit cache needs its scales")
    _need(k_scales.dtype == torch.float32 and v_scales.dtype == torch.float32, "scales must be float32")
    blocks = k_scales.shape
    _need(len(blocks) == 3 and v_scales.shape == blocks and blocks[0] == shape[0] and blocks[2] == shape[2]
          and blocks[1] > 0 and shape[1] % blocks[1] == 0, "scales must be [pages, page_size / block_tokens, H_kv]")
    return _Q8[dtype], shape[1] // blocks[1]


def _int32(*tensors):
    for t in tensors:
        _need(t.dtype == torch.int32, "tables, lengths and indices must be int32")


def _workspace(workspace, n, device):
    """(workspace, its bytes); one that is made here is used by the call's stream alone."""
    if workspace is None:
        workspace = torch.empty(n, dtype=torch.uint8, device=device) if n else None
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor of the same device")
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


# Sizes alone decide a workspace's bytes.
_q8_bytes = functools.lru_cache(4096)(B.paged_attn_q8_workspace_size)
_weights_bytes = functools.lru_cache(4096)(B.paged_attn_weights_workspace_size)
_evict_bytes = functools.lru_cache(4096)(B.paged_kv_evict_workspace_size)


def append_q8(k_new, v_new, cu_new, start_pos, block_table, k_pages, v_pages, k_scales, v_scales,
              stream=None) -> None:
    """Quantise new K/V rows [num_new, H_kv, d] (bf16 or f32) into an 8-bit cache, in place."""
    cache, block = _pools(k_pages, v_pages, k_scales, v_scales)
    if cache not in (B.PKV_I8, B.PKV_E4M3):
        raise TypeError(f"unsupported cache dtype {k_pages.dtype}")
    P, ps, H_kv, d = k_pages.shape
    _need(k_new.dim() == 3 and k_new.shape[1:] == (H_kv, d) and v_new.shape == k_new.shape
          and v_new.dtype == k_new.dtype, "k_new and v_new must be [num_new, H_kv, d] of one type")
    _int32(cu_new, start_pos, block_table)
    S = start_pos.numel()
    _need(cu_new.numel() == S + 1 and block_table.dim() == 2 and block_table.shape[0] == S,
          "cu_new must hold num_seqs + 1 entries and block_table a row for each sequence")
    with _on_device(k_pages, v_pages, k_scales, v_scales, k_new, v_new, cu_new, start_pos, block_table):
        B.paged_kv_append_q8(k_new, v_new, cu_new, start_pos, block_table, block_table.shape[1], S,
                             k_new.shape[0], k_pages, v_pages, k_scales, v_scales, P, ps, block, H_kv, d,
                             _dtype(k_new), cache, _stream_of(stream, k_pages))


def copy_pages_q8(k_pages, v_pages, k_scales, v_scales, src, dst, stream=None) -> None:
    """Copy pages src[i] -> dst[i] of an 8-bit cache, codes and scales."""
    cache, block = _pools(k_pages, v_pages, k_scales, v_scales)
    if cache not in (B.PKV_I8, B.PKV_E4M3):
        raise TypeError(f"unsupported cache dtype {k_pages.dtype}")
    P, ps, H_kv, d = k_pages.shape
    _int32(src, dst)
    _need(src.shape == dst.shape, "as many sources as destinations")
    with _on_device(k_pages, v_pages, k_scales, v_scales, src, dst):
        B.paged_kv_copy_pages_q8(k_pages, v_pages, k_scales, v_scales, src, dst, src.numel(), P, ps, block, H_kv,
                                 d, cache, _stream_of(stream, k_pages))


def _attn_shapes(q, k_pages, block_table, seq_lens, page_size, out):
    _need(q.dim() == 4 and q.dtype == torch.bfloat16, "q must be bf16 [num_seqs, H, q_len, d]")
    S, H, q_len, d = q.shape
    _, ps, H_kv, d2 = k_pages.shape
    _need(ps == page_size and d2 == d, "pages must hold page_size tokens of q's head dim")
    _int32(block_table, seq_lens)
    _need(block_table.dim() == 2 and block_table.shape[0] == S and seq_lens.numel() == S,
          "block_table and seq_lens must hold a row and a length for each sequence")
    _need(out is None or (out.shape == q.shape and out.dtype == q.dtype), "out must look like q")
    return S, H, q_len, d, H_kv


def paged_q8(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, page_size: int, causal: bool,
             scale: float, max_seq_len: int, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention over an 8-bit paged cache: q [S, H, q_len, d] bf16; pages [P, page_size, H_kv, d]."""
    cache, block = _pools(k_pages, v_pages, k_scales, v_scales)
    if cache not in (B.PKV_I8, B.PKV_E4M3):
        raise TypeError(f"unsupported cache dtype {k_pages.dtype}")
    S, H, q_len, d, H_kv = _attn_shapes(q, k_pages, block_table, seq_lens, page_size, out)
    mine = () if out is None else (out,)
    with _on_device(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, *mine):
        with _allocating(stream, q.device):
            o = torch.empty_like(q) if out is None else out
            ws, n = _workspace(workspace, _q8_bytes(S, q_len, H, H_kv, max_seq_len, page_size), q.device)
        B.paged_attn_q8(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, page_size, block, S, q_len,
                        H, H_kv, d, k_pages.shape[0], block_table.shape[1], max_seq_len, causal, scale, cache, o,
                        ws, n, _stream_of(stream, q))
        _used_on(stream, (out, workspace), () if out is not None else (o,))
    return o


def paged_weights(q, k_pages, v_pages, block_table, seq_lens, page_size: int, causal: bool, scale: float,
                  max_seq_len: int, weights, k_scales=None, v_scales=None, out=None, workspace=None,
                  stream=None) -> torch.Tensor:
    """Attention over a bf16 or 8-bit paged cache that adds every key's softmax weight, summed over the
    query rows and the query heads of its kv head, to ``weights`` [S, H_kv, >= max_seq_len] (float32)."""
    cache, block = _pools(k_pages, v_pages, k_scales, v_scales)
    S, H, q_len, d, H_kv = _attn_shapes(q, k_pages, block_table, seq_lens, page_size, out)
    _need(weights.dtype == torch.float32 and weights.dim() == 3 and weights.shape[:2] == (S, H_kv)
          and weights.shape[2] >= max_seq_len, "weights must be float32 [num_seqs, H_kv, >= max_seq_len]")
    more = (() if block == 0 else (k_scales, v_scales)) + (() if out is None else (out,))
    with _on_device(q, k_pages, v_pages, block_table, seq_lens, weights, *more):
        with _allocating(stream, q.device):
            o = torch.empty_like(q) if out is None else out
            ws, n = _workspace(workspace, _weights_bytes(S, q_len, H, H_kv, max_seq_len, page_size), q.device)
        B.paged_attn_weights(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, page_size, block, S,
                             q_len, H, H_kv, d, k_pages.shape[0], block_table.shape[1], max_seq_len, causal, scale,
                             cache, o, weights, weights.shape[2], ws, n, _stream_of(stream, q))
        _used_on(stream, (out, workspace), () if out is not None else (o,))
    return o


def evict(k_pages, v_pages, weights, block_table, seq_lens, budget: int, recent: int, max_seq_len: int,
          dst_table=None, weights_out=None, k_scales=None, v_scales=None, workspace=None, stream=None):
    """Shorten every sequence to ``budget`` tokens: the last ``recent`` ones and those of the largest weight.

    Compacts K, V and (into ``weights_out``, default ``weights`` itself) the weights; ``dst_table`` (default
    ``block_table``: in place) says where kept tokens go.  Returns (kept [S, H_kv, budget] int32: their old
    indices, -1 padded; the new lengths [S] int32)."""
    cache, block = _pools(k_pages, v_pages, k_scales, v_scales)
    P, ps, H_kv, d = k_pages.shape
    dst_table = block_table if dst_table is None else dst_table
    weights_out = weights if weights_out is None else weights_out
    _int32(block_table, dst_table, seq_lens)
    S = seq_lens.numel()
    _need(block_table.dim() == 2 and block_table.shape[0] == S and dst_table.shape == block_table.shape,
          "block_table and dst_table must hold a row for each sequence")
    _need(weights.dtype == torch.float32 and weights.dim() == 3 and weights.shape[:2] == (S, H_kv)
          and weights.shape[2] >= max_seq_len and weights_out.shape == weights.shape
          and weights_out.dtype == torch.float32, "weights must be float32 [num_seqs, H_kv, >= max_seq_len]")
    more = () if block == 0 else (k_scales, v_scales)
    with _on_device(k_pages, v_pages, weights, weights_out, block_table, dst_table, seq_lens, *more):
        with _allocating(stream, k_pages.device):
            kept = torch.empty((S, H_kv, max(budget, 0)), dtype=torch.int32, device=k_pages.device)
            new_lens = torch.empty_like(seq_lens)
            ws, n = _workspace(workspace, _evict_bytes(S, H_kv, budget, block, cache), k_pages.device)
        B.paged_kv_evict(k_pages, v_pages, k_scales, v_scales, weights, weights_out, weights.shape[2], block_table,
                         dst_table, seq_lens, new_lens, kept, budget, recent, S, H_kv, d, P, ps, block,
                         block_table.shape[1], max_seq_len, cache, ws, n, _stream_of(stream, k_pages))
        _used_on(stream, (workspace,), (kept, new_lens))
    return kept, new_lens
