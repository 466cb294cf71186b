"""Serving from the restored cache: K and V in pages, the step's tokens written into them and attending.

    m = page_map(ctx_lens, new_lens, free_pages, block_table, page_size, tokens)   # once a step
    for layer in ...:
        paged_append(K, V, K_pages[layer], V_pages[layer], m.slots)
        O = paged_attention(Q, K_pages[layer], V_pages[layer], block_table, m.q_start, m.kv_lens, max_q=...)

A pool is an fp16 or bf16 CUDA tensor [pages, kv_heads, page_size, head_dim] with any strides that are
multiples of 8 elements and a contiguous last axis: pages that are stored token-major
([pages, page_size, kv_heads, head_dim]) are passed as .transpose(1, 2).  Lengths, tables and slots stay on the
device: no call waits for the GPU, and a step can be captured as a CUDA graph.  All work is enqueued on the
current torch CUDA stream.
"""
import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from .codec import _call, _stream_handle, ctypes_ref, ctypes_void, workspace

__all__ = ["PageMap", "page_map", "paged_append", "paged_attention", "paged_attention_workspace", "paged_status"]

_DTYPES = {torch.float16: _lib.NQ_F16, torch.bfloat16: _lib.NQ_BF16}


@dataclass(frozen=True)
class PageMap:
    """What page_map leaves of a step (see there)."""

    q_start: torch.Tensor
    kv_lens: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    counts: torch.Tensor

    @classmethod
    def empty(cls, requests, tokens, device="cuda"):
        """Uninitialised buffers for steps of `requests` requests and room for `tokens` tokens."""
        def new(n, dtype=torch.int32):
            return torch.empty(n, dtype=dtype, device=device)

        return cls(new(requests + 1), new(requests), new(tokens, torch.int64), new(tokens), new(4))


def _check_vec(x, name, dtype, device, n=None):
    if not (x.is_cuda and x.dtype == dtype and x.dim() == 1 and x.is_contiguous()):
        raise ValueError("%s must be a contiguous 1-D %s CUDA tensor" % (name, str(dtype)[6:]))
    if n is not None and x.shape[0] != n:
        raise ValueError("%s has %d entries; the call needs %d" % (name, x.shape[0], n))
    if device is not None and x.device != device:
        raise ValueError("%s is on %s; the call runs on %s" % (name, x.device, device))


def _check_table(table, requests, device):
    if not (table.is_cuda and table.dtype == torch.int32 and table.dim() == 2 and
            (table.stride(1) == 1 or table.shape[1] <= 1 or table.shape[0] == 0)):
        raise ValueError("block_table must be a 2-D int32 CUDA tensor with contiguous rows")
    if table.shape[0] != requests:
        raise ValueError("block_table has %d rows; there are %d requests" % (table.shape[0], requests))
    if table.device != device:
        raise ValueError("block_table is on %s; the call runs on %s" % (table.device, device))


def _check_rows(x, name, heads, dim, dtype, device, tokens=None):
    """A [tokens, heads, dim] tensor whose rows the kernels read or write 16 bytes at a time."""
    if not (x.is_cuda and x.dtype == dtype and x.dim() == 3 and (x.stride(2) == 1 or x.numel() == 0)):
        raise ValueError("%s must be a 3-D %s CUDA tensor [tokens, heads, head_dim] with a contiguous last axis"
                         % (name, str(dtype)[6:]))
    t = x.shape[0] if tokens is None else tokens
    if tuple(x.shape) != (t, heads, dim):
        raise ValueError("%s has shape %s; the call needs %s" % (name, tuple(x.shape), (t, heads, dim)))
    if x.device != device:
        raise ValueError("%s is on %s; the call runs on %s" % (name, x.device, device))
    _check_strides(x, name, 2)


def _check_strides(x, name, axes):
    if x.data_ptr() % 16:
        raise ValueError("%s must start on a 16-byte boundary" % name)
    for d in range(axes):
        if x.shape[d] > 1 and x.stride(d) % 8:
            raise ValueError("%s has stride %d along axis %d; the kernels need multiples of 8" % (name, x.stride(d), d))


def _pool(K_pages, V_pages):
    if not (K_pages.is_cuda and K_pages.dim() == 4 and K_pages.dtype in _DTYPES and K_pages.stride(3) == 1):
        raise ValueError("K_pages must be a 4-D fp16 or bf16 CUDA tensor [pages, kv_heads, page_size, head_dim] "
                         "with a contiguous last axis")
    _check_strides(K_pages, "K_pages", 3)
    if V_pages is not None:
        if (V_pages.dtype != K_pages.dtype or V_pages.shape != K_pages.shape or V_pages.device != K_pages.device
                or V_pages.stride() != K_pages.stride()):
            raise ValueError("V_pages must have K_pages' type, shape, strides and device")
        _check_strides(V_pages, "V_pages", 3)
    pages, heads, size, dim = K_pages.shape
    s = K_pages.stride()
    return _lib.Pool(_DTYPES[K_pages.dtype], pages, heads, size, dim, 0, s[0], s[1], s[2])


def page_map(ctx_lens, new_lens, free_pages, block_table, page_size, tokens, out=None):
    """Block table and slot map of a step from its lengths (device int32 [requests] each: tokens cached, tokens
    new).  New columns of block_table (int32 [requests, columns], updated in place) take the next entries of
    free_pages (int32), requests in order.  tokens: the step's room, at least the sum of new_lens (the rows past
    the sum are padding).  Returns a PageMap: q_start [requests + 1], kv_lens [requests], slots [tokens] (int64:
    page * page_size + offset, -1 for padding and for tokens without a page), positions [tokens] (-1 for padding) and
    counts [4]: new tokens, pages taken, pages the free list lacked, requests longer than their table row."""
    _check_vec(ctx_lens, "ctx_lens", torch.int32, None)
    dev, n = ctx_lens.device, ctx_lens.shape[0]
    _check_vec(new_lens, "new_lens", torch.int32, dev, n)
    _check_vec(free_pages, "free_pages", torch.int32, dev)
    _check_table(block_table, n, dev)
    if out is None:
        out = PageMap.empty(n, tokens, dev)
    else:
        _check_vec(out.q_start, "out.q_start", torch.int32, dev, n + 1)
        _check_vec(out.kv_lens, "out.kv_lens", torch.int32, dev, n)
        _check_vec(out.slots, "out.slots", torch.int64, dev, tokens)
        _check_vec(out.positions, "out.positions", torch.int32, dev, tokens)
        _check_vec(out.counts, "out.counts", torch.int32, dev, 4)
    _call(dev, "nq_page_map", ctx_lens.data_ptr(), new_lens.data_ptr(), n, free_pages.data_ptr(),
          free_pages.shape[0], block_table.data_ptr(), block_table.stride(0), block_table.shape[1], page_size, tokens,
          out.q_start.data_ptr(), out.kv_lens.data_ptr(), out.slots.data_ptr(), out.positions.data_ptr(),
          out.counts.data_ptr(), _stream_handle(dev))
    return out


def paged_append(K, V, K_pages, V_pages, slots):
    """Write K and V ([tokens, kv_heads, head_dim], strided) into the pools at slots (int64 [tokens], from
    page_map; slots outside the pool write nothing).  A decompressed cache [L, B, H, T, D] goes in as
    K[l, b].transpose(0, 1).  Returns the pools."""
    pool = _pool(K_pages, V_pages)
    dev = K_pages.device
    _check_rows(K, "K", pool.kv_heads, pool.head_dim, K_pages.dtype, dev)
    _check_rows(V, "V", pool.kv_heads, pool.head_dim, K_pages.dtype, dev, K.shape[0])
    _check_vec(slots, "slots", torch.int64, dev, K.shape[0])
    _call(dev, "nq_paged_append", K.data_ptr(), K.stride(0), K.stride(1), V.data_ptr(), V.stride(0), V.stride(1),
          K.shape[0], slots.data_ptr(), ctypes_ref(pool), K_pages.data_ptr(), V_pages.data_ptr(), _stream_handle(dev))
    return K_pages, V_pages


def _attention(Q, out, block_table, requests, max_q, scale, causal, window, head_dim):
    s = block_table.stride(0)
    qs, os = Q.stride(), out.stride()
    return _lib.Attention(Q.shape[0], Q.shape[1], requests, block_table.shape[1],
                          Q.shape[0] if max_q is None else max_q, int(bool(causal)), window,
                          head_dim ** -0.5 if scale is None else scale, s, qs[0], qs[1], os[0], os[1])


def paged_attention_workspace(Q, K_pages, block_table, max_q=None):
    """A scratch tensor for paged_attention calls with these shapes (None when they need none).  Reuse it across
    calls on one stream."""
    a = _attention(Q, Q, block_table, block_table.shape[0], max_q, None, True, 0, Q.shape[2])
    return workspace(_ws_bytes(a, _pool(K_pages, None)), Q.device)


def _ws_bytes(a, pool):
    need = ctypes.c_uint64(0)
    _lib.check("nq_paged_attention_workspace",
               _lib.lib().nq_paged_attention_workspace(ctypes_ref(a), ctypes_ref(pool), ctypes_ref(need)))
    return need.value


def paged_attention(Q, K_pages, V_pages, block_table, q_start, kv_lens, max_q=None, scale=None, causal=True,
                    window=0, out=None, lse=None, ws=None):
    """Attention of the step's tokens over the paged cache, their own keys included (append first).

    Q [tokens, q_heads, head_dim] of the pool's type, strided; request r's rows are q_start[r] .. q_start[r + 1], and
    its row i stands at position kv_lens[r] - n + i of n.  max_q: a bound on a request's rows, which picks the
    kernel (default: all rows; results do not depend on it).  scale: head_dim ** -0.5 by default.  causal: keys up to
    the row's own position.  window > 0: only the last `window` of those.  A row that sees nothing is 0.
    Returns out (as Q); with lse (float32 [tokens, q_heads], filled with the log of the sum of exponentials) (out,
    lse).  ws: scratch from paged_attention_workspace, allocated here when not given."""
    pool = _pool(K_pages, V_pages)
    dev = K_pages.device
    if Q.dim() != 3:
        raise ValueError("Q must be [tokens, q_heads, head_dim], got %s" % (tuple(Q.shape),))
    heads = Q.shape[1]
    _check_rows(Q, "Q", heads, pool.head_dim, K_pages.dtype, dev)
    if heads == 0 or heads % pool.kv_heads:
        raise ValueError("%d query heads cannot share %d KV heads" % (heads, pool.kv_heads))
    if out is None:
        out = torch.empty(Q.shape, dtype=Q.dtype, device=dev)
    _check_rows(out, "out", heads, pool.head_dim, K_pages.dtype, dev, Q.shape[0])
    _check_vec(kv_lens, "kv_lens", torch.int32, dev)
    n = kv_lens.shape[0]
    _check_vec(q_start, "q_start", torch.int32, dev, n + 1)
    _check_table(block_table, n, dev)
    if lse is not None and not (lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous() and
                                tuple(lse.shape) == (Q.shape[0], heads) and lse.device == dev):
        raise ValueError("lse must be a contiguous float32 tensor [tokens, q_heads] on the call's device")
    a = _attention(Q, out, block_table, n, max_q, scale, causal, window, pool.head_dim)
    need = _ws_bytes(a, pool)
    if ws is None:
        ws = workspace(need, dev)
    elif not (ws.is_cuda and ws.dtype == torch.uint8 and ws.is_contiguous() and ws.device == dev):
        raise ValueError("ws must be a contiguous uint8 CUDA tensor on the call's device")
    elif ws.numel() < need:
        raise ValueError("ws has %d bytes; the call needs %d" % (ws.numel(), need))
    _call(dev, "nq_paged_attention", ctypes_ref(a), Q.data_ptr(), ctypes_ref(pool), K_pages.data_ptr(),
          V_pages.data_ptr(), block_table.data_ptr(), q_start.data_ptr(), kv_lens.data_ptr(), out.data_ptr(),
          None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(),
          0 if ws is None else ws.numel(), _stream_handle(dev))
    return out if lse is None else (out, lse)


def paged_status(device=None):
    """Waits for the device's current stream; raises NQError when it failed or when an attention kernel gave up
    waiting for its loads (outputs since the last paged_status are then void)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    _call(dev, "nq_paged_status", _stream_handle(dev))
