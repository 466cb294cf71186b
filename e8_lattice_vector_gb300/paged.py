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
import functools
from dataclasses import dataclass

import torch

from . import _lib
from .codec import _on, ctypes_ref, workspace

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


def _launch(device, name, *args):
    """One library call on the device's current stream, with the device current (a step makes several such calls per
    layer, and the GPU is done with a small one in microseconds: nothing here that is not needed)."""
    fn, index = getattr(_lib.lib(), name), device.index
    if torch.cuda.current_device() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with _on(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(name, st)


def _check_vec(x, name, dtype, device, n):
    if x.dtype is dtype and x.shape == (n,) and x.is_contiguous() and x.device == device and x.is_cuda:
        return
    if not (x.is_cuda and x.dtype == dtype and x.dim() == 1 and x.is_contiguous()):
        raise ValueError("%s must be a contiguous 1-D %s CUDA tensor" % (name, str(dtype)[6:]))
    if x.shape[0] != n:
        raise ValueError("%s has %d entries; the call needs %d" % (name, x.shape[0], n))
    raise ValueError("%s is on %s; the call runs on %s" % (name, x.device, device))


def _check_table(table, requests, device):
    """(columns, row stride)"""
    if not (table.is_cuda and table.dtype is torch.int32 and table.dim() == 2 and
            (table.stride(1) == 1 or table.shape[1] <= 1 or table.shape[0] == 0)):
        raise ValueError("block_table must be a 2-D int32 CUDA tensor with contiguous rows")
    rows, cols = table.shape
    if rows != requests:
        raise ValueError("block_table has %d rows; there are %d requests" % (rows, requests))
    if table.device != device:
        raise ValueError("block_table is on %s; the call runs on %s" % (table.device, device))
    return cols, table.stride(0)


def _check_rows(x, name, shape, dtype, device):
    """A [tokens, heads, dim] tensor whose rows the kernels read or write 16 bytes at a time; its strides."""
    stride = x.stride()
    if not (x.is_cuda and x.dtype is dtype and len(stride) == 3 and (stride[2] == 1 or x.numel() == 0)):
        raise ValueError("%s must be a 3-D %s CUDA tensor [tokens, heads, head_dim] with a contiguous last axis"
                         % (name, str(dtype)[6:]))
    if x.shape != shape:
        raise ValueError("%s has shape %s; the call needs %s" % (name, tuple(x.shape), tuple(shape)))
    if x.device != device:
        raise ValueError("%s is on %s; the call runs on %s" % (name, x.device, device))
    if stride[0] % 8 or stride[1] % 8:
        _check_strides(name, shape, stride)
    if x.data_ptr() % 16:
        raise ValueError("%s must start on a 16-byte boundary" % name)
    return stride


def _check_strides(name, shape, stride):
    for d in range(len(shape) - 1):
        if shape[d] > 1 and stride[d] % 8:
            raise ValueError("%s has stride %d along axis %d; the kernels need multiples of 8" % (name, stride[d], d))


@functools.lru_cache(maxsize=256)
def _pool_struct(dtype, shape, stride):
    _check_strides("K_pages", shape, stride)
    return _lib.Pool(_DTYPES[dtype], *shape, 0, *stride[:3])


def _pool(K_pages, V_pages):
    """(the pool's description, its device)"""
    dtype, stride, dev = K_pages.dtype, K_pages.stride(), K_pages.device
    if not (K_pages.is_cuda and dtype in _DTYPES and len(stride) == 4 and stride[3] == 1):
        raise ValueError("K_pages must be a 4-D fp16 or bf16 CUDA tensor [pages, kv_heads, page_size, head_dim] "
                         "with a contiguous last axis")
    pool = _pool_struct(dtype, K_pages.shape, stride)
    if V_pages is not None and (V_pages.dtype is not dtype or V_pages.shape != K_pages.shape or
                                V_pages.device != dev or V_pages.stride() != stride):
        raise ValueError("V_pages must have K_pages' type, shape, strides and device")
    for x, name in ((K_pages, "K_pages"), (V_pages, "V_pages")):
        if x is not None and x.data_ptr() % 16:
            raise ValueError("%s must start on a 16-byte boundary" % name)
    return pool, dev


def page_map(ctx_lens, new_lens, free_pages, block_table, page_size, tokens, out=None):
    """Block table and slot map of a step from its lengths (device int32 [requests] each: tokens cached, tokens
    new).  New columns of block_table (int32 [requests, columns], updated in place) take the next entries of
    free_pages (int32), requests in order.  tokens: the step's room, at least the sum of new_lens (the rows past
    the sum are padding).  Returns a PageMap: q_start [requests + 1], kv_lens [requests], slots [tokens] (int64:
    page * page_size + offset, -1 for padding and for tokens without a page), positions [tokens] (-1 for padding) and
    counts [4]: new tokens, pages taken, pages the free list lacked, requests longer than their table row."""
    dev, n = ctx_lens.device, ctx_lens.numel()
    i32 = torch.int32
    _check_vec(ctx_lens, "ctx_lens", i32, dev, n)
    _check_vec(new_lens, "new_lens", i32, dev, n)
    n_free = free_pages.numel()
    _check_vec(free_pages, "free_pages", i32, dev, n_free)
    cols, stride = _check_table(block_table, n, dev)
    if out is None:
        out = PageMap.empty(n, tokens, dev)
    else:
        _check_vec(out.q_start, "out.q_start", i32, dev, n + 1)
        _check_vec(out.kv_lens, "out.kv_lens", i32, dev, n)
        _check_vec(out.slots, "out.slots", torch.int64, dev, tokens)
        _check_vec(out.positions, "out.positions", i32, dev, tokens)
        _check_vec(out.counts, "out.counts", i32, dev, 4)
    _launch(dev, "nq_page_map", ctx_lens.data_ptr(), new_lens.data_ptr(), n, free_pages.data_ptr(), n_free,
            block_table.data_ptr(), stride, cols, page_size, tokens, out.q_start.data_ptr(), out.kv_lens.data_ptr(),
            out.slots.data_ptr(), out.positions.data_ptr(), out.counts.data_ptr())
    return out


def paged_append(K, V, K_pages, V_pages, slots):
    """Write K and V ([tokens, kv_heads, head_dim], strided) into the pools at slots (int64 [tokens], from
    page_map; slots outside the pool write nothing).  A decompressed cache [L, B, H, T, D] goes in as
    K[l, b].transpose(0, 1).  Returns the pools."""
    pool, dev = _pool(K_pages, V_pages)
    shape = (K.shape[0], pool.kv_heads, pool.head_dim)
    ks = _check_rows(K, "K", shape, K_pages.dtype, dev)
    vs = _check_rows(V, "V", shape, K_pages.dtype, dev)
    _check_vec(slots, "slots", torch.int64, dev, shape[0])
    _launch(dev, "nq_paged_append", K.data_ptr(), ks[0], ks[1], V.data_ptr(), vs[0], vs[1], shape[0], slots.data_ptr(),
            ctypes_ref(pool), K_pages.data_ptr(), V_pages.data_ptr())
    return K_pages, V_pages


@functools.lru_cache(maxsize=256)
def _attention_struct(dtype, pool_shape, pool_stride, shape, q_stride, out_stride, requests, cols, table_stride, max_q,
                      scale, causal, window):
    """(the call's description, the workspace that it needs): from sizes, strides and types alone."""
    a = _lib.Attention(shape[0], shape[1], requests, cols, shape[0] if max_q is None else max_q, int(bool(causal)), window,
                       shape[2] ** -0.5 if scale is None else scale, table_stride, q_stride[0], q_stride[1],
                       out_stride[0], out_stride[1])
    need = ctypes.c_uint64(0)
    _lib.check("nq_paged_attention_workspace", _lib.lib().nq_paged_attention_workspace(
        ctypes_ref(a), ctypes_ref(_pool_struct(dtype, pool_shape, pool_stride)), ctypes_ref(need)))
    return a, need.value


def paged_attention_workspace(Q, K_pages, block_table, max_q=None):
    """A scratch tensor for paged_attention calls with these shapes (None when they need none).  Reuse it across
    calls on one stream."""
    _pool(K_pages, None)
    _, need = _attention_struct(K_pages.dtype, K_pages.shape, K_pages.stride(), Q.shape, Q.stride(), Q.stride(),
                                block_table.shape[0], block_table.shape[1], block_table.stride(0), max_q, None, True, 0)
    return workspace(need, Q.device)


def paged_attention(Q, K_pages, V_pages, block_table, q_start, kv_lens, max_q=None, scale=None, causal=True,
                    window=0, out=None, lse=None, ws=None):
    """Attention of the step's tokens over the paged cache, their own keys included (append first).

    Q [tokens, q_heads, head_dim] of the pool's type, strided; request r's rows are q_start[r] .. q_start[r + 1], and
    its row i stands at position kv_lens[r] - n + i of n.  max_q: a bound on a request's rows, which picks the
    kernel (default: all rows; results do not depend on it).  scale: head_dim ** -0.5 by default.  causal: keys up to
    the row's own position.  window > 0: only the last `window` of those.  A row that sees nothing is 0.
    Returns out (as Q); with lse (float32 [tokens, q_heads], filled with the log of the sum of exponentials) (out,
    lse).  ws: scratch from paged_attention_workspace, allocated here when not given."""
    pool, dev = _pool(K_pages, V_pages)
    dtype, shape = K_pages.dtype, Q.shape
    if len(shape) != 3:
        raise ValueError("Q must be [tokens, q_heads, head_dim], got %s" % (tuple(shape),))
    tokens, heads = shape[0], shape[1]
    if heads == 0 or heads % pool.kv_heads:
        raise ValueError("%d query heads cannot share %d KV heads" % (heads, pool.kv_heads))
    shape = (tokens, heads, pool.head_dim)
    q_stride = _check_rows(Q, "Q", shape, dtype, dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    out_stride = _check_rows(out, "out", shape, dtype, dev)
    n = kv_lens.numel()
    _check_vec(kv_lens, "kv_lens", torch.int32, dev, n)
    _check_vec(q_start, "q_start", torch.int32, dev, n + 1)
    cols, table_stride = _check_table(block_table, n, dev)
    if lse is not None and not (lse.dtype is torch.float32 and lse.is_contiguous() and lse.shape == (tokens, heads) and
                                lse.device == dev):
        raise ValueError("lse must be a contiguous float32 tensor [tokens, q_heads] on the call's device")
    a, need = _attention_struct(dtype, K_pages.shape, K_pages.stride(), shape, q_stride, out_stride, n, cols, table_stride,
                                max_q, scale, causal, window)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not (ws.is_cuda and ws.dtype is torch.uint8 and ws.is_contiguous() and ws.device == dev):
        raise ValueError("ws must be a contiguous uint8 CUDA tensor on the call's device")
    elif ws.numel() < need:
        raise ValueError("ws has %d bytes; the call needs %d" % (ws.numel(), need))
    _launch(dev, "nq_paged_attention", ctypes_ref(a), Q.data_ptr(), ctypes_ref(pool), K_pages.data_ptr(),
            V_pages.data_ptr(), block_table.data_ptr(), q_start.data_ptr(), kv_lens.data_ptr(), out.data_ptr(),
            None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel())
    return out if lse is None else (out, lse)


def paged_status(device=None):
    """Waits for the device's current stream; raises NQError when it failed or when an attention kernel gave up
    waiting for its loads (outputs since the last paged_status are then void)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    _launch(dev, "nq_paged_status")
