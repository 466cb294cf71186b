"""Serving from the restored cache: K and V in pages, the step's tokens written into them and attending.

    m = page_map(ctx_lens, new_lens, free_pages, block_table, page_size, tokens)   # once a step
    for layer in ...:
        paged_append(K, V, K_pages[layer], V_pages[layer], m.slots)
        O = paged_attention(Q, K_pages[layer], V_pages[layer], block_table, m.q_start, m.kv_lens, max_q=...)

A pool is an fp16 or bf16 CUDA tensor [pages, kv_heads, page_size, head_dim] with any strides that are
multiples of 8 elements and a contiguous last axis: pages that are stored token-major
([pages, page_size, kv_heads, head_dim]) are passed as .transpose(1, 2).  Lengths, tables and slots stay on the
device: no call waits for the GPU, and a step can be captured as a CUDA graph (for one place in the free list, whose address page_map
is given).  All work is enqueued on the
current torch CUDA stream.
"""
import ctypes
import operator
import threading
from dataclasses import dataclass

import torch

from . import _lib
from .codec import _on, ctypes_ref, workspace

__all__ = ["PageMap", "page_map", "page_release", "paged_append", "paged_attention", "paged_attention_workspace",
           "paged_compact", "paged_status"]

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


# A step makes several of these calls per layer, and the GPU is done with a small one in ten microseconds.  So the checks of
# types, shapes, strides and devices run once for each combination of them, and what they yield is kept under that combination
# (never under a tensor or its address); a later call looks it up, checks its pointers and launches.
_KEPT, _KEPT_LOCK = {}, threading.Lock()


def _keep(key, checked):
    with _KEPT_LOCK:
        while len(_KEPT) >= 1024:
            del _KEPT[next(iter(_KEPT))]  # the oldest
        _KEPT[key] = checked
    return checked


def _meta(x):
    return x.dtype, x.shape, x.stride(), x.get_device()


def _launch(index, fn, *args):
    """One library call on the current stream of device `index`, with that device current."""
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with _on(index):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(fn.__name__, st)


_I32_MAX = 2 ** 31 - 1


def _bound(n):
    """A number that only bounds others, for a 32-bit argument (ctypes would keep its low 32 bits): past them, the largest; below
    zero, one that is refused."""
    return max(min(operator.index(n), _I32_MAX), -1)


def _check_size(n, name):
    if not 0 <= n <= _I32_MAX:
        raise ValueError("%s is %d; the kernels count in 32 bits" % (name, n))


def _check_vec(x, name, dtype, device, n):
    _check_size(n, "the length of %s" % name)
    if not (x.is_cuda and x.dtype == dtype and x.dim() == 1 and x.is_contiguous()):
        raise ValueError("%s must be a contiguous 1-D %s CUDA tensor" % (name, str(dtype)[6:]))
    if x.shape[0] != n:
        raise ValueError("%s has %d entries; the call needs %d" % (name, x.shape[0], n))
    if x.device != device:
        raise ValueError("%s is on %s; the call runs on %s" % (name, x.device, device))


def _check_table(table, requests, device):
    """Also that its columns fit 32 bits; its rows are `requests`, a length that was checked."""
    if not (table.is_cuda and table.dtype == torch.int32 and table.dim() == 2 and
            (table.stride(1) == 1 or table.shape[1] <= 1 or table.shape[0] == 0)):
        raise ValueError("block_table must be a 2-D int32 CUDA tensor with contiguous rows")
    if table.shape[0] != requests:
        raise ValueError("block_table has %d rows; there are %d requests" % (table.shape[0], requests))
    _check_size(table.shape[1], "the width of block_table")
    if table.device != device:
        raise ValueError("block_table is on %s; the call runs on %s" % (table.device, device))


def _check_rows(x, name, shape, dtype, device):
    """A [tokens, heads, dim] tensor whose rows the kernels read or write 16 bytes at a time."""
    if not (x.is_cuda and x.dtype == dtype and x.dim() == 3 and (x.stride(2) == 1 or x.numel() == 0)):
        raise ValueError("%s must be a 3-D %s CUDA tensor [tokens, heads, head_dim] with a contiguous last axis"
                         % (name, str(dtype)[6:]))
    if tuple(x.shape) != shape:
        raise ValueError("%s has shape %s; the call needs %s" % (name, tuple(x.shape), shape))
    if x.device != device:
        raise ValueError("%s is on %s; the call runs on %s" % (name, x.device, device))
    _check_strides(x, name, 2)


def _check_strides(x, name, axes):
    for d in range(axes):
        if x.shape[d] > 1 and x.stride(d) % 8:
            raise ValueError("%s has stride %d along axis %d; the kernels need multiples of 8" % (name, x.stride(d), d))


def _check_starts(**tensors):
    for name, x in tensors.items():
        if x.data_ptr() % 16:
            raise ValueError("%s must start on a 16-byte boundary" % name)


def _pool(K_pages, V_pages):
    """The pools' description."""
    if not (K_pages.is_cuda and K_pages.dim() == 4 and K_pages.dtype in _DTYPES and K_pages.stride(3) == 1):
        raise ValueError("K_pages must be a 4-D fp16 or bf16 CUDA tensor [pages, kv_heads, page_size, head_dim] "
                         "with a contiguous last axis")
    _check_strides(K_pages, "K_pages", 3)
    if V_pages is not None and (V_pages.dtype != K_pages.dtype or V_pages.shape != K_pages.shape or
                                V_pages.device != K_pages.device or V_pages.stride() != K_pages.stride()):
        raise ValueError("V_pages must have K_pages' type, shape, strides and device")
    for n in K_pages.shape:
        _check_size(n, "a size of K_pages")
    return _lib.Pool(_DTYPES[K_pages.dtype], *K_pages.shape, 0, *K_pages.stride()[:3])


def page_map(ctx_lens, new_lens, free_pages, block_table, page_size, tokens, out=None):
    """Block table and slot map of a step from its lengths (device int32 [requests] each: tokens cached, tokens
    new).  New columns of block_table (int32 [requests, columns], updated in place) take the next entries of
    free_pages (int32), requests in order.  tokens: the step's room, at least the sum of new_lens (the rows past
    the sum are padding; columns that only tokens past the room would begin stay as they are).  Returns a PageMap: q_start [requests + 1], kv_lens [requests], slots [tokens] (int64:
    page * page_size + offset, -1 for padding and for tokens without a page), positions [tokens] (-1 for padding) and
    counts [4]: new tokens, pages taken, pages the free list lacked, requests longer than their table row."""
    # the free list's length changes from step to step, and is checked here
    n_free = free_pages.numel()
    if n_free > _I32_MAX:
        _check_size(n_free, "the length of free_pages")
    key = ("map", page_size, tokens, *_meta(ctx_lens), *_meta(new_lens), *_meta(block_table), free_pages.dtype,
           free_pages.dim(), free_pages.is_contiguous(), free_pages.get_device())
    if out is not None:
        key += (*_meta(out.q_start), *_meta(out.kv_lens), *_meta(out.slots), *_meta(out.positions), *_meta(out.counts))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _check_map(ctx_lens, new_lens, free_pages, block_table, page_size, tokens, out))
    index, fn, n, cols, stride = kept
    if out is None:
        out = PageMap.empty(n, tokens, ctx_lens.device)
    _launch(index, fn, ctx_lens.data_ptr(), new_lens.data_ptr(), n, free_pages.data_ptr(), n_free, block_table.data_ptr(),
            stride, cols, page_size, tokens, out.q_start.data_ptr(), out.kv_lens.data_ptr(), out.slots.data_ptr(),
            out.positions.data_ptr(), out.counts.data_ptr())
    return out


def _check_map(ctx_lens, new_lens, free_pages, block_table, page_size, tokens, out):
    dev, n, i32 = ctx_lens.device, ctx_lens.numel(), torch.int32
    if page_size > 0:  # others are the library's to refuse
        _check_size(page_size, "page_size")
    _check_size(tokens, "tokens")
    _check_vec(ctx_lens, "ctx_lens", i32, dev, n)
    _check_vec(new_lens, "new_lens", i32, dev, n)
    _check_vec(free_pages, "free_pages", i32, dev, free_pages.numel())
    _check_table(block_table, n, dev)
    if out is not None:
        _check_vec(out.q_start, "out.q_start", i32, dev, n + 1)
        _check_vec(out.kv_lens, "out.kv_lens", i32, dev, n)
        _check_vec(out.slots, "out.slots", torch.int64, dev, tokens)
        _check_vec(out.positions, "out.positions", i32, dev, tokens)
        _check_vec(out.counts, "out.counts", i32, dev, 4)
    return dev.index, _lib.lib().nq_page_map, n, block_table.shape[1], block_table.stride(0)


def paged_append(K, V, K_pages, V_pages, slots):
    """Write K and V ([tokens, kv_heads, head_dim], strided) into the pools at slots (int64 [tokens], from
    page_map; slots outside the pool write nothing).  A decompressed cache [L, B, H, T, D] goes in as
    K[l, b].transpose(0, 1).  Returns the pools."""
    key = ("append", *_meta(K), *_meta(V), *_meta(K_pages), *_meta(V_pages), *_meta(slots))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _check_append(K, V, K_pages, V_pages, slots))
    index, fn, pool, tokens, kt, kh, vt, vh = kept
    k, v, kp, vp = K.data_ptr(), V.data_ptr(), K_pages.data_ptr(), V_pages.data_ptr()
    if (k | v | kp | vp) & 15:
        _check_starts(K=K, V=V, K_pages=K_pages, V_pages=V_pages)
    _launch(index, fn, k, kt, kh, v, vt, vh, tokens, slots.data_ptr(), pool, kp, vp)
    return K_pages, V_pages


def _check_append(K, V, K_pages, V_pages, slots):
    pool, dev = _pool(K_pages, V_pages), K_pages.device
    shape = (K.shape[0], pool.kv_heads, pool.head_dim)
    _check_rows(K, "K", shape, K_pages.dtype, dev)
    _check_rows(V, "V", shape, K_pages.dtype, dev)
    _check_vec(slots, "slots", torch.int64, dev, shape[0])
    return (dev.index, _lib.lib().nq_paged_append, ctypes_ref(pool), shape[0], K.stride(0), K.stride(1), V.stride(0),
            V.stride(1))


def _attention(Q, out, K_pages, V_pages, block_table, requests, max_q, scale, causal, window):
    """(the pools' description, the call's, the workspace that it needs); out = None: a contiguous one"""
    pool = _pool(K_pages, V_pages)
    out_stride = (Q.shape[1] * Q.shape[2], Q.shape[2]) if out is None else out.stride()
    a = _lib.Attention(Q.shape[0], Q.shape[1], requests, block_table.shape[1], Q.shape[0] if max_q is None else max_q,
                       causal, window, Q.shape[2] ** -0.5 if scale is None else scale, block_table.stride(0), Q.stride(0),
                       Q.stride(1), out_stride[0], out_stride[1])
    need = ctypes.c_uint64(0)
    _lib.check("nq_paged_attention_workspace", _lib.lib().nq_paged_attention_workspace(
        ctypes_ref(a), ctypes_ref(pool), ctypes_ref(need)))
    return pool, a, need.value


def paged_attention_workspace(Q, K_pages, block_table, max_q=None):
    """A scratch tensor for paged_attention calls with these shapes (None when they need none).  Reuse it across
    calls on one stream."""
    if max_q is not None:
        max_q = _bound(max_q)
    return workspace(_attention(Q, Q, K_pages, None, block_table, block_table.shape[0], max_q, None, 1, 0)[2], Q.device)


def paged_attention(Q, K_pages, V_pages, block_table, q_start, kv_lens, max_q=None, scale=None, causal=True,
                    window=0, out=None, lse=None, ws=None, tree=None):
    """Attention of the step's tokens over the paged cache, their own keys included (append first).

    Q [tokens, q_heads, head_dim] of the pool's type, strided; request r's rows are q_start[r] .. q_start[r + 1], and
    its row i stands at position kv_lens[r] - n + i of n.  max_q: a bound on a request's rows, which picks the
    kernel (default: all rows; results do not depend on it).  scale: head_dim ** -0.5 by default.  causal: keys up to
    the row's own position.  window > 0: only the last `window` of those.  A row that sees nothing is 0; rows of no
    request (a padded step's) are not written.
    tree: the DraftTree of a step whose rows are drafted trees: a row sees the request's cached tokens (the last `window` before
    its position) and, of the drafted ones, those that its bits name up to itself.
    Returns out (as Q); with lse (float32 [tokens, q_heads], filled with the log of the sum of exponentials) (out,
    lse).  ws: scratch from paged_attention_workspace, allocated here when not given."""
    if max_q is not None and (type(max_q) is not int or not 0 <= max_q <= _I32_MAX):
        max_q = _bound(max_q)
    if type(window) is not int or not 0 <= window <= _I32_MAX:
        window = _bound(window)
    if scale is not None and type(scale) is not float:
        scale = float(scale)
    causal = 1 if causal else 0
    key = ("attention", max_q, scale, causal, window, *_meta(Q), *_meta(K_pages), *_meta(V_pages), *_meta(block_table),
           *_meta(q_start), *_meta(kv_lens), None if out is None else _meta(out), None if lse is None else _meta(lse))
    if tree is not None:
        key += (*_meta(tree.ancestors), *_meta(tree.positions))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _check_attention(Q, K_pages, V_pages, block_table, q_start, kv_lens, max_q, scale, causal, window,
                                           out, lse, tree))
    index, fn, pool, a, need = kept
    if out is None:
        out = torch.empty(Q.shape, dtype=Q.dtype, device=Q.device)
    q, k, v, o = Q.data_ptr(), K_pages.data_ptr(), V_pages.data_ptr(), out.data_ptr()
    if (q | k | v | o) & 15:
        _check_starts(Q=Q, K_pages=K_pages, V_pages=V_pages, out=out)
    what = (a,) if tree is None else (a, tree.ancestors.data_ptr(), tree.positions.data_ptr(), tree.ancestors.shape[1])
    args = (*what, q, pool, k, v, block_table.data_ptr(), q_start.data_ptr(), kv_lens.data_ptr(), o,
            None if lse is None else lse.data_ptr())
    if ws is not None:
        if not (ws.is_cuda and ws.dtype == torch.uint8 and ws.is_contiguous() and ws.device == Q.device):
            raise ValueError("ws must be a contiguous uint8 CUDA tensor on the call's device")
        if ws.numel() < need:
            raise ValueError("ws has %d bytes; the call needs %d" % (ws.numel(), need))
        _launch(index, fn, *args, ws.data_ptr(), ws.numel())
    elif torch._C._cuda_getDevice() == index:
        # straight from torch's allocator, in stream order (and into a graph's own memory) like a tensor's: making and dropping the tensor
        # would take 6 us of a call's 20
        scratch = torch._C._cuda_cudaCachingAllocator_raw_alloc(need, torch._C._cuda_getCurrentRawStream(index))
        try:
            _launch(index, fn, *args, scratch, need)
        finally:
            torch._C._cuda_cudaCachingAllocator_raw_delete(scratch)
    else:
        ws = torch.empty(need, dtype=torch.uint8, device=Q.device)
        _launch(index, fn, *args, ws.data_ptr(), need)
    return out if lse is None else (out, lse)


def _check_attention(Q, K_pages, V_pages, block_table, q_start, kv_lens, max_q, scale, causal, window, out, lse,
                     tree=None):
    pool, dev, dtype = _pool(K_pages, V_pages), K_pages.device, K_pages.dtype
    if Q.dim() != 3:
        raise ValueError("Q must be [tokens, q_heads, head_dim], got %s" % (tuple(Q.shape),))
    tokens, heads = Q.shape[0], Q.shape[1]
    _check_size(tokens, "the length of Q")
    if heads == 0 or heads % pool.kv_heads:
        raise ValueError("%d query heads cannot share %d KV heads" % (heads, pool.kv_heads))
    shape = (tokens, heads, pool.head_dim)
    _check_rows(Q, "Q", shape, dtype, dev)
    if out is not None:
        _check_rows(out, "out", shape, dtype, dev)
    n = kv_lens.numel()
    _check_vec(kv_lens, "kv_lens", torch.int32, dev, n)
    _check_vec(q_start, "q_start", torch.int32, dev, n + 1)
    _check_table(block_table, n, dev)
    if lse is not None and not (lse.dtype == torch.float32 and lse.is_contiguous() and tuple(lse.shape) == (tokens, heads) and
                                lse.device == dev):
        raise ValueError("lse must be a contiguous float32 tensor [tokens, q_heads] on the call's device")
    fn = _lib.lib().nq_paged_attention
    if tree is not None:
        check_tree(tree, tokens, dev)
        if not causal:
            raise ValueError("a drafted tree is causal: every token sees its ancestors")
        fn = _lib.lib().nq_paged_tree_attention
    pool, a, need = _attention(Q, out, K_pages, V_pages, block_table, n, max_q, scale, causal, window)
    return dev.index, fn, ctypes_ref(pool), ctypes_ref(a), need


def check_tree(tree, tokens, device, name="tree"):
    """A DraftTree's tensors, whose width the caller may read afterwards."""
    bits = tree.ancestors
    if not (bits.is_cuda and bits.dtype == torch.int64 and bits.dim() == 2 and bits.is_contiguous()):
        raise ValueError("%s.ancestors must be a contiguous 2-D int64 CUDA tensor [tokens, words]" % name)
    if bits.shape[0] != tokens or not 1 <= bits.shape[1] <= _lib.NQ_TREE_WORDS:
        raise ValueError("%s.ancestors has shape %s; the call needs %d rows of 1 to %d words"
                         % (name, tuple(bits.shape), tokens, _lib.NQ_TREE_WORDS))
    if bits.device != device:
        raise ValueError("%s.ancestors is on %s; the call runs on %s" % (name, bits.device, device))
    _check_vec(tree.positions, name + ".positions", torch.int32, device, tokens)


def paged_compact(K_pages, V_pages, block_table, q_start, kv_lens, path):
    """Move the accepted rows of a step's drafted tokens to the front of their requests' rows, in all layers at once.

    Pools as elsewhere, or [layers, pages, kv_heads, page_size, head_dim].  q_start and kv_lens are the step's; path
    (int32 [tokens], from verify_drafts) holds at a request's rows the accepted ones in order: its k-th entry's K and V become
    row k's, up to the first entry that does not increase (-1 behind the last).  Returns the pools."""
    key = ("compact", *_meta(K_pages), *_meta(V_pages), *_meta(block_table), *_meta(q_start), *_meta(kv_lens), *_meta(path))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _check_compact(K_pages, V_pages, block_table, q_start, kv_lens, path))
    index, fn, pool, layers, layer_stride, stride, cols, requests, tokens = kept
    k, v = K_pages.data_ptr(), V_pages.data_ptr()
    if (k | v) & 15:
        _check_starts(K_pages=K_pages, V_pages=V_pages)
    _launch(index, fn, pool, layers, layer_stride, k, v, block_table.data_ptr(), stride, cols, q_start.data_ptr(),
            kv_lens.data_ptr(), requests, path.data_ptr(), tokens)
    return K_pages, V_pages


def _check_compact(K_pages, V_pages, block_table, q_start, kv_lens, path):
    layers = layer_stride = 0
    if K_pages.dim() == 5:
        layers, layer_stride = K_pages.shape[0], K_pages.stride(0)
        _check_size(layers, "the layers of K_pages")
        if V_pages.dim() != 5 or V_pages.shape[0] != layers or V_pages.stride(0) != layer_stride:
            raise ValueError("V_pages must have K_pages' type, shape, strides and device")
        if layers == 0:
            raise ValueError("K_pages has no layers")
        if layers > 1 and layer_stride % 8:
            raise ValueError("K_pages has stride %d along axis 0; the kernels need multiples of 8" % layer_stride)
        pool = _pool(K_pages[0], V_pages[0])
    else:
        pool = _pool(K_pages, V_pages)
    dev, n = K_pages.device, kv_lens.numel()
    _check_vec(path, "path", torch.int32, dev, path.numel())
    _check_vec(kv_lens, "kv_lens", torch.int32, dev, n)
    _check_vec(q_start, "q_start", torch.int32, dev, n + 1)
    _check_table(block_table, n, dev)
    return (dev.index, _lib.lib().nq_paged_compact, ctypes_ref(pool), max(layers, 1), layer_stride, block_table.stride(0),
            block_table.shape[1], n, path.shape[0])


def page_release(block_table, kv_lens, keep_lens, page_size, free_pages, top, out=None, clear=False):
    """Give back the pages past the tokens that requests keep (device int32 [requests] each: tokens with pages, tokens to keep).

    free_pages (int32, updated in place) is the whole free list, a stack whose free part begins at `top`: free_pages[top:] is what
    page_map is given.  The k-th released page, requests and columns in order, goes to free_pages[top - 1 - k]; columns that never
    got a page (entries below zero) give none back.
    Returns counts [2]: pages released, those that found no room (top is lower by the difference).  The table stays as it is; with
    clear, columns whose pages went on the list become -1, as they must where a later step may bring more tokens than its room
    (page_map writes no column for those, and the old entry would name a page that another request has by then)."""
    n_free = free_pages.numel()
    if not 0 <= top <= n_free or n_free > _I32_MAX:
        raise ValueError("top is %d; free_pages has %d entries" % (top, n_free))
    clear = bool(clear)
    key = ("release", page_size, clear, *_meta(block_table), *_meta(kv_lens), *_meta(keep_lens), free_pages.dtype, free_pages.dim(),
           free_pages.is_contiguous(), free_pages.get_device(), None if out is None else _meta(out))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _check_release(block_table, kv_lens, keep_lens, page_size, free_pages, out, clear))
    index, fn, n, cols, stride = kept
    if out is None:
        out = torch.empty(2, dtype=torch.int32, device=kv_lens.device)
    _launch(index, fn, block_table.data_ptr(), stride, cols, kv_lens.data_ptr(), keep_lens.data_ptr(), n, page_size,
            free_pages.data_ptr(), operator.index(top), out.data_ptr())
    return out


def _check_release(block_table, kv_lens, keep_lens, page_size, free_pages, out, clear):
    dev, n, i32 = kv_lens.device, kv_lens.numel(), torch.int32
    if page_size > 0:  # others are the library's to refuse
        _check_size(page_size, "page_size")
    _check_vec(kv_lens, "kv_lens", i32, dev, n)
    _check_vec(keep_lens, "keep_lens", i32, dev, n)
    _check_vec(free_pages, "free_pages", i32, dev, free_pages.numel())
    _check_table(block_table, n, dev)
    if out is not None:
        _check_vec(out, "out", i32, dev, 2)
    fn = _lib.lib().nq_page_release_clear if clear else _lib.lib().nq_page_release
    return dev.index, fn, n, block_table.shape[1], block_table.stride(0)


def paged_status(device=None):
    """Waits for the device's current stream; raises NQError when it failed or when an attention kernel gave up
    waiting for its loads (outputs since the last paged_status are then void)."""
    dev = torch.device("cuda" if device is None else device)
    if dev.type != "cuda":
        raise ValueError("paged_status needs a CUDA device, got %s" % dev)
    _launch(torch.cuda.current_device() if dev.index is None else dev.index, _lib.lib().nq_paged_status)
