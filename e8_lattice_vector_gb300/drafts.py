"""Drafted token trees: their map, and their verification against the model's probabilities.

    m = page_map(ctx_lens, new_lens, free_pages[top:], block_table, page_size, tokens)      # once a step
    t = draft_tree(parents, m.q_start, m.kv_lens, max_q)                                    # t.positions: for the rotary embedding
    for layer in ...:
        paged_append(K, V, K_pages[layer], V_pages[layer], m.slots)
        O = paged_attention(Q, K_pages[layer], V_pages[layer], block_table, m.q_start, m.kv_lens, max_q=max_q, tree=t)
    v = verify_drafts(probs, tokens, parents, m.q_start, uniform, draft_probs)              # v.tokens: the step's answer
    paged_compact(K_pages, V_pages, block_table, m.q_start, m.kv_lens, v.path)              # all layers
    page_release(block_table, m.kv_lens, ctx_lens + v.accepted, page_size, free_pages, top)

A request's rows are its tree's nodes, the root first and every node after its parent.  The root is the token that the last step
ended with: certain, but not cached yet.  Nothing here waits for the GPU, and a step can be captured as a CUDA graph.  The graph
holds for one `top`: page_map has the address of free_pages[top:] and page_release the number, while how far `top` moves is in their
counts on the device.  Steps that follow each other are replayed from one graph only without these two, which are called around it.
"""
from dataclasses import dataclass

import torch

from . import _lib
from .paged import _KEPT, _bound, _check_size, _check_vec, _keep, _launch, _meta, check_tree

__all__ = ["DraftTree", "Verdict", "draft_tree", "verify_drafts"]

_DTYPES = {torch.float16: _lib.NQ_F16, torch.bfloat16: _lib.NQ_BF16, torch.float32: _lib.NQ_F32}


@dataclass(frozen=True)
class DraftTree:
    """What draft_tree leaves of a step's trees (see there)."""

    ancestors: torch.Tensor
    positions: torch.Tensor

    @classmethod
    def empty(cls, tokens, max_q, device="cuda"):
        """Uninitialised buffers for steps of `tokens` rows, at most max_q of them a request's."""
        return cls(torch.empty((tokens, max(-(-max_q // 64), 1)), dtype=torch.int64, device=device),
                   torch.empty(tokens, dtype=torch.int32, device=device))


@dataclass(frozen=True)
class Verdict:
    """What verify_drafts leaves of a step (see there)."""

    accepted: torch.Tensor
    path: torch.Tensor
    tokens: torch.Tensor

    @classmethod
    def empty(cls, requests, tokens, device="cuda"):
        """Uninitialised buffers for steps of `requests` requests and `tokens` rows."""
        return cls(*(torch.empty(n, dtype=torch.int32, device=device) for n in (requests, tokens, tokens)))


def draft_tree(parents, q_start, kv_lens, max_q, window=0, out=None):
    """Which drafted tokens each one sees, and where it stands.

    parents (int32 [tokens]): each node's parent as a number in its request's rows, -1 for a node that follows the cached
    tokens (so does any number that is not below the node's own).  q_start and kv_lens: the step's, from page_map.  max_q: a bound
    on a request's rows, at most 4096.  window > 0: only ancestors fewer than `window` levels up count.
    Returns a DraftTree: ancestors (int64 [tokens, ceil(max_q / 64)]: bit j & 63 of word j >> 6 for the node itself and each of its
    ancestors j) and positions (int32 [tokens]: cached tokens + ancestors).  Rows of no request are not written."""
    if not 0 <= max_q <= 64 * _lib.NQ_TREE_WORDS:
        raise ValueError("max_q is %d; a tree has at most %d nodes" % (max_q, 64 * _lib.NQ_TREE_WORDS))
    if window < 0:
        raise ValueError("window is %d; 0 means none" % window)
    window = _bound(window)
    key = ("tree", max_q, window, *_meta(parents), *_meta(q_start), *_meta(kv_lens))
    if out is not None:
        key += (*_meta(out.ancestors), *_meta(out.positions))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _check_draft_tree(parents, q_start, kv_lens, max_q, out))
    index, fn, tokens, requests, words = kept
    if out is None:
        out = DraftTree.empty(tokens, max_q, parents.device)
    _launch(index, fn, parents.data_ptr(), tokens, q_start.data_ptr(), kv_lens.data_ptr(), requests, window, words,
            out.ancestors.data_ptr(), out.positions.data_ptr())
    return out


def _check_draft_tree(parents, q_start, kv_lens, max_q, out):
    dev, tokens, n, i32 = parents.device, parents.numel(), kv_lens.numel(), torch.int32
    _check_vec(parents, "parents", i32, dev, tokens)
    _check_vec(kv_lens, "kv_lens", i32, dev, n)
    _check_vec(q_start, "q_start", i32, dev, n + 1)
    words = max(-(-max_q // 64), 1)
    if out is not None:
        check_tree(out, tokens, dev, "out")
        if out.ancestors.shape[1] != words:
            raise ValueError("out.ancestors has %d words; the call needs %d" % (out.ancestors.shape[1], words))
    return dev.index, _lib.lib().nq_draft_tree, tokens, n, words


def verify_drafts(probs, tokens, parents, q_start, uniform, draft_probs=None, out=None):
    """Which drafted tokens the model's probabilities accept, and the token that follows them.

    probs [tokens, vocab] (fp32, fp16 or bf16, rows contiguous): row i holds the model's probabilities of the token after node i.
    tokens (int32 [tokens]): the nodes' tokens, the root's first; one outside the vocabulary is no draft.  parents and q_start
    as in draft_tree.  uniform (float32 [tokens], in [0, 1)): a number for each draft at its row, and for the token that
    follows at the request's first row.  draft_probs (as probs): the draft's probabilities, whose row i the children of node i were
    drawn from, each independently; None when they were not drawn but chosen.
    From the root on, a node's children are accepted with probability p / q each in turn, what is left of p after a rejection being
    max(p - q, 0), normalised; the walk goes on from the accepted child, and the token that follows the last one is drawn from what is
    left.  So the results are distributed as the model's own.
    Returns a Verdict: accepted (int32 [requests]: accepted nodes, the root included), path (int32 [tokens]: their numbers at the
    request's rows, then -1) and tokens (int32 [tokens]: the tokens that the step adds, `accepted` of them, then -1).  Rows of
    no request are not written."""
    key = ("verify", *_meta(probs), *_meta(tokens), *_meta(parents), *_meta(q_start), *_meta(uniform),
           None if draft_probs is None else _meta(draft_probs))
    if out is not None:
        key += (*_meta(out.accepted), *_meta(out.path), *_meta(out.tokens))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _check_verify(probs, tokens, parents, q_start, uniform, draft_probs, out))
    index, fn, stride, draft_stride, dtype, vocab, rows, requests = kept
    if out is None:
        out = Verdict.empty(requests, rows, probs.device)
    _launch(index, fn, probs.data_ptr(), stride, None if draft_probs is None else draft_probs.data_ptr(), draft_stride, dtype, vocab,
            tokens.data_ptr(), parents.data_ptr(), uniform.data_ptr(), rows, q_start.data_ptr(), requests,
            out.accepted.data_ptr(), out.path.data_ptr(), out.tokens.data_ptr())
    return out


def _check_probs(x, name, like=None):
    if not (x.is_cuda and x.dim() == 2 and x.dtype in _DTYPES and (x.stride(1) == 1 or x.shape[1] <= 1)):
        raise ValueError("%s must be a 2-D fp32, fp16 or bf16 CUDA tensor [tokens, vocab] with contiguous rows" % name)
    if like is not None and (x.dtype != like.dtype or x.shape != like.shape or x.device != like.device):
        raise ValueError("%s must have probs' type, shape and device" % name)


def _check_verify(probs, tokens, parents, q_start, uniform, draft_probs, out):
    _check_probs(probs, "probs")
    dev, i32 = probs.device, torch.int32
    rows, vocab = probs.shape
    n = q_start.numel() - 1
    if n < 0:
        raise ValueError("q_start has no entries; the call needs one more than requests")
    if draft_probs is not None:
        _check_probs(draft_probs, "draft_probs", probs)
    _check_size(vocab, "the width of probs")
    _check_vec(tokens, "tokens", i32, dev, rows)
    _check_vec(parents, "parents", i32, dev, rows)
    _check_vec(uniform, "uniform", torch.float32, dev, rows)
    _check_vec(q_start, "q_start", i32, dev, n + 1)
    if out is not None:
        _check_vec(out.accepted, "out.accepted", i32, dev, n)
        _check_vec(out.path, "out.path", i32, dev, rows)
        _check_vec(out.tokens, "out.tokens", i32, dev, rows)
    return (dev.index, _lib.lib().nq_verify_drafts, probs.stride(0), 0 if draft_probs is None else draft_probs.stride(0),
            _DTYPES[probs.dtype], vocab, rows, n)
