"""Serving from a compressed cache: what the paged operators do together with the codec.

    python -m e8_lattice_vector_gb300.serve --config tiny --steps 4 --new 1
    python -m e8_lattice_vector_gb300.serve --config tiny --steps 4 --tree 8

A prompt's cache is compressed and decompressed, put into pages, and then served from: every step maps the new tokens
of each request to slots, appends their keys and values and lets them attend over everything cached, layer by
layer.  The same steps also run over the cache as it was before compression; the relative difference of the two attention
outputs says what the code's loss costs where it is used.  The synthetic caches of synth.py stand in for a
model's, and random queries, keys and values for its new tokens.

With --tree every request brings a tree of drafted tokens instead: the step maps and attends to the trees, verifies them
against the model's probabilities (random ones again), keeps the accepted rows and gives back the pages of the others.
"""
import argparse
import json
import random
from dataclasses import dataclass

import torch

from . import _lib
from .codec import RopeTable, compress_kv, decompress_kv
from .drafts import DraftTree, draft_tree, verify_drafts
from .paged import (PageMap, page_map, page_release, paged_append, paged_attention, paged_attention_workspace,
                    paged_compact, paged_status)
from .synth import CONFIGS, make_cache


@dataclass(frozen=True)
class DraftStep:
    """A step of drafted trees that has been mapped: its pages and slots, its trees, each node's parent, and nodes per request."""

    map: PageMap
    tree: DraftTree
    parents: torch.Tensor
    nodes: list


class PagedCache:
    """One layer stack's pools, block table and free list for a fixed set of requests."""

    def __init__(self, layers, requests, kv_heads, head_dim, page_size, max_tokens, dtype, device):
        self.page_size, self.columns = page_size, -(-max_tokens // page_size)
        pages = requests * self.columns
        shape = (layers, pages, kv_heads, page_size, head_dim)
        self.K = torch.empty(shape, dtype=dtype, device=device)
        self.V = torch.empty(shape, dtype=dtype, device=device)
        self.table = torch.full((requests, self.columns), -1, dtype=torch.int32, device=device)
        self.stack, self.top = torch.randperm(pages, device=device).to(torch.int32), 0  # free pages: stack[top:]
        self.ran_out = False  # some columns may have no page: only the device knows how many come back
        self.lengths = [0] * requests  # the scheduler's copy: only accepted drafts are read back from the device
        self.pending = None  # the step of trees that was mapped last, until its rows are kept or the requests' lengths change otherwise

    @property
    def free(self):
        return self.stack[self.top:]

    @free.setter
    def free(self, pages):
        # on a stack with room for those that the requests hold
        held = sum(self._pages(n) for n in self.lengths)
        self.top = max(self.stack.numel() - pages.numel(), held)
        self.stack = torch.cat([pages.new_full((self.top,), -1), pages])

    def _pages(self, tokens):
        return -(-tokens // self.page_size)

    def _ints(self, rows):
        dev, x = self.table.device, torch.tensor(rows, dtype=torch.int32)
        # from pinned memory, so that the copy does not wait for the work before it
        return (x.pin_memory() if dev.type == "cuda" else x).to(dev, non_blocking=True)

    def extend(self, new):
        """Map a step that brings new[r] tokens for request r; returns its PageMap."""
        if len(new) != len(self.lengths) or any(n < 0 for n in new):
            raise ValueError("a step brings a number of tokens for each of %d requests, got %s" % (len(self.lengths), new))
        for c, n in zip(self.lengths, new):
            if c + n > self.columns * self.page_size:
                raise ValueError("%d tokens do not fit %d pages of %d" % (c + n, self.columns, self.page_size))
        ctx, fresh = self._ints([self.lengths, new])
        m = page_map(ctx, fresh, self.free, self.table, self.page_size, sum(new))
        taken, left = sum(self._pages(c + n) - self._pages(c) for c, n in zip(self.lengths, new)), self.stack.numel() - self.top
        self.top += min(taken, left)
        self.ran_out |= taken > left
        self.lengths = [c + n for c, n in zip(self.lengths, new)]
        self.pending = None
        return m

    def draft(self, trees):
        """Map a step whose request r brings the tree trees[r] (its nodes' parents, the root first; [] for none)."""
        nodes = [len(t) for t in trees]
        if max(nodes, default=0) > 64 * _lib.NQ_TREE_WORDS:  # before the step takes pages
            raise ValueError("a tree has %d nodes; there may be %d at most" % (max(nodes), 64 * _lib.NQ_TREE_WORDS))
        parents = self._ints([p for t in trees for p in t])
        m = self.extend(nodes)
        self.pending = DraftStep(m, draft_tree(parents, m.q_start, m.kv_lens, max(nodes, default=0)), parents, nodes)
        return self.pending

    def _check_pending(self, step):
        """A step's pages and lengths are those of the cache until the next change."""
        if step is not self.pending:
            raise ValueError("the step is not the one that was drafted last, or its rows have been kept already")

    def keep(self, step, verdict):
        """Keep the step's accepted rows alone: they move to the front of their request's, and pages past them are free again.
        Returns how many each request keeps (read back, so this waits for the step).  Only the step that was drafted last can be
        kept, once, and before requests are extended or end."""
        self._check_pending(step)
        if verdict.accepted.numel() != len(step.nodes) or verdict.path.numel() != sum(step.nodes):
            raise ValueError("the verdict is of %d requests and %d nodes; the step has %d and %d" % (
                verdict.accepted.numel(), verdict.path.numel(), len(step.nodes), sum(step.nodes)))
        m = step.map
        paged_compact(self.K, self.V, self.table, m.q_start, m.kv_lens, verdict.path)
        kept = verdict.accepted.tolist()
        self._release(m.kv_lens, [n - d + a for n, d, a in zip(self.lengths, step.nodes, kept)])
        return kept

    def end(self, requests):
        """Give back all pages of requests that have ended."""
        gone = set(requests)
        if not gone <= set(range(len(self.lengths))):
            raise ValueError("there are %d requests, numbered from 0; got %s" % (len(self.lengths), sorted(gone)))
        self._release(self._ints(self.lengths), [0 if r in gone else n for r, n in enumerate(self.lengths)])

    def _release(self, lens, keep):
        # a step has room for all its tokens, so no length covers a column that was not written: the table need not be cleared
        counts = page_release(self.table, lens, self._ints(keep), self.page_size, self.stack, self.top)
        if self.ran_out:
            released, no_room = counts.tolist()
            self.top -= released - no_room
        else:
            self.top -= sum(self._pages(n) - self._pages(k) for n, k in zip(self.lengths, keep))
        self.lengths = keep
        self.pending = None

    def fill(self, K, V):
        """Put a prompt's cache [layers, requests, kv_heads, tokens, head_dim] into the pages, as the codec leaves it."""
        layers, requests, _, tokens, _ = K.shape
        m = self.extend([tokens] * requests)
        for layer in range(layers):
            for r in range(requests):
                paged_append(K[layer, r].transpose(0, 1), V[layer, r].transpose(0, 1), self.K[layer], self.V[layer],
                             m.slots[r * tokens:(r + 1) * tokens])

    def step(self, q, k, v, new, ws=None):
        """Append and attend: q [layers, tokens, q_heads, head_dim], k and v [layers, tokens, kv_heads, head_dim]."""
        return self._attend(self.extend(new), q, k, v, max(new), ws)

    def draft_step(self, q, k, v, step, ws=None):
        """Append a mapped step's trees and let them attend; shapes as in step().  The step must be the one that was drafted last."""
        self._check_pending(step)
        return self._attend(step.map, q, k, v, max(step.nodes), ws, step.tree)

    def _attend(self, m, q, k, v, max_q, ws, tree=None):
        out = torch.empty_like(q)
        for layer in range(q.shape[0]):
            paged_append(k[layer], v[layer], self.K[layer], self.V[layer], m.slots)
            paged_attention(q[layer], self.K[layer], self.V[layer], self.table, m.q_start, m.kv_lens, max_q=max_q,
                            out=out[layer], ws=ws, tree=tree)
        return out


def random_tree(nodes, rng):
    """Parents of a tree whose levels widen by two to four, as drafts of the likeliest continuations do."""
    return [-1] + [max(0, i // rng.choice([2, 3, 4])) for i in range(1, nodes)]


def random_verdict(step, vocab, generator, device):
    """The step's trees against random probabilities of a model and of a draft near it, from which the drafts are drawn."""
    rows = step.parents.numel()
    x = torch.randn((rows, vocab), generator=generator, device=device) * 3
    probs = torch.softmax(x, 1)
    draft = torch.softmax(x + 0.5 * torch.randn((rows, vocab), generator=generator, device=device), 1)
    first = torch.repeat_interleave(step.map.q_start[:-1].long(), step.map.q_start.diff().long(), output_size=rows)
    source = first + step.parents.clamp(min=0)
    tokens = torch.multinomial(draft[source], 1, generator=generator).squeeze(1).to(torch.int32)
    uniform = torch.rand(rows, generator=generator, device=device)
    return verify_drafts(probs, tokens, step.parents, step.map.q_start, uniform, draft_probs=draft)


def serve(cfg, steps=4, new=1, q_heads=None, page_size=16, layers=None, tokens=None, mode=0, seed=0, device="cuda", tree=0,
          vocab=32000):
    """Run `steps` steps of `new` tokens per request, or of a tree of `tree` drafted ones; returns the report as a dict."""
    device = torch.device(device, torch.cuda.current_device()) if device == "cuda" else torch.device(device)
    K, V = make_cache(cfg, device=device, layers=layers, tokens=tokens)
    L, B, H, T, D = K.shape
    heads = 4 * H if q_heads is None else q_heads
    params = cfg.modes[mode]
    rope = RopeTable.build(T, D, params.rope_theta, device=device)
    buf = compress_kv(K, V, params, rope)
    K2, V2 = decompress_kv(buf, (L, B, H, T, D), params, rope)
    new = tree or new
    caches = [PagedCache(L, B, H, D, page_size, T + steps * new, K.dtype, device) for _ in range(2)]
    caches[0].fill(K, V)
    caches[1].fill(K2, V2)
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def draw(h):
        return torch.randn((L, B * new, h, D), generator=g, device=device).to(K.dtype)

    rng = random.Random(seed)
    ws = None
    accepted = 0
    diff = norm = 0.0
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ms = []
    for _ in range(steps):
        q, k, v = draw(heads), draw(H), draw(H)
        if ws is None:
            ws = paged_attention_workspace(q[0], caches[0].K[0], caches[0].table, max_q=new)
        if tree:
            trees = [random_tree(tree, rng) for _ in range(B)]
            step = caches[0].draft(trees)
            exact = caches[0].draft_step(q, k, v, step, ws)
            verdict = random_verdict(step, vocab, g, device)
            accepted += sum(caches[0].keep(step, verdict))
            events[0].record()
            step = caches[1].draft(trees)
            coded = caches[1].draft_step(q, k, v, step, ws)
            caches[1].keep(step, verdict)
        else:
            exact = caches[0].step(q, k, v, [new] * B, ws)
            events[0].record()
            coded = caches[1].step(q, k, v, [new] * B, ws)
        events[1].record()
        events[1].synchronize()
        ms.append(events[0].elapsed_time(events[1]))
        diff += float((coded.double() - exact.double()).square().sum())
        norm += float(exact.double().square().sum())
    paged_status(device)  # the report is void when a kernel gave up a wait
    report = {"config": cfg.name, "layers": L, "requests": B, "cached_tokens": T, "new_tokens": new, "steps": steps,
            "q_heads": heads, "kv_heads": H, "head_dim": D, "page_size": page_size,
            "bits": [params.key_bits, params.value_bits], "compressed_share": buf.numel() / (2 * 2 * K.numel()),
            "attention_rel_error": (diff / norm) ** 0.5, "ms_per_step": sorted(ms)[len(ms) // 2]}
    if tree:
        report.update(tree=tree, vocab=vocab, accepted_per_step=accepted / (steps * B))
    return report


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--config", default="tiny", choices=sorted(CONFIGS))
    ap.add_argument("--mode", type=int, default=0, help="which of the config's codec modes")
    ap.add_argument("--layers", type=int, default=None)
    ap.add_argument("--tokens", type=int, default=None)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--new", type=int, default=1, help="tokens that every request brings per step")
    ap.add_argument("--tree", type=int, default=0, help="drafted tokens in each request's tree (0: no drafts)")
    ap.add_argument("--vocab", type=int, default=32000, help="tokens of the random probabilities that verify drafts")
    ap.add_argument("--q-heads", type=int, default=None, help="query heads (default: four per KV head)")
    ap.add_argument("--page-size", type=int, default=16)
    a = ap.parse_args(argv)
    print(json.dumps(serve(CONFIGS[a.config], a.steps, a.new, a.q_heads, a.page_size, a.layers, a.tokens, a.mode, tree=a.tree,
                           vocab=a.vocab)))


if __name__ == "__main__":
    main()
