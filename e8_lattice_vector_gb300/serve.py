"""Serving from a compressed cache: what the paged operators do together with the codec.

    python -m e8_lattice_vector_gb300.serve --config tiny --steps 4 --new 1

A prompt's cache is compressed and decompressed, put into pages, and then served from: every step maps the new tokens
of each request to slots, appends their keys and values and lets them attend over everything cached, layer by
layer.  The same steps also run over the cache as it was before compression; the relative difference of the two attention
outputs says what the code's loss costs where it is used.  The synthetic caches of synth.py stand in for a
model's, and random queries, keys and values for its new tokens.
"""
import argparse
import json

import torch

from .codec import RopeTable, compress_kv, decompress_kv
from .paged import page_map, paged_append, paged_attention, paged_attention_workspace, paged_status
from .synth import CONFIGS, make_cache


class PagedCache:
    """One layer stack's pools, block table and free list for a fixed set of requests."""

    def __init__(self, layers, requests, kv_heads, head_dim, page_size, max_tokens, dtype, device):
        self.page_size, self.columns = page_size, -(-max_tokens // page_size)
        pages = requests * self.columns
        shape = (layers, pages, kv_heads, page_size, head_dim)
        self.K = torch.empty(shape, dtype=dtype, device=device)
        self.V = torch.empty(shape, dtype=dtype, device=device)
        self.table = torch.full((requests, self.columns), -1, dtype=torch.int32, device=device)
        self.free = torch.randperm(pages, device=device).to(torch.int32)
        self.lengths = [0] * requests  # the scheduler's copy: nothing is read back from the device

    def extend(self, new):
        """Map a step that brings new[r] tokens for request r; returns its PageMap."""
        if len(new) != len(self.lengths) or any(n < 0 for n in new):
            raise ValueError("a step brings a number of tokens for each of %d requests, got %s" % (len(self.lengths), new))
        for c, n in zip(self.lengths, new):
            if c + n > self.columns * self.page_size:
                raise ValueError("%d tokens do not fit %d pages of %d" % (c + n, self.columns, self.page_size))
        dev, lens = self.table.device, torch.tensor([self.lengths, new], dtype=torch.int32)
        # from pinned memory, so that the copy does not wait for the work before it
        ctx, fresh = (lens.pin_memory() if dev.type == "cuda" else lens).to(dev, non_blocking=True)
        m = page_map(ctx, fresh, self.free, self.table, self.page_size, sum(new))
        taken = sum(-(-(c + n) // self.page_size) - -(-c // self.page_size) for c, n in zip(self.lengths, new))
        self.free = self.free[taken:]
        self.lengths = [c + n for c, n in zip(self.lengths, new)]
        return m

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
        m = self.extend(new)
        out = torch.empty_like(q)
        for layer in range(q.shape[0]):
            paged_append(k[layer], v[layer], self.K[layer], self.V[layer], m.slots)
            paged_attention(q[layer], self.K[layer], self.V[layer], self.table, m.q_start, m.kv_lens, max_q=max(new),
                            out=out[layer], ws=ws)
        return out


def serve(cfg, steps=4, new=1, q_heads=None, page_size=16, layers=None, tokens=None, mode=0, seed=0, device="cuda"):
    """Run `steps` steps of `new` tokens per request; returns the report as a dict."""
    device = torch.device(device, torch.cuda.current_device()) if device == "cuda" else torch.device(device)
    K, V = make_cache(cfg, device=device, layers=layers, tokens=tokens)
    L, B, H, T, D = K.shape
    heads = 4 * H if q_heads is None else q_heads
    params = cfg.modes[mode]
    rope = RopeTable.build(T, D, params.rope_theta, device=device)
    buf = compress_kv(K, V, params, rope)
    K2, V2 = decompress_kv(buf, (L, B, H, T, D), params, rope)
    caches = [PagedCache(L, B, H, D, page_size, T + steps * new, K.dtype, device) for _ in range(2)]
    caches[0].fill(K, V)
    caches[1].fill(K2, V2)
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def draw(h):
        return torch.randn((L, B * new, h, D), generator=g, device=device).to(K.dtype)

    ws = None
    diff = norm = 0.0
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ms = []
    for _ in range(steps):
        q, k, v = draw(heads), draw(H), draw(H)
        if ws is None:
            ws = paged_attention_workspace(q[0], caches[0].K[0], caches[0].table, max_q=new)
        exact = caches[0].step(q, k, v, [new] * B, ws)
        events[0].record()
        coded = caches[1].step(q, k, v, [new] * B, ws)
        events[1].record()
        events[1].synchronize()
        ms.append(events[0].elapsed_time(events[1]))
        diff += float((coded.double() - exact.double()).square().sum())
        norm += float(exact.double().square().sum())
    paged_status(device)  # the report is void when a kernel gave up a wait
    return {"config": cfg.name, "layers": L, "requests": B, "cached_tokens": T, "new_tokens": new, "steps": steps,
            "q_heads": heads, "kv_heads": H, "head_dim": D, "page_size": page_size,
            "bits": [params.key_bits, params.value_bits], "compressed_share": buf.numel() / (2 * 2 * K.numel()),
            "attention_rel_error": (diff / norm) ** 0.5, "ms_per_step": sorted(ms)[len(ms) // 2]}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--config", default="tiny", choices=sorted(CONFIGS))
    ap.add_argument("--mode", type=int, default=0, help="which of the config's codec modes")
    ap.add_argument("--layers", type=int, default=None)
    ap.add_argument("--tokens", type=int, default=None)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--new", type=int, default=1, help="tokens that every request brings per step")
    ap.add_argument("--q-heads", type=int, default=None, help="query heads (default: four per KV head)")
    ap.add_argument("--page-size", type=int, default=16)
    a = ap.parse_args(argv)
    print(json.dumps(serve(CONFIGS[a.config], a.steps, a.new, a.q_heads, a.page_size, a.layers, a.tokens, a.mode)))


if __name__ == "__main__":
    main()
