"""Cases of the paged-cache operators: the page map of a serving step, the append of a step's keys and values
through it, and the attention of the step's tokens over the paged cache.

Every case is one such call with the sizes of this repository's cache shapes (8 or 32 KV heads, head_dim 64, 96
or 128, 512 to 131072 tokens) and the pages of a serving engine (16 to 128 tokens).  `prepare` makes what the
engine holds before the call: the pools, the block table, the lengths on the device and, as host numbers, the
bound on a request's new tokens that the engine's scheduler knows.  Lengths come from the case alone, so that
`work` can count them; values, page orders and free lists come from the seed.
"""
import random

import torch

own = False

F16, BF16 = "float16", "bfloat16"


# ------------------------------------------------------------------ cases


def _attn(name, requests, new, ctx, heads, kv_heads, dim, page, dtype=F16, window=0, spread="ragged", causal=True,
          nhd=False, lens=1):
    c = {"op": "attention", "requests": requests, "new": new, "ctx": ctx, "heads": heads, "kv_heads": kv_heads,
         "dim": dim, "page": page, "dtype": dtype, "window": window, "spread": spread, "causal": causal, "nhd": nhd,
         "lens": lens}
    return dict(c, name=name) if name else c


def _append(name, requests, new, ctx, kv_heads, dim, page, dtype=F16, spread="ragged", head_major=False, nhd=False,
            lens=1):
    c = {"op": "append", "requests": requests, "new": new, "ctx": ctx, "kv_heads": kv_heads, "dim": dim, "page": page,
         "dtype": dtype, "spread": spread, "head_major": head_major, "nhd": nhd, "lens": lens}
    return dict(c, name=name) if name else c


def _map(name, requests, new, ctx, page, pad=0, spread="ragged", lens=1):
    c = {"op": "map", "requests": requests, "new": new, "ctx": ctx, "page": page, "pad": pad, "spread": spread,
         "lens": lens}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step of 64 requests: one token each, padded to a graph's 96 rows
        _map("map decode 64", 64, 1, 8192, 16, pad=32),
        # prompts of up to 32768 tokens for 16 requests, nothing cached yet
        _map("map prompts 16x32k", 16, 32768, 0, 16),
        # the K and V of a decode step, written into 16-token pages
        _append("append decode 64", 64, 1, 8192, 8, 128, 16),
        # a decompressed 131072-token cache (head-major, as the codec leaves it) going into pages
        _append("append cache 131k", 1, 131072, 0, 8, 128, 64, spread="even", head_major=True),
        # one user, a short context: latency only
        _attn("decode 1x1.5k", 1, 1, 1500, 32, 8, 128, 16, spread="even"),
        # one user, the longest context: the cache split over the whole GPU (five query heads per KV head)
        _attn("decode 1x131k", 1, 1, 131071, 40, 8, 128, 64, spread="even", dtype=BF16),
        # a decode batch of ragged lengths
        _attn("decode 64x32k", 64, 1, 32767, 32, 8, 128, 16),
        # verification of a drafted run of 5 tokens with a sliding window, head_dim 64
        _attn("verify 32x5 window", 32, 5, 16000, 32, 8, 64, 32, dtype=BF16, window=4096),
        # a chunk of a long prompt among requests that decode
        _attn("chunk 512 + 31 decodes", 32, 512, 8000, 32, 8, 128, 16, spread="mixed", dtype=BF16),
        # one chunk of a long prompt over what is cached of it
        _attn("chunk 2000 over 30k", 1, 2000, 30000, 32, 8, 128, 64, spread="even"),
        # whole prompts, every head with its own keys, head_dim 96, pages in token-major order
        _attn("prompts 8x2k dim 96", 8, 2048, 0, 32, 32, 96, 16, nhd=True),
        # whole prompts with grouped heads
        _attn("prompts 2x8k", 2, 8192, 0, 32, 8, 128, 128, dtype=BF16),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["map", "append", "decode", "decode", "chunk", "chunk", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1 << 20)
    dtype = rng.choice([F16, BF16])
    nhd = rng.random() < 0.3
    spread = rng.choice(["ragged", "ragged", "mixed", "even"])
    if kind == "map":
        requests = _log(rng, 1, 2048)
        new = _log(rng, 1, max(1, min(32768, 300000 // requests)))
        return _map(None, requests, new, _log(rng, 16, 32768), page, rng.choice([0, 0, rng.randrange(1, 200)]), spread,
                    lens)
    kv_heads = rng.choice([1, 2, 4, 8, 8, 32])
    dim = rng.choice([64, 96, 128, 128])
    if kind == "append":
        requests = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, (1 << 20) // (requests * kv_heads)))
        return _append(None, requests, new, _log(rng, 16, 8192), kv_heads, dim, page, dtype, spread,
                       rng.random() < 0.3, nhd, lens)
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8] if kv_heads < 32 else [1])
    window = _log(rng, 16, 8192) if rng.random() < 0.25 else 0
    if kind == "decode":
        requests = _log(rng, 1, 128)
        new = rng.choice([1, 1, 1, 2, 3, 4, 6])
        ctx = _log(rng, 16, max(17, min(131072, (1 << 23) // (requests * kv_heads))))
    elif kind == "chunk":
        requests = _log(rng, 1, 16)
        new = _log(rng, 7, max(8, min(2048, 65536 // heads) // requests))
        ctx = _log(rng, 16, max(17, min(30000, (1 << 22) // (requests * kv_heads))))
    else:
        requests = _log(rng, 1, 8)
        new = _log(rng, 64, max(65, min(8192, int(((1 << 31) // (requests * heads)) ** 0.5))))
        ctx = 0
    return _attn(None, requests, new, ctx, heads, kv_heads, dim, page, dtype, window, spread,
                 rng.random() < 0.85, nhd, lens)


# ---------------------------------------------------------------- lengths


def _lengths(case):
    """(ctx, new) per request: "even" gives every request the case's numbers; "ragged" spreads them down to an
    eighth and leaves some requests out of the step; "mixed" gives the first request the whole chunk and the
    others one token."""
    rng = random.Random(case["lens"])
    ctx, new = [], []
    for r in range(case["requests"]):
        c, n = case["ctx"], case["new"]
        if case["spread"] != "even" and r > 0:
            c = rng.randint(c // 8, c) if c else 0
            n = 1 if case["spread"] == "mixed" else rng.randint((n + 7) // 8, n)
            if case["spread"] == "ragged" and r % 16 == 15:
                n = 0
        ctx.append(c)
        new.append(n)
    return ctx, new


def _ceil(a, b):
    return -(-a // b)


def _columns(case, ctx, new):
    """The block table's width: what the longest request needs, and a few columns to spare."""
    return _ceil(max(c + n for c, n in zip(ctx, new)), case["page"]) + 3


def _pairs(case):
    """(query, key) pairs that the mask leaves, and the cached rows that some query sees, summed over requests."""
    pairs = rows = 0
    w = case["window"]
    for c, n in zip(*_lengths(case)):
        if n == 0:
            continue
        lo = max(0, c - w + 1) if w else 0
        rows += c + n - lo
        for i in range(n):
            p = c + i
            hi = p + 1 if case["causal"] else c + n
            pairs += hi - (max(0, p - w + 1) if w else 0)
    return pairs, rows


def work(case):
    ctx, new = _lengths(case)
    tokens, R, P = sum(new), case["requests"], case["page"]
    if case["op"] == "map":
        need = sum(_ceil(c + n, P) - _ceil(c, P) for c, n in zip(ctx, new))
        return {"bytes": 16 * R + 8 * need + 12 * (tokens + case["pad"]) + 20, "flops": tokens}
    row = case["kv_heads"] * case["dim"] * 2
    if case["op"] == "append":
        return {"bytes": 4 * tokens * row + 8 * tokens, "flops": 0}
    pairs, rows = _pairs(case)
    q = tokens * case["heads"] * case["dim"] * 2
    return {"bytes": 2 * q + 4 * tokens * case["heads"] + 2 * rows * row, "flops": 4 * pairs * case["heads"] * case["dim"]}


# ----------------------------------------------------------------- inputs


def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _pool(case, pages, g, dev):
    """A pool [pages, kv_heads, page, dim]; `nhd`: the same seen through token-major storage."""
    shape = (pages, case["page"], case["kv_heads"], case["dim"]) if case["nhd"] else (
        pages, case["kv_heads"], case["page"], case["dim"])
    x = torch.empty(shape, dtype=getattr(torch, case["dtype"]), device=dev).normal_(generator=g)
    return x.transpose(1, 2) if case["nhd"] else x


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7 + 3)
    ctx, new = _lengths(case)
    R, P, M, tokens = case["requests"], case["page"], _columns(case, ctx, new), sum(new)
    held = [_ceil(c, P) for c in ctx]
    full = [_ceil(c + n, P) for c, n in zip(ctx, new)]
    pages = sum(full) + 9  # page 0 stays out of use, and a few are free
    order = torch.randperm(pages - 1, generator=g, device=dev).to(torch.int32) + 1
    # columns in use before the step (map) or after it (append, attention); -1 elsewhere
    have = held if case["op"] == "map" else full
    count = torch.tensor(have, device=dev)
    col = torch.arange(M, device=dev)
    used = col[None, :] < count[:, None]
    at = (torch.cumsum(count, 0) - count)[:, None] + col[None, :]
    table = torch.where(used, order[at.clamp(max=pages - 2)], torch.full_like(order[:1], -1)).contiguous()
    state = {"case": case, "table": table, "seed": seed}
    if case["op"] == "map":
        state.update(ctx=_i32(ctx, dev), new=_i32(new, dev), free=order[sum(held):].contiguous(),
                     tokens=tokens + case["pad"])
        # the step's buffers, which an engine keeps
        state["map"] = (torch.empty(R + 1, dtype=torch.int32, device=dev), torch.empty(R, dtype=torch.int32, device=dev),
                        torch.empty(state["tokens"], dtype=torch.int64, device=dev),
                        torch.empty(state["tokens"], dtype=torch.int32, device=dev),
                        torch.empty(4, dtype=torch.int32, device=dev))
        return state
    dtype = getattr(torch, case["dtype"])
    state["K_pages"], state["V_pages"] = _pool(case, pages, g, dev), _pool(case, pages, g, dev)
    if case["op"] == "append":
        shape = (case["kv_heads"], tokens, case["dim"]) if case["head_major"] else (tokens, case["kv_heads"], case["dim"])
        K = torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)
        V = torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)
        state["K"], state["V"] = (K.transpose(0, 1), V.transpose(0, 1)) if case["head_major"] else (K, V)
        req = torch.repeat_interleave(torch.arange(R, device=dev), torch.tensor(new, device=dev))
        start = torch.cumsum(torch.tensor([0] + new, device=dev), 0)
        pos = torch.arange(tokens, device=dev) - start[req] + torch.tensor(ctx, device=dev)[req]
        state["slots"] = table[req, pos // P].long() * P + pos % P
        return state
    # attention: the step's own keys are in the pages already; scores as peaked as a model's
    state["Q"] = torch.empty((tokens, case["heads"], case["dim"]), dtype=dtype, device=dev).normal_(generator=g) * 1.5
    state["q_start"] = _i32([0] + new, dev).cumsum(0).to(torch.int32)
    state["kv_lens"] = _i32([c + n for c, n in zip(ctx, new)], dev)
    state["max_q"] = max(new)
    state["out"] = torch.empty_like(state["Q"])
    state["lse"] = torch.empty((tokens, case["heads"]), dtype=torch.float32, device=dev)
    return state


# -------------------------------------------------------------- the passes


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"map": _plain_map, "append": _plain_append, "attention": _plain_attention}[case["op"]](state, case)


def _run_own(state, case):
    import e8_lattice_vector_gb300 as nq

    if case["op"] == "map":
        m = nq.page_map(state["ctx"], state["new"], state["free"], state["table"], case["page"], state["tokens"],
                        out=nq.PageMap(*state["map"]))
        return {"q_start": m.q_start, "kv_lens": m.kv_lens, "slots": m.slots, "positions": m.positions,
                "counts": m.counts, "table": state["table"]}
    if case["op"] == "append":
        K, V = nq.paged_append(state["K"], state["V"], state["K_pages"], state["V_pages"], state["slots"])
        return {"K": K, "V": V}
    O, lse = nq.paged_attention(state["Q"], state["K_pages"], state["V_pages"], state["table"], state["q_start"],
                                state["kv_lens"], max_q=state["max_q"], causal=case["causal"], window=case["window"],
                                out=state["out"], lse=state["lse"])
    return {"out": O, "lse": lse}


def _plain_map(state, case):
    ctx, new, table, free, T = state["ctx"], state["new"], state["table"], state["free"], state["tokens"]
    P, R, M, F = case["page"], ctx.numel(), table.shape[1], free.numel()
    start = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    total = ctx + new
    a = ((ctx + P - 1) // P).clamp(max=M)
    b = ((total + P - 1) // P).clamp(max=M)
    need = b - a
    base = torch.cumsum(need, 0) - need
    col = torch.arange(M, device=table.device)
    fresh = (col[None, :] >= a[:, None]) & (col[None, :] < b[:, None])
    at = base[:, None] + col[None, :] - a[:, None]
    page = torch.where(at < F, free[at.clamp(0, F - 1)], -1)
    table.copy_(torch.where(fresh, page, table))
    row = torch.arange(T, device=table.device)
    req = torch.searchsorted(start[1:].contiguous(), row, right=True)
    live = req < R
    req = req.clamp(max=R - 1)
    pos = row - start[req] + ctx[req]
    column = pos // P
    page = table[req, column.clamp(0, M - 1)].long()
    slot = torch.where(live & (column < M) & (page >= 0), page * P + pos % P, -1)
    pos = torch.where(live, pos, -1).to(torch.int32)
    asked = need.sum()
    past = (total > M * P).sum()
    counts = torch.stack([start[R], asked, (asked - F).clamp(min=0), past]).to(torch.int32)
    return {"q_start": start.to(torch.int32), "kv_lens": total, "slots": slot, "positions": pos, "counts": counts,
            "table": table}


def _plain_append(state, case):
    P, slots = case["page"], state["slots"]
    page, at = slots // P, slots % P
    # index [page, :, at] puts the indexed axis first: [tokens, kv_heads, dim]
    state["K_pages"][page, :, at] = state["K"]
    state["V_pages"][page, :, at] = state["V"]
    return {"K": state["K_pages"], "V": state["V_pages"]}


def _plain_attention(state, case):
    """Requests padded to the longest chunk and the longest cache; 32-bit products, exponentials and sums."""
    Q, table, q_start, kv_lens, n = state["Q"], state["table"], state["q_start"], state["kv_lens"], state["max_q"]
    T, Hq, D = Q.shape
    R, H, P = kv_lens.numel(), case["kv_heads"], case["page"]
    L = (table.shape[1] - 3) * P  # the longest request's pages
    page = table[:, : L // P].clamp(min=0).reshape(-1)
    K = state["K_pages"][page].view(R, L // P, H, P, D).transpose(1, 2).reshape(R, H, L, D).float()
    V = state["V_pages"][page].view(R, L // P, H, P, D).transpose(1, 2).reshape(R, H, L, D).float()
    q_len = q_start[1:] - q_start[:-1]
    i = torch.arange(n, device=Q.device)
    j = torch.arange(L, device=Q.device)
    row = (q_start[:-1, None] + i[None, :]).clamp(max=T - 1).long()
    q = Q[row].float().view(R, n, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(R, H, (Hq // H) * n, D)
    pos = (kv_lens - q_len)[:, None] + i[None, :]
    seen = (j[None, None, :] < kv_lens[:, None, None]).expand(R, n, L)
    if case["causal"]:
        seen = seen & (j[None, None, :] <= pos[:, :, None])
    if case["window"]:
        seen = seen & (j[None, None, :] > pos[:, :, None] - case["window"])
    s = torch.matmul(q, K.transpose(2, 3)) * (D ** -0.5)
    s = s.view(R, H, Hq // H, n, L).masked_fill_(~seen[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, H, (Hq // H) * n, L), V).view(R, H, Hq // H, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).squeeze(-1)
    out, out_lse = state["out"], state["lse"]
    # one row of the padded result for each row of Q
    req = torch.searchsorted(q_start[1:].contiguous(), torch.arange(T, device=Q.device, dtype=torch.int32), right=True)
    at = torch.arange(T, device=Q.device) - q_start[req].long()
    out.copy_(o.permute(0, 3, 1, 2, 4).reshape(R, n, Hq, D)[req, at])
    out_lse.copy_(lse.permute(0, 3, 1, 2).reshape(R, n, Hq)[req, at])
    return {"out": out, "lse": out_lse}


# --------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "map":
        return None  # whole numbers: compared as they are
    P = case["page"]
    if case["op"] == "append":
        got = {}
        for name in ("K", "V"):
            # pages flattened to slot-major rows, one assignment per slot
            pool = state[name + "_pages"].double().transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])
            pool.index_copy_(0, state["slots"], state[name].double())
            got[name] = pool.view(-1, P, case["kv_heads"], case["dim"]).transpose(1, 2)
        return got
    ctx, new = _lengths(case)
    Hq, H, D = case["heads"], case["kv_heads"], case["dim"]
    if 4 * D * Hq * sum(n * (c + n) for c, n in zip(ctx, new)) > 8e12:
        return None
    out = torch.zeros((sum(new), Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), Hq), float("-inf"), dtype=torch.float64, device="cuda")
    at = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        length = c + n
        pages = state["table"][r, : _ceil(length, P)].long()
        j = torch.arange(length, device="cuda")
        for h in range(H):
            k = state["K_pages"][pages, h].reshape(-1, D)[:length].double()
            v = state["V_pages"][pages, h].reshape(-1, D)[:length].double()
            for part in range(0, n, 512):
                stop = min(part + 512, n)
                q = state["Q"][at + part: at + stop, h * (Hq // H): (h + 1) * (Hq // H)].double()
                s = torch.einsum("tgd,jd->tgj", q, k) / D ** 0.5
                p = torch.arange(c + part, c + stop, device="cuda")[:, None]
                hide = torch.zeros((stop - part, length), dtype=torch.bool, device="cuda")
                if case["causal"]:
                    hide |= j[None] > p
                if case["window"]:
                    hide |= j[None] <= p - case["window"]
                s = s.masked_fill(hide[:, None], float("-inf"))
                rows, heads = slice(at + part, at + stop), slice(h * (Hq // H), (h + 1) * (Hq // H))
                lse[rows, heads] = torch.logsumexp(s, -1)
                out[rows, heads] = torch.einsum("tgj,jd->tgd", torch.softmax(s, -1), v)
        at += n
    return {"out": out, "lse": lse}
