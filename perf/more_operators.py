"""Cases of the operators that serve trees of drafted tokens from the paged cache: the tree's map, the attention of its
tokens over the pages, the verification of the drafts against the model's probabilities, and what follows from that: the
accepted rows move to the front of the request's drafted rows in every layer, and pages past them go back to the free list.

Every case is one such call of a serving step.  A request's tree has its root first (the token that is certain already) and every
node after its parent.  Sizes are those of this repository's cache shapes (8 or 32 KV heads, head_dim 64, 96 or 128, 16 to 48
layers) and generic ones.  Lengths and trees come from the case alone, so that `work` can count them; values, page orders, accepted
paths and random numbers come from the seed.
"""
import random

import torch

own = False

F16, BF16, F32 = "float16", "bfloat16", "float32"


# ------------------------------------------------------------------ cases


def _tree(name, requests, nodes, ctx, shape="wide", window=0, lens=1):
    c = {"op": "tree", "requests": requests, "nodes": nodes, "ctx": ctx, "shape": shape, "window": window, "lens": lens}
    return dict(c, name=name) if name else c


def _attn(name, requests, nodes, ctx, heads, kv_heads, dim, page, dtype=F16, window=0, spread="ragged", shape="wide", nhd=False,
          lens=1):
    c = {"op": "attention", "requests": requests, "nodes": nodes, "ctx": ctx, "heads": heads, "kv_heads": kv_heads, "dim": dim,
         "page": page, "dtype": dtype, "window": window, "spread": spread, "shape": shape, "nhd": nhd, "lens": lens}
    return dict(c, name=name) if name else c


def _verify(name, requests, nodes, vocab, dtype=F32, sampled=True, shape="wide", spread="ragged", lens=1):
    c = {"op": "verify", "requests": requests, "nodes": nodes, "vocab": vocab, "dtype": dtype, "sampled": sampled, "shape": shape,
         "spread": spread, "lens": lens}
    return dict(c, name=name) if name else c


def _compact(name, layers, requests, nodes, ctx, kv_heads, dim, page, dtype=F16, spread="ragged", nhd=False, lens=1):
    c = {"op": "compact", "layers": layers, "requests": requests, "nodes": nodes, "ctx": ctx, "kv_heads": kv_heads, "dim": dim,
         "page": page, "dtype": dtype, "spread": spread, "nhd": nhd, "lens": lens}
    return dict(c, name=name) if name else c


def _release(name, requests, ctx, gone, page, spread="ragged", lens=1):
    c = {"op": "release", "requests": requests, "ctx": ctx, "gone": gone, "page": page, "spread": spread, "lens": lens}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's step: a root and seven drafts
        _tree("tree 1x8", 1, 8, 1500),
        # a large batch with wide trees
        _tree("tree 256x64", 256, 64, 8192),
        # one user, a short context: latency only
        _attn("tree attention 1x8 over 1.5k", 1, 8, 1500, 32, 8, 128, 16, spread="even"),
        # a batch whose trees fill 64 rows for each KV head
        _attn("tree attention 32x16 over 16k", 32, 16, 16000, 32, 8, 128, 16, dtype=BF16),
        # every head with its own keys, head_dim 96, a sliding window, pages in token-major order
        _attn("tree attention 16x12 window dim 96", 16, 12, 6000, 32, 32, 96, 64, window=4096, nhd=True),
        # trees as large as pay, head_dim 64: 256 rows for each KV head
        _attn("tree attention 16x64 over 32k", 16, 64, 32000, 32, 8, 64, 32, dtype=BF16),
        # one user, a chain of five drafts whose draft model decodes greedily
        _verify("verify 1x6 chain", 1, 6, 32000, dtype=BF16, sampled=False, shape="chain", spread="even"),
        # a batch of trees that were sampled from a draft model's probabilities
        _verify("verify 64x16 sampled", 64, 16, 128256),
        # one user's accepted rows in all layers
        _compact("compact 1x16, 32 layers", 32, 1, 16, 1500, 8, 128, 16, spread="even"),
        # a batch's accepted rows in all layers
        _compact("compact 64x16, 48 layers", 48, 64, 16, 1000, 8, 128, 16, dtype=BF16),
        # after a step of 64 requests: the pages that rejected drafts had begun
        _release("release 64 steps", 64, 8192, 16, 16, spread="tail"),
        # requests that have ended give back whole prompts
        _release("release 512 prompts", 512, 8192, 8192, 16),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["tree", "attention", "attention", "attention", "verify", "verify", "compact", "release"])
    lens, page = rng.randrange(1 << 20), rng.choice([16, 32, 64, 128])
    shape, spread = rng.choice(["wide", "wide", "chain", "random"]), rng.choice(["ragged", "ragged", "even"])
    if kind == "tree":
        nodes = _log(rng, 1, 200)
        requests = _log(rng, 1, max(1, min(1024, 16384 // (nodes * _ceil(nodes, 64)))))
        return _tree(None, requests, nodes, _log(rng, 16, 32768), shape, rng.choice([0, 0, 2, 4096]), lens)
    if kind == "verify":
        vocab = rng.choice([32000, 32064, 50257, 65536, 100277, 128256, _log(rng, 300, 200000)])
        nodes = _log(rng, 1, 64)
        requests = _log(rng, 1, max(1, min(256, (1 << 23) // vocab, (1 << 27) // (nodes * vocab))))
        return _verify(None, requests, nodes, vocab, rng.choice([F32, F32, F16, BF16]), rng.random() < 0.6, shape, spread, lens)
    kv_heads, dim = rng.choice([1, 2, 4, 8, 8, 32]), rng.choice([64, 96, 128, 128])
    dtype, nhd = rng.choice([F16, BF16]), rng.random() < 0.3
    if kind == "compact":
        layers, nodes = rng.choice([1, 16, 32, 48]), _log(rng, 2, 64)
        requests = _log(rng, 1, min(64, 512 // kv_heads))
        ctx = _log(rng, 16, max(17, min(8192, (1 << 25) // (layers * requests * kv_heads))))
        return _compact(None, layers, requests, nodes, ctx, kv_heads, dim, page, dtype, spread, nhd, lens)
    if kind == "release":
        requests, ctx = _log(rng, 1, 512), _log(rng, 16, 8192)
        return _release(None, requests, ctx, _log(rng, 1, ctx), page, rng.choice(["ragged", "tail", "even"]), lens)
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8] if kv_heads < 32 else [1])
    nodes, requests = _log(rng, 2, 100), _log(rng, 1, 64)
    nodes = max(2, min(nodes, 1024 // requests))
    ctx = _log(rng, 16, max(17, min(131072, (1 << 21) // (requests * kv_heads), (1 << 28) // (requests * nodes * heads))))
    return _attn(None, requests, nodes, ctx, heads, kv_heads, dim, page, dtype, _log(rng, 16, 8192) if rng.random() < 0.25 else 0,
                 spread, shape, nhd, lens)


# ------------------------------------------------------- lengths and trees


def _lengths(case):
    """(ctx, nodes) per request: "even" gives every request the case's numbers; "ragged" spreads contexts down to an eighth and trees
    to a half, and leaves some requests out of the step."""
    rng = random.Random(case["lens"])
    ctx, new = [], []
    for r in range(case["requests"]):
        c, n = case.get("ctx", 0), case["nodes"]
        if case.get("spread", "ragged") != "even" and r > 0:
            c = rng.randint(c // 8, c) if c else 0
            n = rng.randint((n + 1) // 2, n)
            if r % 16 == 15:
                n = 0
        ctx.append(c)
        new.append(n)
    return ctx, new


def _parents(shape, n, rng):
    """Parents of a tree's nodes: "chain" is one draft after another, "wide" gives each level's first nodes the most children, as
    drafts of the most likely continuations do, "random" any earlier node."""
    parents = [-1]
    for i in range(1, n):
        if shape == "chain":
            parents.append(i - 1)
        elif shape == "random":
            parents.append(rng.randrange(i))
        else:
            parents.append(max(0, min(i - 1, int(i / rng.choice([1.5, 2, 3, 4])))))
    return parents[:n]


def _trees(case):
    rng = random.Random(case["lens"] + 1)
    return [_parents(case["shape"], n, rng) for n in _lengths(case)[1]]


def _ceil(a, b):
    return -(-a // b)


def _seen(parents, window):
    """Per node: its depth, and the nodes on its way to the root that a window leaves, itself first."""
    got = []
    for i in range(len(parents)):
        way = [i]
        while parents[way[-1]] >= 0:
            way.append(parents[way[-1]])
        got.append((len(way) - 1, way[:window] if window else way))
    return got


def _keep(case):
    """release: (length, length to keep) per request.  "tail" ends some tokens after the last kept page, as a step's drafts do."""
    rng = random.Random(case["lens"])
    lens, keep = [], []
    for r in range(case["requests"]):
        c, g = case["ctx"], case["gone"]
        if case["spread"] != "even" and r > 0:
            c = rng.randint(c // 8, c)
            g = rng.randint(0, min(g, c)) if case["spread"] == "tail" or r % 4 == 3 else min(g, c)
        lens.append(c)
        keep.append(c - min(g, c))
    return lens, keep


def work(case):
    if case["op"] == "release":
        lens, keep = _keep(case)
        pages = sum(_ceil(a, case["page"]) - _ceil(b, case["page"]) for a, b in zip(lens, keep))
        return {"bytes": 8 * case["requests"] + 8 * pages + 8, "flops": pages}
    ctx, new = _lengths(case)
    tokens, R = sum(new), case["requests"]
    if case["op"] == "tree":
        return {"bytes": 8 * R + tokens * (8 + 8 * _ceil(case["nodes"], 64)), "flops": tokens}
    if case["op"] == "verify":
        # the row of the last accepted node, and of the draft's there (nearly every walk ends at a rejected node)
        size = {F32: 4, F16: 2, BF16: 2}[case["dtype"]]
        rows = sum(1 for n in new if n) * (2 if case["sampled"] else 1)
        return {"bytes": rows * case["vocab"] * size + tokens * (20 + 2 * size) + 4 * R, "flops": rows * case["vocab"] * 2}
    row = case["kv_heads"] * case["dim"] * 2
    if case["op"] == "compact":
        moved = sum(len([k for k, j in enumerate(p) if j != k]) for p in _paths(case, 0))
        return {"bytes": 4 * moved * case["layers"] * row + 4 * tokens + 8 * R, "flops": 0}
    pairs = rows = 0
    w = case["window"]
    for c, n, parents in zip(ctx, new, _trees(case)):
        if n == 0:
            continue
        rows += n + (min(c, w - 1) if w else c)
        for depth, way in _seen(parents, w):
            pairs += len(way) + (max(min(c, w - 1 - depth), 0) if w else c)
    q = tokens * case["heads"] * case["dim"] * 2
    return {"bytes": 2 * q + 4 * tokens * case["heads"] + 12 * tokens + 2 * rows * row,
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ----------------------------------------------------------------- inputs


def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _starts(new, dev):
    return _i32([0] + new, dev).cumsum(0).to(torch.int32)


def _tables(need, page_count, columns, g, dev):
    """A block table with `need[r]` pages of a random order in row r, -1 behind them; the order (page 0 stays out of use)."""
    order = torch.randperm(page_count - 1, generator=g, device=dev).to(torch.int32) + 1
    count = torch.tensor(need, device=dev)
    col = torch.arange(columns, device=dev)
    at = (torch.cumsum(count, 0) - count)[:, None] + col[None, :]
    table = torch.where(col[None, :] < count[:, None], order[at.clamp(max=page_count - 2)], torch.full_like(order[:1], -1))
    return table.contiguous(), order


def _pool(case, pages, g, dev, layers=None):
    """A pool [pages, kv_heads, page, dim], with `layers` one of them for each; `nhd`: the same seen through token-major storage."""
    shape = (pages, case["page"], case["kv_heads"], case["dim"]) if case["nhd"] else (
        pages, case["kv_heads"], case["page"], case["dim"])
    shape = shape if layers is None else (layers,) + shape
    x = torch.empty(shape, dtype=getattr(torch, case["dtype"]), device=dev).normal_(generator=g)
    return x.transpose(-3, -2) if case["nhd"] else x


def _paths(case, seed):
    """compact: the accepted nodes of each request, the root first.  A row that moves comes from behind all kept ones, so that a
    second pass over the same rows changes nothing."""
    rng, sizes = random.Random(seed * 31 + 5), random.Random(case["lens"] + 2)
    paths = []
    for n in _lengths(case)[1]:
        if n == 0:
            paths.append([])
            continue
        kept = sizes.randint(1, max(1, min(n // 2, 6)))
        stay = sizes.randint(1, kept)
        paths.append(list(range(stay)) + sorted(rng.sample(range(kept, n), kept - stay)))
    return paths


def _words(trees, case, ctx, dev):
    """(ancestors, positions) of a step's trees."""
    words = _ceil(case["nodes"], 64)
    bits, pos = [], []
    for c, parents in zip(ctx, trees):
        for depth, way in _seen(parents, case["window"]):
            x = sum(1 << j for j in way)
            row = [(x >> (64 * k)) & (2 ** 64 - 1) for k in range(words)]
            bits.append([v - 2 ** 64 if v >= 2 ** 63 else v for v in row])
            pos.append(c + depth)
    return torch.tensor(bits, dtype=torch.int64, device=dev).view(-1, words), _i32(pos, dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7 + 3)
    state = {"case": case}
    if case["op"] == "release":
        lens, keep = _keep(case)
        held = [_ceil(n, case["page"]) for n in lens]
        pages = sum(held) + 9
        state["table"], order = _tables(held, pages, max(held) + 2, g, dev)
        # the free list fills the end of its buffer; what is given back goes on top of it, towards the front
        state["top"] = sum(held) + 1
        state["free"] = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        state["free"][state["top"]:] = order[sum(held):][: pages - state["top"]]
        state["lens"], state["keep"] = _i32(lens, dev), _i32(keep, dev)
        state["counts"] = torch.empty(2, dtype=torch.int32, device=dev)
        return state
    ctx, new = _lengths(case)
    R, tokens = case["requests"], sum(new)
    state["max_q"] = case["nodes"]
    state["q_start"] = _starts(new, dev)
    state["kv_lens"] = _i32([c + n for c, n in zip(ctx, new)], dev)
    if case["op"] == "tree":
        # other trees for other seeds, of the same shape
        rng = random.Random(int(seed))
        state["parents"] = _i32([p for n in new for p in _parents(case["shape"], n, rng)], dev)
        state["tree"] = (torch.empty((tokens, _ceil(case["nodes"], 64)), dtype=torch.int64, device=dev),
                         torch.empty(tokens, dtype=torch.int32, device=dev))
        return state
    if case["op"] == "verify":
        return _prepare_verify(case, state, new, g, dev)
    P = case["page"]
    full = [_ceil(c + n, P) for c, n in zip(ctx, new)]
    pages = sum(full) + 9
    state["table"], _ = _tables(full, pages, max(full) + 3, g, dev)
    if case["op"] == "compact":
        state["K_pages"] = _pool(case, pages, g, dev, case["layers"])
        state["V_pages"] = _pool(case, pages, g, dev, case["layers"])
        state["path"] = _i32([j for n, p in zip(new, _paths(case, int(seed))) for j in p + [-1] * (n - len(p))], dev)
        return state
    # attention: the tree's own keys are in the pages already; scores as peaked as a model's
    state["K_pages"], state["V_pages"] = _pool(case, pages, g, dev), _pool(case, pages, g, dev)
    state["Q"] = torch.empty((tokens, case["heads"], case["dim"]), dtype=getattr(torch, case["dtype"]), device=dev)
    state["Q"].normal_(generator=g).mul_(1.5)
    state["ancestors"], state["positions"] = _words(_trees(case), case, ctx, dev)
    state["out"] = torch.empty_like(state["Q"])
    state["lse"] = torch.empty((tokens, case["heads"]), dtype=torch.float32, device=dev)
    return state


def _prepare_verify(case, state, new, g, dev):
    """A model's probabilities (a few likely tokens over a long tail), a draft's that are near them, and drafts that come from those:
    sampled, or the most likely tokens in turn."""
    V, tokens, R, dtype = case["vocab"], sum(new), case["requests"], getattr(torch, case["dtype"])
    trees = _trees(case)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    source, rank = [], []  # of each node: its parent's row, and which of the parent's children it is
    for r, parents in enumerate(trees):
        for i, p in enumerate(parents):
            source.append(start[r] + max(p, 0))
            rank.append(sum(1 for x in parents[:i] if x == p))
    probs = torch.empty((tokens, V), dtype=dtype, device=dev)
    draft = torch.empty((tokens, V), dtype=dtype, device=dev)
    for a in range(0, tokens, 256):
        b = min(a + 256, tokens)
        x = torch.randn((b - a, V), generator=g, device=dev) * 2.5
        at = torch.randint(0, V, (b - a, 4), generator=g, device=dev)
        x.scatter_(1, at, torch.tensor([18.0, 17.0, 16.0, 15.0], device=dev).expand(b - a, 4).contiguous())
        y = x + 0.7 * torch.randn((b - a, V), generator=g, device=dev)
        for z, to in ((x, probs), (y, draft)):
            z = torch.exp(z - z.amax(1, keepdim=True))
            to[a:b] = (z / z.sum(1, keepdim=True)).to(dtype)
    ids = torch.zeros(tokens, dtype=torch.int32, device=dev)
    src, nth = torch.tensor(source, device=dev), torch.tensor(rank, device=dev)
    for a in range(0, tokens, 256):
        q = draft[src[a:a + 256]].float()
        if case["sampled"]:
            noise = torch.empty_like(q).exponential_(generator=g)
            ids[a:a + 256] = (q / noise).argmax(1).to(torch.int32)
        else:
            top = q.topk(min(64, V), dim=1).indices
            ids[a:a + 256] = top.gather(1, nth[a:a + 256, None].clamp(max=min(64, V) - 1)).squeeze(1).to(torch.int32)
    state.update(probs=probs, draft=draft if case["sampled"] else None, tokens=ids,
                 parents=_i32([p for t in trees for p in t], dev), uniform=torch.rand(tokens, generator=g, device=dev),
                 verdict=tuple(torch.empty(n, dtype=torch.int32, device=dev) for n in (R, tokens, tokens)))
    return state


# -------------------------------------------------------------- the passes


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"tree": _plain_tree, "attention": _plain_attention, "verify": _plain_verify, "compact": _plain_compact,
            "release": _plain_release}[case["op"]](state, case)


def _run_own(state, case):
    import e8_lattice_vector_gb300 as nq

    if case["op"] == "tree":
        t = nq.draft_tree(state["parents"], state["q_start"], state["kv_lens"], state["max_q"], window=case["window"],
                          out=nq.DraftTree(*state["tree"]))
        return {"ancestors": t.ancestors, "positions": t.positions}
    if case["op"] == "verify":
        v = nq.verify_drafts(state["probs"], state["tokens"], state["parents"], state["q_start"], state["uniform"],
                             draft_probs=state["draft"], out=nq.Verdict(*state["verdict"]))
        return {"accepted": v.accepted, "path": v.path, "tokens": v.tokens}
    if case["op"] == "compact":
        K, V = nq.paged_compact(state["K_pages"], state["V_pages"], state["table"], state["q_start"], state["kv_lens"],
                                state["path"])
        return {"K": K, "V": V}
    if case["op"] == "release":
        counts = nq.page_release(state["table"], state["lens"], state["keep"], case["page"], state["free"], state["top"],
                                 out=state["counts"])
        return {"free": state["free"], "counts": counts}
    O, lse = nq.paged_attention(state["Q"], state["K_pages"], state["V_pages"], state["table"], state["q_start"],
                                state["kv_lens"], max_q=state["max_q"], window=case["window"],
                                tree=nq.DraftTree(state["ancestors"], state["positions"]), out=state["out"], lse=state["lse"])
    return {"out": O, "lse": lse}


def _rows(q_start, n):
    """[requests, n]: the row of each request's i-th token, and whether it has one."""
    i = torch.arange(n, device=q_start.device)
    row = q_start[:-1, None].long() + i[None, :]
    return row, row < q_start[1:, None]


def _plain_tree(state, case):
    """Every node walks up at once, a level a time."""
    n, T = state["max_q"], state["parents"].numel()
    row, live = _rows(state["q_start"], n)
    at = row.clamp(max=max(T - 1, 0))
    parent = torch.where(live, state["parents"][at], -1).long()
    here = torch.arange(n, device=at.device).expand_as(parent)
    seen = torch.zeros(parent.shape + (n,), dtype=torch.bool, device=at.device)
    depth = torch.full_like(parent, -1)
    for level in range(n):
        up = here >= 0
        depth += up
        if case["window"] == 0 or level < case["window"]:
            seen |= up[:, :, None] & (torch.arange(n, device=at.device) == here[:, :, None])
        here = torch.where(up, parent.gather(1, here.clamp(min=0)), -1)
    words = state["tree"][0].shape[1]
    bit = torch.arange(n, device=at.device)
    word = torch.stack([torch.where(seen & (bit // 64 == k), torch.ones_like(bit) << (bit % 64), 0).sum(-1) for k in range(words)], -1)
    ctx = state["kv_lens"] - (state["q_start"][1:] - state["q_start"][:-1])
    ancestors, positions = state["tree"]
    ancestors[at[live]] = word[live]
    positions[at[live]] = (ctx[:, None] + depth)[live].to(torch.int32)
    return {"ancestors": ancestors, "positions": positions}


def _plain_attention(state, case):
    """Requests padded to the longest tree and the longest cache; 32-bit products, exponentials and sums."""
    Q, table, q_start, kv_lens, n = state["Q"], state["table"], state["q_start"], state["kv_lens"], state["max_q"]
    T, Hq, D = Q.shape
    R, H, P = kv_lens.numel(), case["kv_heads"], case["page"]
    L = (table.shape[1] - 3) * P  # the longest request's pages
    page = table[:, : L // P].clamp(min=0).reshape(-1)
    K = state["K_pages"][page].view(R, L // P, H, P, D).transpose(1, 2).reshape(R, H, L, D).float()
    V = state["V_pages"][page].view(R, L // P, H, P, D).transpose(1, 2).reshape(R, H, L, D).float()
    row, live = _rows(q_start, n)
    row = row.clamp(max=T - 1)
    ctx = (kv_lens - (q_start[1:] - q_start[:-1])).long()
    q = Q[row].float().view(R, n, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(R, H, (Hq // H) * n, D)
    j = torch.arange(L, device=Q.device)
    context = (j[None, None, :] < ctx[:, None, None]).expand(R, n, L)
    if case["window"]:
        context = context & (j[None, None, :] > state["positions"][row][:, :, None] - case["window"])
    node = j[None, :] - ctx[:, None]  # [R, L]
    words = state["ancestors"][row]  # [R, n, words]
    drafted = torch.zeros((R, n, L), dtype=torch.bool, device=Q.device)
    for k in range(words.shape[2]):
        here = (node >= 64 * k) & (node < 64 * (k + 1))
        bit = (words[:, :, k, None] >> (node.clamp(min=0) % 64)[:, None, :]) & 1
        drafted |= here[:, None, :] & (bit == 1)
    seen = context | (drafted & (j[None, None, :] < kv_lens[:, None, None]))
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


def _plain_verify(state, case):
    """All requests a node at a time; sums and comparisons in 64 bits, where they decide between two whole numbers."""
    probs, draft, q_start, n = state["probs"], state["draft"], state["q_start"], state["max_q"]
    T, V = probs.shape
    accepted, path, tokens = state["verdict"]
    R, dev = accepted.numel(), probs.device
    row, live = _rows(q_start, n)
    row = row.clamp(max=T - 1)
    ids, parent, u = state["tokens"][row].long(), state["parents"][row].long(), state["uniform"][row].double()
    req = torch.arange(R, device=dev)
    cur = torch.zeros(R, dtype=torch.long, device=dev)
    p = probs[row[:, 0]].double()  # what is left of the current node's probabilities
    total = torch.ones(R, dtype=torch.float64, device=dev)
    kept = torch.zeros((R, n), dtype=torch.bool, device=dev)
    kept[:, 0] = live[:, 0]
    for i in range(1, n):
        x = ids[:, i:i + 1]
        w = p.gather(1, x).squeeze(1)
        asked = live[:, i] & (parent[:, i] == cur)
        if draft is None:
            yes = asked & (u[:, i] * total < w)
            no = asked & ~yes
            total = torch.where(no, total - w, total)
            p.scatter_(1, x, torch.where(no, 0.0, w)[:, None])
        else:
            q = draft[row[req, cur]].double()
            yes = asked & (u[:, i] * (total * q.gather(1, x).squeeze(1)) < w)
            no = asked & ~yes
            p = torch.where(no[:, None], (p - total[:, None] * q).clamp(min=0), p)
            total = torch.where(no, p.sum(1), total)
        cur = torch.where(yes, i, cur)
        kept[:, i] = yes
        p = torch.where(yes[:, None], probs[row[:, i]].double(), p)
        total = torch.where(yes, 1.0, total)
    p = torch.where(p.sum(1, keepdim=True) > 0, p, probs[row[req, cur]].double())
    sums = p.cumsum(1)
    last = torch.searchsorted(sums, (u[:, :1] * sums[:, -1:]).contiguous(), right=True).squeeze(1)
    top = torch.where(p > 0, torch.arange(V, device=dev), -1).amax(1)
    last = torch.minimum(last, top)
    count = kept.sum(1)
    accepted.copy_(count.to(torch.int32))
    # kept nodes in order, then -1; their tokens without the root's, then the new one
    i = torch.arange(n, device=dev)
    order = torch.where(kept, i, n + i).argsort(1)
    nodes = torch.where(i < count[:, None], order, -1)
    after = torch.cat([nodes[:, 1:], torch.full_like(nodes[:, :1], -1)], 1)
    said = torch.where(after >= 0, ids.gather(1, after.clamp(min=0)), -1)
    said = torch.where(i == count[:, None] - 1, last[:, None], said)
    path[row[live]] = nodes[live].to(torch.int32)
    tokens[row[live]] = said[live].to(torch.int32)
    return {"accepted": accepted, "path": path, "tokens": tokens}


def _plain_compact(state, case):
    P, q_start, n, T = case["page"], state["q_start"], state["max_q"], state["path"].numel()
    row, live = _rows(q_start, n)
    path = torch.where(live, state["path"][row.clamp(max=T - 1)], -1).long()
    ctx = (state["kv_lens"] - (q_start[1:] - q_start[:-1])).long()
    k = torch.arange(n, device=path.device)
    r, k = torch.nonzero((path >= 0) & (path != k), as_tuple=True)
    src, dst = ctx[r] + path[r, k], ctx[r] + k
    src_page, dst_page = state["table"][r, src // P].long(), state["table"][r, dst // P].long()
    for pool in (state["K_pages"], state["V_pages"]):
        # index [:, page, :, at] puts the indexed axis first: [moves, layers, kv_heads, dim]
        pool[:, dst_page, :, dst % P] = pool[:, src_page, :, src % P]
    return {"K": state["K_pages"], "V": state["V_pages"]}


def _plain_release(state, case):
    P, table, free, top = case["page"], state["table"], state["free"], state["top"]
    lens = state["lens"].clamp(min=0, max=table.shape[1] * P)
    a = (torch.minimum(state["keep"].clamp(min=0), lens) + P - 1) // P
    b = (lens + P - 1) // P
    col = torch.arange(table.shape[1], device=table.device)
    gone = table[(col >= a[:, None]) & (col < b[:, None])]
    at = top - 1 - torch.arange(gone.numel(), device=table.device)
    free[at[at >= 0]] = gone[at >= 0]
    n = (b - a).sum()
    state["counts"].copy_(torch.stack([n, (n - top).clamp(min=0)]).to(torch.int32))
    return {"free": free, "counts": state["counts"]}


# --------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    if case["op"] not in ("attention", "compact"):
        return None  # whole numbers: compared as they are
    ctx, new = _lengths(case)
    P, D = case["page"], case["dim"]
    if case["op"] == "compact":
        state = prepare(case, seed)
        got = {}
        paths = _paths(case, int(seed))
        for name in ("K", "V"):
            pool = state[name + "_pages"].double()
            for r, (c, kept) in enumerate(zip(ctx, paths)):
                pages = state["table"][r].tolist()
                for k, j in enumerate(kept):  # one row after the other
                    pool[:, pages[(c + k) // P], :, (c + k) % P] = pool[:, pages[(c + j) // P], :, (c + j) % P]
            got[name] = pool
        return got
    Hq, H, w = case["heads"], case["kv_heads"], case["window"]
    if 4 * D * Hq * sum(n * (c + n) for c, n in zip(ctx, new)) > 8e12:
        return None
    state = prepare(case, seed)
    out = torch.zeros((sum(new), Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), Hq), float("-inf"), dtype=torch.float64, device="cuda")
    at = 0
    for r, (c, n, parents) in enumerate(zip(ctx, new, _trees(case))):
        if n == 0:
            continue
        length = c + n
        pages = state["table"][r, : _ceil(length, P)].long()
        see = torch.zeros((n, length), dtype=torch.bool)
        for i, (depth, way) in enumerate(_seen(parents, w)):
            see[i, max(0, c + depth - w + 1) if w else 0: c] = True
            see[i, [c + a for a in way]] = True
        hide = ~see.cuda()
        for h in range(H):
            heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
            k = state["K_pages"][pages, h].reshape(-1, D)[:length].double()
            v = state["V_pages"][pages, h].reshape(-1, D)[:length].double()
            s = torch.einsum("tgd,jd->tgj", state["Q"][at:at + n, heads].double(), k) / D ** 0.5
            s = s.masked_fill(hide[:, None], float("-inf"))
            lse[at:at + n, heads] = torch.logsumexp(s, -1)
            out[at:at + n, heads] = torch.einsum("tgj,jd->tgd", torch.softmax(s, -1), v)
        at += n
    return {"out": out, "lse": lse}
