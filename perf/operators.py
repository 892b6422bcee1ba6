"""Workloads of the decoding operators: appending to the paged cache, attention
over it, choosing tokens and keeping an accepted path.

``run`` computes them either with elementary torch operations in 32 bits (the
plain forms, ``own = False``) or through the library's entry points.  ``exact``
computes the same results in 64 bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases

def _append(name, tokens, hq, hk, d, rot, cache, page, norm, interleaved=False):
    return {"name": name, "op": "append", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot": rot, "cache": cache,
            "page": page, "norm": norm, "interleaved": interleaved}


def _attend(name, seqs, nodes, kv, hq, hk, d, cache, page, tree, window=0):
    return {"name": name, "op": "attend", "seqs": seqs, "nodes": nodes, "kv": kv, "hq": hq, "hk": hk, "d": d,
            "cache": cache, "page": page, "tree": tree, "window": window}


def _sample(name, rows, vocab, dtype, filters):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "filters": filters}


def _move(name, seqs, layers, nodes, path, hk, d, cache, page):
    return {"name": name, "op": "move", "seqs": seqs, "layers": layers, "nodes": nodes, "path": path, "hk": hk,
            "d": d, "cache": cache, "page": page}


def listed():
    return [
        # one decode step of five users of a small model: launch latency
        _append("append_decode", 5, 9, 3, 64, 64, "bf16", 16, False),
        # a long prompt of a model that norms its heads, into an 8-bit cache
        _append("append_prompt", 4100, 32, 8, 128, 128, "e4m3", 64, True),
        # one user, a short chat, a small model: launch latency
        _attend("decode_one", 1, 1, 517, 9, 3, 64, "bf16", 16, False),
        # ordinary batched decode, lengths from half to all of 8000
        _attend("decode_batch", 48, 1, 8000, 32, 8, 128, "bf16", 64, False),
        # drafted trees of up to 60 nodes, large head groups
        _attend("tree_batch", 16, 60, 4000, 64, 8, 128, "bf16", 64, True),
        # smaller trees, wide heads, 8-bit cache, a sliding window
        _attend("tree_window", 24, 17, 5000, 16, 8, 256, "e4m3", 32, True, 1024),
        # a chunk of a prompt behind what is cached already
        _attend("prompt_chunk", 3, 777, 6000, 32, 8, 128, "bf16", 64, False),
        # one very long context, a chain of drafted tokens, 8-bit cache
        _attend("long_context", 1, 8, 131000, 64, 8, 128, "e4m3", 128, False),
        # one user's token from fp32 logits: launch latency
        _sample("sample_one", 1, 50001, "f32", True),
        # the nodes of a verified batch, bf16 logits as the products give them
        _sample("sample_batch", 200, 131072, "bf16", True),
        # one user's accepted path, all layers
        _move("move_one", 1, 24, 12, 4, 3, 64, "bf16", 16),
        # a batch's accepted paths, all layers
        _move("move_batch", 64, 32, 60, 7, 8, 128, "bf16", 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = [(9, 3, 64), (16, 8, 64), (32, 8, 128), (64, 8, 128), (28, 4, 128), (12, 12, 128), (8, 1, 128), (16, 8, 256), (8, 4, 256)]


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "sample", "move"])
    hq, hk, d = rng.choice(_HEADS)
    cache = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "append":
        return {k: v for k, v in _append("", _log(rng, 1, 4096), hq, hk, d, rng.choice([d, d // 2]), cache, page,
                                         rng.random() < 0.5, rng.random() < 0.4).items() if k != "name"}
    if op == "sample":
        rows, vocab = _log(rng, 1, 200), _log(rng, 1000, 262144)
        rows = max(1, min(rows, 26000000 // vocab))
        return {k: v for k, v in _sample("", rows, vocab, rng.choice(["bf16", "f32"]), rng.random() < 0.8).items() if k != "name"}
    if op == "move":
        nodes = _log(rng, 2, 64)
        return {k: v for k, v in _move("", _log(rng, 1, 64), rng.randint(1, 24), nodes, rng.randint(1, min(nodes, 8)), hk, d, cache, page).items() if k != "name"}
    kind = rng.choice(["one", "tree", "tree", "chain"])
    nodes = 1 if kind == "one" else _log(rng, 2, 128) if kind == "tree" else _log(rng, 2, 700)
    kv = max(nodes, _log(rng, 64, 65536))
    # no more cached tokens, and no more pairs of a row and a key, than the listed cases hold
    pairs = int(4e10 / (nodes * hq * d))
    kv = max(nodes, min(kv, pairs))
    seqs = max(1, min(_log(rng, 1, 64), int(2.5e8 / (kv * hk * d)), pairs // kv))
    window = rng.choice([0, 0, 0, 100, 1024])
    return {k: v for k, v in _attend("", seqs, nodes, kv, hq, hk, d, cache, page, kind == "tree", window).items() if k != "name"}


# ------------------------------------------------------------------ lengths

def _spread(most, least, n, step):
    """n lengths from `least` to `most`, the first of them `most`."""
    return [most - (i * step) % (most - least + 1) for i in range(n)]


def _nodes(c):
    return _spread(c["nodes"], max(1, 2 * c["nodes"] // 3), c["seqs"], 5)


def _lengths(c):
    nodes = _nodes(c)
    return [max(a, b) for a, b in zip(_spread(c["kv"], max(1, c["kv"] // 2), c["seqs"], 977), nodes)]


def work(c):
    e = 1 if c.get("cache") == "e4m3" else 2
    if c["op"] == "append":
        t, dh = c["tokens"], c["d"]
        return {"bytes": t * dh * (4 * c["hq"] + c["hk"] * (4 + 2 * e)) + 4 * t * c["rot"], "flops": 10 * t * dh * (c["hq"] + c["hk"])}
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * (2 if c["dtype"] == "bf16" else 4), "flops": 4 * n}
    if c["op"] == "move":
        # the first node of a path stays where it is
        moved = sum(max(0, p - 1) for p in _paths(c)) * c["layers"]
        return {"bytes": 4 * moved * c["hk"] * c["d"] * e, "flops": 0}
    keys = rows = pairs = 0
    for n, length in zip(_nodes(c), _lengths(c)):
        window = c["window"] or length
        keys += min(length, window + n - 1)
        rows += n
        # a node of a tree sees its few ancestors, one of a chain all before it
        pairs += sum(min(length - n + (min(4, i + 1) if c["tree"] else i + 1), window) for i in range(n))
    return {"bytes": 2 * keys * c["hk"] * c["d"] * e + 4 * rows * c["hq"] * c["d"], "flops": 4 * pairs * c["hq"] * c["d"]}


def _paths(c):
    return _spread(c["path"], max(1, c["path"] // 2), c["seqs"], 3)


# ------------------------------------------------------------------ prepare

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _cache(g, lead, hk, d, page, cache):
    """Random cache contents in the cache's layout (K, V), with scales for 8 bits."""
    c = 16 if cache == "e4m3" else 8
    shapes = (*lead, hk, page // 16, d // c, 16, c), (*lead, hk, page // 16, 16 // c, d, c)
    out = []
    for s in shapes:
        if cache == "e4m3":
            out.append((40 * _normal(g, *s)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            out.append(torch.empty(s, dtype=torch.bfloat16, device=DEV).normal_(generator=g))
    return out


def _scales(g, hk, cache):
    if cache != "e4m3":
        return None, None
    return tuple(0.02 + 0.01 * torch.rand(hk, generator=g, device=DEV) for _ in range(2))


def _int(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _pages_of(lengths, page, rng, pages=0):
    need = [-(-n // page) for n in lengths]
    pages = max(pages, sum(need) + 3)
    order = rng.permutation(pages)
    table = np.zeros((len(lengths), max(need)), np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pages, table


def _trees(nodes, rng):
    """Ancestor masks (bit j of row i: node i is j or below it) and depths of one tree for each sequence."""
    words = -(-max(nodes) // 64)
    masks, depths = [], []
    for n in nodes:
        mask, depth = [], []
        for i in range(n):
            p = int(rng.integers(max(0, i - 6), i)) if i else -1
            mask.append((mask[p] if i else 0) | 1 << i)
            depth.append(depth[p] + 1 if i else 0)
        masks += [[(m >> 64 * w) & (1 << 64) - 1 for w in range(words)] for m in mask]
        depths.append(np.array(depth))
    return np.array(masks, dtype=np.uint64).view(np.int64).reshape(-1, words), depths


def prepare(case, seed):
    c, g, rng = case, _gen(seed), np.random.default_rng(int(seed))
    s = {"c": c}
    if c["op"] == "sample":
        x = 2.5 * _normal(g, c["rows"], c["vocab"])
        # a few likely tokens over a long tail
        x.scatter_add_(1, torch.randint(c["vocab"], (c["rows"], 12), generator=g, device=DEV), 4 + 4 * torch.rand(c["rows"], 12, generator=g, device=DEV))
        s["logits"] = x.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        s["u"] = torch.rand(c["rows"], generator=g, device=DEV)
        s["temperature"] = torch.tensor(rng.choice([0.0, 0.6, 0.8, 1.0, 1.3], c["rows"], p=[0.1, 0.2, 0.2, 0.3, 0.2]), dtype=torch.float32, device=DEV)
        s["top_k"] = s["top_p"] = s["min_p"] = None
        if c["filters"]:
            s["top_k"] = _int(rng.choice([0, 20, 50, 400], c["rows"]))
            s["top_p"] = torch.tensor(rng.choice([1.0, 0.95, 0.9, 0.5], c["rows"]), dtype=torch.float32, device=DEV)
            s["min_p"] = torch.tensor(rng.choice([0.0, 0.02, 0.1], c["rows"]), dtype=torch.float32, device=DEV)
        return s
    if c["op"] == "append":
        t, hq, hk, d = c["tokens"], c["hq"], c["hk"], c["d"]
        pages, table = _pages_of([t + 5], c["page"], rng)
        s["k_cache"], s["v_cache"] = _cache(g, (pages,), hk, d, c["page"], c["cache"])
        s["k_scale"], s["v_scale"] = _scales(g, hk, c["cache"])
        # the rows of one product: queries, keys and values side by side
        qkv = _normal(g, t, (hq + 2 * hk) * d).to(torch.bfloat16).view(t, hq + 2 * hk, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_norm"] = s["k_norm"] = None
        if c["norm"]:
            s["q_norm"], s["k_norm"] = (1 + 0.2 * _normal(g, d) for _ in range(2))
        at = np.arange(t) + int(rng.integers(0, 6))
        s["slots"] = _int(table[0][at // c["page"]] * c["page"] + at % c["page"])
        s["positions"] = _int(at)
        a = torch.arange(t + 8, device=DEV).float()[:, None] * (10000.0 ** (-torch.arange(c["rot"] // 2, device=DEV) / (c["rot"] / 2)))
        s["table"] = torch.cat([a.cos(), a.sin()], 1).contiguous()
        return s
    if c["op"] == "move":
        base = [int(x) for x in rng.integers(0, 3 * c["page"], c["seqs"])]
        pages, table = _pages_of([x + c["nodes"] for x in base], c["page"], rng,
                                 c["seqs"] * (5 + c["nodes"] // c["page"]) + 3)
        s["k_cache"], s["v_cache"] = _cache(g, (c["layers"], pages), c["hk"], c["d"], c["page"], c["cache"])
        path = np.zeros((c["seqs"], c["path"]), np.int32)
        for b, n in enumerate(_paths(c)):
            path[b, 1:n] = np.sort(rng.choice(np.arange(1, c["nodes"]), n - 1, replace=False))
        s["page_table"], s["base"], s["path"], s["count"] = _int(table), _int(base), _int(path), _int(_paths(c))
        return s
    nodes, lengths, d = _nodes(c), _lengths(c), c["d"]
    pages, table = _pages_of(lengths, c["page"], rng)
    s["k_cache"], s["v_cache"] = _cache(g, (pages,), c["hk"], d, c["page"], c["cache"])
    s["k_scale"], s["v_scale"] = _scales(g, c["hk"], c["cache"])
    total = sum(nodes)
    s["q"] = (1.5 * _normal(g, total, c["hq"], d)).to(torch.bfloat16)
    s["page_table"], s["kv_len"] = _int(table), _int(lengths)
    s["q_start"] = _int(np.concatenate([[0], np.cumsum(nodes)]))
    s["max_q"], s["max_kv"] = max(nodes), max(lengths)
    s["tree"] = None
    depths = [np.arange(n) for n in nodes]
    if c["tree"]:
        mask, depths = _trees(nodes, rng)
        s["tree"] = torch.from_numpy(mask).to(DEV)
    s["positions"] = _int(np.concatenate([length - n + dep for length, n, dep in zip(lengths, nodes, depths)]))
    return s


# -------------------------------------------------------------- plain forms

def _values(x):
    return x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x


def _head_rows(x, norm, table, positions, rot, interleaved):
    x = x.float()
    if norm is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * norm
    cs = table[positions.long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


def _plain_append(s):
    c = s["c"]
    args = s["table"], s["positions"], c["rot"], c["interleaved"]
    q = _head_rows(s["q"], s["q_norm"], *args).to(torch.bfloat16)
    k, v = _head_rows(s["k"], s["k_norm"], *args), s["v"].float()
    if s["k_scale"] is not None:
        k, v = k / s["k_scale"][:, None], v / s["v_scale"][:, None]
        k, v = (x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    t, hk, d = k.shape
    n = s["k_cache"].shape[-1]
    slot = s["slots"].long()
    page, block, at = slot // c["page"], slot % c["page"] // 16, slot % 16
    s["k_cache"][page, :, block, :, at] = k.view(t, hk, d // n, n)
    s["v_cache"][page, :, block, at // n, :, at % n] = v
    return q, _values(s["k_cache"]), _values(s["v_cache"])


def _plain_attend(s):
    c = s["c"]
    table, hk, d = s["page_table"].long(), c["hk"], c["d"]
    seqs = table.shape[0]
    k = _values(s["k_cache"][table].permute(0, 2, 1, 3, 5, 4, 6).reshape(seqs, hk, -1, d)).float()
    v = _values(s["v_cache"][table].permute(0, 2, 1, 3, 4, 6, 5).reshape(seqs, hk, -1, d)).float()
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    keys, most = k.shape[2], s["max_q"]
    start = s["q_start"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(most, device=DEV)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(seqs, most, hk, -1, d).transpose(1, 2).reshape(seqs, hk, -1, d)
    j = torch.arange(keys, device=DEV)
    length = s["kv_len"].long()[:, None, None]
    past = length - count[:, None, None]
    node = j - past
    if s["tree"] is not None:
        n = node.clamp(0, most - 1).expand(seqs, most, keys)
        drafted = (s["tree"][row].gather(2, n // 64) >> (n % 64)) & 1 != 0
    else:
        drafted = node <= i[:, None]
    seen = (node < 0) | drafted
    seen = seen & (j < length)
    if c["window"]:
        at = s["positions"].long()[row]
        key_at = torch.where(node < 0, j, at.gather(1, node[:, 0].clamp(0, most - 1))[:, None])
        seen = seen & (key_at > at[:, :, None] - c["window"])
    seen = seen[:, None, :, None].expand(seqs, 1, most, c["hq"] // hk, keys).reshape(seqs, 1, -1, keys)
    p = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    p = p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    o = o.view(seqs, hk, most, -1, d).transpose(1, 2).reshape(seqs, most, -1, d)
    return o[i < count[:, None]].to(torch.bfloat16)


def _of_2_24(x, most):
    return (x * 2.0 ** 24).floor().to(torch.int64).clamp(0, most)


def _part(m, total):
    """m * total / 2^24 in whole numbers, and whether anything is left over."""
    low = m * (total & (1 << 24) - 1)
    return m * (total >> 24) + (low >> 24), low & (1 << 24) - 1 != 0


def _plain_sample(s):
    x, t = s["logits"].float(), s["temperature"][:, None]
    x = torch.where(x.isnan(), -math.inf, x)
    greedy = t == 0
    top = x.amax(1, keepdim=True)
    diff = torch.where(x == top, 0.0, x - top)
    e = torch.where(x == -math.inf, 0.0, torch.exp(diff * (1.0 / torch.where(greedy, 1.0, t))))
    w = (e * 2.0 ** 31).round().to(torch.int64)
    order = x.sort(dim=1, descending=True, stable=True).indices
    w = w.gather(1, order)
    k = s["top_k"][:, None].long() if s["top_k"] is not None else torch.zeros_like(t, dtype=torch.int64)
    k = torch.where(greedy, 1, torch.where(k > 0, k, x.shape[1]))
    w = torch.where(torch.arange(x.shape[1], device=DEV) < k, w, 0)
    upto = w.cumsum(1)
    if s["top_p"] is not None:
        whole, more = _part(_of_2_24(s["top_p"][:, None], 1 << 24), upto[:, -1:])
        need = (whole + more).clamp(min=1)
        w = torch.where(upto - w < need, w, 0)
    if s["min_p"] is not None:
        w = torch.where(w >= (s["min_p"][:, None] * 2.0 ** 31).ceil().to(torch.int64), w, 0)
    w = torch.zeros_like(w).scatter_(1, order, w)
    upto = w.cumsum(1)
    total = upto[:, -1:]
    target = _part(_of_2_24(s["u"][:, None], (1 << 24) - 1), total)[0]
    token = (upto <= target).sum(1, keepdim=True)
    prob = w.gather(1, token.clamp(max=x.shape[1] - 1)).float() / total.clamp(min=1).float()
    # a row without any weight gives no token
    return torch.where(total == 0, -1, token)[:, 0].to(torch.int32), prob[:, 0]


def _plain_move(s):
    c = s["c"]
    n = s["k_cache"].shape[-1]
    path, base = s["path"].long(), s["base"].long()[:, None]
    j = torch.arange(path.shape[1], device=DEV).expand_as(path)
    live = j < s["count"][:, None]

    def place(token):
        token = (base + token)
        page = s["page_table"].long().gather(1, token // c["page"])[live]
        token = token[live]
        return page, token % c["page"] // 16, token % 16

    (p0, b0, a0), (p1, b1, a1) = place(path), place(j)
    s["k_cache"][:, p1, :, b1, :, a1] = s["k_cache"][:, p0, :, b0, :, a0]
    s["v_cache"][:, p1, :, b1, a1 // n, :, a1 % n] = s["v_cache"][:, p0, :, b0, a0 // n, :, a0 % n]
    return _values(s["k_cache"]), _values(s["v_cache"])


def run(state):
    s, c = state, state["c"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "sample": _plain_sample, "move": _plain_move}[c["op"]](s)
    import w4_dequant_gemm_amd as w4
    if c["op"] == "append":
        q = w4.w4_kv_append(s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], rope=s["table"],
                            positions=s["positions"], interleaved=c["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                            eps=1e-6, k_scale=s["k_scale"], v_scale=s["v_scale"])
        return q, _values(s["k_cache"]), _values(s["v_cache"])
    if c["op"] == "attend":
        return w4.w4_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["q_start"],
                                    s["max_q"], s["max_kv"], tree=s["tree"], window=c["window"],
                                    positions=s["positions"] if c["window"] else None,
                                    k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "sample":
        return w4.w4_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                            min_p=s["min_p"])
    w4.w4_kv_move(s["k_cache"], s["v_cache"], s["page_table"], s["base"], s["path"], s["count"])
    return _values(s["k_cache"]), _values(s["v_cache"])


# -------------------------------------------------------------------- exact

def _exact_append(s):
    c = s["c"]
    rot, half = c["rot"], c["rot"] // 2
    first = torch.arange(half, device=DEV) * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)
    angle = s["table"].double()[s["positions"].long()].unsqueeze(1)

    def turned(x, norm):
        x = x.double()
        if norm is not None:
            x = x / (x.square().sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * norm.double()
        y = x.clone()
        y[..., first] = x[..., first] * angle[..., :half] - x[..., second] * angle[..., half:]
        y[..., second] = x[..., first] * angle[..., half:] + x[..., second] * angle[..., :half]
        return y

    k_cache, v_cache = (_values(s[n]).double() for n in ("k_cache", "v_cache"))
    k, v = turned(s["k"], s["k_norm"]), s["v"].double()
    if s["k_scale"] is not None:
        k = (k / s["k_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    n = k_cache.shape[-1]
    dims = torch.arange(c["d"], device=DEV)
    slots = s["slots"].long()
    for h in range(c["hk"]):
        at = slots[:, None]
        k_cache[at // c["page"], h, at % c["page"] // 16, dims // n, at % 16, dims % n] = k[:, h]
        v_cache[at // c["page"], h, at % c["page"] // 16, at % 16 // n, dims, at % n] = v[:, h]
    return turned(s["q"], s["q_norm"]), k_cache, v_cache


def _exact_attend(s):
    c = s["c"]
    d, hk, group = c["d"], c["hk"], c["hq"] // c["hk"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    start, length = s["q_start"].tolist(), s["kv_len"].tolist()
    tree = None if s["tree"] is None else s["tree"].cpu().numpy().view(np.uint64)
    for b in range(c["seqs"]):
        lo, hi, n = start[b], start[b + 1], length[b]
        rows, past = hi - lo, n - (hi - lo)
        seen = np.ones((rows, n), bool)
        if tree is None:
            seen[:, past:] = np.tril(np.ones((rows, rows), bool))
        else:
            for i in range(rows):
                bits = sum(int(w) << 64 * k for k, w in enumerate(tree[lo + i]))
                seen[i, past:] = [bits >> j & 1 for j in range(rows)]
        if c["window"]:
            at = s["positions"][lo:hi].cpu().numpy()
            seen &= np.concatenate([np.arange(past), at])[None] > at[:, None] - c["window"]
        seen = torch.from_numpy(seen).to(DEV)
        pages = s["page_table"][b, :-(-n // c["page"])].long()
        for h in range(hk):
            k = _values(s["k_cache"][pages, h].transpose(2, 3).reshape(-1, d)).double()[:n]
            v = _values(s["v_cache"][pages, h].transpose(3, 4).reshape(-1, d)).double()[:n]
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for r in range(group):
                score = s["q"][lo:hi, h * group + r].double() @ k.T / math.sqrt(d)
                score = torch.where(seen, score, torch.full_like(score, -math.inf))
                out[lo:hi, h * group + r] = torch.softmax(score, 1) @ v
    return out


def _exact_sample(s):
    tokens, probs = [], []
    for r in range(s["logits"].shape[0]):
        x = s["logits"][r].double()
        t = float(s["temperature"][r])
        order = torch.argsort(x, descending=True, stable=True)
        p = torch.softmax(x / t, 0)[order] if t else (torch.arange(x.numel(), device=DEV) == 0).double()
        if s["top_k"] is not None and int(s["top_k"][r]) > 0:
            p[int(s["top_k"][r]):] = 0
        keep = p > 0
        if s["top_p"] is not None:
            before = p.cumsum(0) - p
            keep &= before < float(s["top_p"][r]) * p.sum()
        if s["min_p"] is not None:
            keep &= p >= float(s["min_p"][r]) * p[0]
        kept = torch.zeros_like(p).scatter_(0, order, torch.where(keep, p, torch.zeros_like(p)))
        upto = kept.cumsum(0)
        token = int((upto <= float(s["u"][r]) * upto[-1]).sum())
        tokens.append(token)
        probs.append(float(kept[token] / kept.sum()))
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64)


def _exact_move(s):
    c = s["c"]
    out = []
    for name, axis in (("k_cache", 3), ("v_cache", 4)):
        x = _values(s[name]).double()
        n = x.shape[-1]
        for b, count in enumerate(s["count"].tolist()):
            base, pages = int(s["base"][b]), s["page_table"][b].tolist()

            def piece(token):
                block = x[:, pages[token // c["page"]], :, token % c["page"] // 16]
                at = token % 16
                return block[:, :, :, at] if axis == 3 else block[:, :, at // n, :, at % n]

            for j in range(count):
                piece(base + j).copy_(piece(base + int(s["path"][b, j])).clone())
        out.append(x)
    return tuple(out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample, "move": _exact_move}[case["op"]](s)
