"""Workloads of the calls around the products of a served model: the product
with bias, activation and residual in its epilogue, a mixture-of-experts layer
over 4-bit experts, and the changes made to logits before a token is chosen.

``run`` computes them either with elementary torch operations in 32 bits (the
plain forms, ``own = False``) or through the library's entry points.  ``exact``
computes the same results in 64 bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"


# ------------------------------------------------------------------- cases

def _linear(name, rows, n, k, group, kind, bias, act, residual):
    return {"name": name, "op": "linear", "rows": rows, "n": n, "k": k, "group": group, "kind": kind, "bias": bias,
            "act": act, "residual": residual}


def _moe(name, tokens, experts, top_k, hidden, inner, group, score, act, residual):
    return {"name": name, "op": "moe", "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden,
            "inner": inner, "group": group, "score": score, "act": act, "residual": residual}


def _adjust(name, rows, vocab, dtype, history, biases, mask):
    return {"name": name, "op": "adjust", "rows": rows, "vocab": vocab, "dtype": dtype, "history": history,
            "biases": biases, "mask": mask}


def listed():
    return [
        # one token through a small model's down projection, added to the stream: launch latency
        _linear("linear_one", 1, 576, 1536, 32, "a16", False, "none", True),
        # a few users' tokens through an 8B model's down projection, added to the stream
        _linear("linear_decode", 5, 4096, 14336, 128, "a16", False, "none", True),
        # a chunk of 77 tokens, 8-bit activations, an MLP without a gate: bias and GELU
        _linear("linear_chunk", 77, 15360, 3840, 128, "a8", True, "gelu_tanh", False),
        # a prompt through a 70B model's down projection, bias and residual
        _linear("linear_prompt", 2048, 8192, 28672, 128, "a16", True, "none", True),
        # one token, few small experts: launch latency
        _moe("moe_one", 1, 8, 2, 576, 1536, 32, "softmax", "silu", True),
        # one token, many experts
        _moe("moe_token", 1, 64, 8, 2048, 1024, 128, "softmax", "silu", True),
        # a batch's tokens spread thinly over many experts, sigmoid scores with a selection bias
        _moe("moe_batch", 33, 128, 8, 2048, 768, 128, "sigmoid", "silu", True),
        # a batch over few large experts of an 8B model's size
        _moe("moe_wide", 24, 8, 2, 4096, 14336, 128, "softmax", "gelu_tanh", False),
        # a prompt: every expert has many tokens
        _moe("moe_prompt", 1999, 64, 6, 2048, 1024, 128, "softmax", "silu", True),
        # one user's logits, a short chat
        _adjust("adjust_one", 1, 50001, "f32", 700, 20, False),
        # a batch, some rows bound to a grammar
        _adjust("adjust_batch", 200, 131072, "bf16", 4000, 100, True),
        # few users with very long contexts
        _adjust("adjust_long", 3, 131072, "f32", 100000, 0, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_EXPERTS = [(576, 1536), (1024, 512), (2048, 768), (2048, 1024), (1536, 4096), (4096, 1280), (3840, 1920)]
_ACTS = ["none", "silu", "gelu_tanh", "gelu", "relu"]


def draw(rng):
    op = rng.choice(["linear", "linear", "moe", "moe", "moe", "adjust"])
    if op == "linear":
        group = rng.choice([32, 64, 128, 128])
        kind = rng.choice(["a16", "a16", "a8"])
        k = group * _log(rng, max(1, 512 // group), 28672 // group)
        n = _log(rng, 500, 28672)
        rows = max(1, min(_log(rng, 1, 2048), int(4.8e11 / n / k)))
        c = _linear("", rows, n, k, group, kind, rng.random() < 0.5, rng.choice(_ACTS), rng.random() < 0.6)
    elif op == "moe":
        hidden, inner = rng.choice(_EXPERTS)
        group = rng.choice([g for g in (32, 64, 128, 128) if hidden % g == 0 and inner % g == 0])
        experts = _log(rng, 4, 128)
        top_k = rng.randint(1, min(8, experts))
        # no more products of a token and an expert than the listed prompt has
        tokens = max(1, min(_log(rng, 1, 2048), int(2.6e11 / experts / hidden / inner)))
        c = _moe("", tokens, experts, top_k, hidden, inner, group, rng.choice(["softmax", "sigmoid"]),
                 rng.choice(["silu", "gelu_tanh"]), rng.random() < 0.5)
    else:
        vocab = _log(rng, 1000, 262144)
        rows = max(1, min(_log(rng, 1, 200), 26000000 // vocab))
        history = max(1, min(_log(rng, 1, 100000), 800000 // rows))
        c = _adjust("", rows, vocab, rng.choice(["bf16", "f32"]), history, rng.choice([0, 5, 300]), rng.random() < 0.6)
    del c["name"]
    return c


def work(c):
    if c["op"] == "linear":
        m, n, k = c["rows"], c["n"], c["k"]
        bytes_ = 2 * m * k + n * k / 2 + 4 * n * k / c["group"] + 2 * m * n * (2 if c["residual"] else 1)
        bytes_ += 4 * n if c["bias"] else 0
        bytes_ += m * k + 4 * m if c["kind"] == "a8" else 0
        return {"bytes": int(bytes_), "flops": 2 * m * n * k}
    if c["op"] == "moe":
        t, e, k, h, i = c["tokens"], c["experts"], c["top_k"], c["hidden"], c["inner"]
        # experts that some token chooses, were the choices even
        active = e * (1 - (1 - k / e) ** t)
        bytes_ = active * 3 * h * i * (0.5 + 4 / c["group"]) + 2 * t * h * (3 if c["residual"] else 2) + 2 * e * h + 8 * t * k
        return {"bytes": int(bytes_), "flops": 6 * t * k * h * i + 2 * t * e * h}
    n = c["rows"] * c["vocab"]
    return {"bytes": 2 * n * (2 if c["dtype"] == "bf16" else 4) + (n // 8 if c["mask"] else 0) + 4 * sum(_lengths(c)),
            "flops": 4 * n}


def _lengths(c):
    """Tokens behind each row: the longest first, down to half of it."""
    return [c["history"] - (r * 389) % (c["history"] // 2 + 1) for r in range(c["rows"])]


# ------------------------------------------------------------------ prepare

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 6007 + 29)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _weight(g, n, k, group):
    """One weight [n, k]: 4-bit codes with a scale and zero point for each group of k, as they are kept in files
    (`packed`, `scale`, `zero`) and as the products read them (`wq`, `sz`)."""
    x = (0.7 / math.sqrt(k)) * _normal(g, n, k // group, group)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).half().float()
    z = (-lo / s).round()
    u = ((x / s).round() + z).clamp(0, 15).to(torch.int32).view(n, k)
    del x
    s, z = s.view(n, -1).half(), z.view(n, -1).half()
    packed = (u[:, 0::2] | u[:, 1::2] << 4).to(torch.uint8)
    # eight codes to a word, the even ones in its low half; then rows by sixteens, 32 codes of each in turn
    word = torch.zeros(n, k // 8, dtype=torch.int32, device=DEV)
    for j in range(8):
        word |= u[:, j::8] << (4 * (j // 2) + 16 * (j % 2))
    both = s.view(torch.int16).int() & 0xFFFF | z.view(torch.int16).int() << 16
    return {"packed": packed, "scale": s, "zero": z, "wq": _by_sixteens(word, 4).view(n, -1),
            "sz": _by_sixteens(both, 1).view(n, -1)}


def _by_sixteens(x, run):
    n, k = x.shape
    whole = n // 16 * 16
    parts = [y.view(-1, rows, k // run, run).transpose(1, 2).reshape(-1)
             for y, rows in ((x[:whole], 16), (x[whole:], n - whole)) if y.numel()]
    return torch.cat(parts)


def _stack(weights):
    return {key: torch.stack([w[key] for w in weights]) for key in weights[0]}


def _int(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _prepare_linear(c, g):
    m, n, k = c["rows"], c["n"], c["k"]
    x = _normal(g, m, k)
    x[:, torch.randint(k, (4,), generator=g, device=DEV)] *= 8        # a few features stand out
    return {"x": x.to(torch.bfloat16), "w": _weight(g, n, k, c["group"]),
            "bias": 0.3 * _normal(g, n) if c["bias"] else None,
            "residual": (2 * _normal(g, m, n)).to(torch.bfloat16) if c["residual"] else None}


def _prepare_moe(c, g):
    t, e, h = c["tokens"], c["experts"], c["hidden"]
    router = (1.5 / math.sqrt(h) * _normal(g, e, h)).to(torch.bfloat16)
    pick = 0.02 * _normal(g, e) if c["score"] == "sigmoid" else None
    # a token whose last chosen expert is next to even with the first left out has no one answer in any
    # arithmetic: of a few tokens too many, those with the clearest choice are taken
    x = _normal(g, t + 16 + t // 2, h).to(torch.bfloat16)
    if c["top_k"] < e:
        v = x.double() @ router.double().T
        v = v if pick is None else torch.sigmoid(v) + pick
        v = v.sort(dim=1, descending=True).values
        clear = (v[:, c["top_k"] - 1] - v[:, c["top_k"]]).argsort(descending=True)[:t]
        x = x[clear.sort().values]
    x = x[:t].contiguous()
    # (expert by expert: their numbers in 32 bits do not lie in memory all at once)
    size = {"gate": (c["inner"], h), "up": (c["inner"], h), "down": (h, c["inner"])}
    s = {name: _stack([_weight(g, *nk, c["group"]) for _ in range(e)]) for name, nk in size.items()}
    return {**s, "x": x, "router": router, "pick": pick,
            "residual": _normal(g, t, h).to(torch.bfloat16) if c["residual"] else None}


def _prepare_adjust(c, g, rng):
    b, v = c["rows"], c["vocab"]
    s = {"logits": (3 * _normal(g, b, v)).to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)}
    lengths = _lengths(c)
    # words come again as words do, a few of them often
    s["history"] = (v * torch.rand(sum(lengths), generator=g, device=DEV) ** 4).to(torch.int32).clamp(max=v - 1)
    s["history_start"] = _int(np.concatenate([[0], np.cumsum(lengths)]))
    s["prompt_len"] = _int([int(rng.integers(0, n + 1)) for n in lengths])
    s["repetition"] = torch.tensor(rng.choice([1.0, 1.1, 1.3], b), dtype=torch.float32, device=DEV)
    s["presence"] = torch.tensor(rng.choice([0.0, 0.4, 1.0], b), dtype=torch.float32, device=DEV)
    s["frequency"] = torch.tensor(rng.choice([0.0, 0.2, 0.5], b), dtype=torch.float32, device=DEV)
    s["bias_start"] = s["bias_ids"] = s["bias_values"] = s["mask"] = None
    if c["biases"]:
        counts = [min(v, int(rng.integers(0, c["biases"] + 1))) for _ in range(b)]
        s["bias_start"] = _int(np.concatenate([[0], np.cumsum(counts)]))
        s["bias_ids"] = _int(np.concatenate([rng.choice(v, n, replace=False) for n in counts]))
        s["bias_values"] = 4 * _normal(g, sum(counts))
    if c["mask"]:
        # a third of the rows may say anything, some next to nothing, the others a part of the vocabulary
        share = torch.tensor(rng.choice([1.0, 0.003, 0.2], b), dtype=torch.float32, device=DEV)[:, None]
        words = -(-v // 32)
        s["mask"] = torch.zeros(b, words, dtype=torch.int32, device=DEV)
        for j in range(32):
            s["mask"] |= (torch.rand(b, words, generator=g, device=DEV) < share).int() << j
    return s


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng(int(seed))
    if case["op"] == "linear":
        s = _prepare_linear(case, g)
    elif case["op"] == "moe":
        s = _prepare_moe(case, g)
    else:
        s = _prepare_adjust(case, g, rng)
    s["c"] = case
    return s


# -------------------------------------------------------------- plain forms

def _dequantized(w):
    packed, scale, zero = w["packed"], w["scale"].float(), w["zero"].float()
    u = torch.stack([packed & 15, packed >> 4], -1).view(*scale.shape, -1).float()
    return ((u - zero[..., None]) * scale[..., None]).view(*packed.shape[:-1], -1)


def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    return x.clamp(min=0) if act == "relu" else x


def _rows_e4m3(x):
    scale = (x.float().abs().amax(1) / 448).clamp(min=1e-8)
    # (the quotient to the last bit: a code hangs on it)
    q = (x.double() / scale.double()[:, None]).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    return q, scale


def _plain_linear(s):
    c = s["c"]
    if c["kind"] == "a8":
        q, scale = _rows_e4m3(s["x"])
        y = q.float() @ _dequantized(s["w"]).T * scale[:, None]
    else:
        y = s["x"].float() @ _dequantized(s["w"]).T
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(torch.bfloat16)
    return (y, q, scale) if c["kind"] == "a8" else y


def _plain_moe(s):
    c = s["c"]
    x = s["x"].float()
    logits = x @ s["router"].float().T
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
        ids = (score + s["pick"]).sort(dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    else:
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        score = p / p.sum(1, keepdim=True)
        ids = logits.sort(dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    weights = score.gather(1, ids)
    weights = weights / weights.sum(1, keepdim=True)
    # the experts to go through: those of each choice where these are fewer, else all of them
    if ids.numel() < c["experts"]:
        chosen = ids.flatten()
        place = torch.arange(ids.numel(), device=DEV).view_as(ids)
    else:
        chosen, place = torch.arange(c["experts"], device=DEV), ids
    share = torch.zeros(x.shape[0], chosen.numel(), device=DEV).scatter_(1, place, weights)
    gate, up, down = (_dequantized({key: v[chosen] for key, v in s[name].items() if key not in ("wq", "sz")})
                      for name in ("gate", "up", "down"))
    h = _act(gate.flatten(0, 1) @ x.T, c["act"]) * (up.flatten(0, 1) @ x.T)
    h = (h.view(chosen.numel(), -1, x.shape[0]) * share.T[:, None]).flatten(0, 1)
    y = (down.transpose(0, 1).flatten(1) @ h).T
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16), ids.to(torch.int32), weights


def _plain_adjust(s):
    x = s["logits"].float()
    b, v = x.shape
    start = s["history_start"].long()
    at = torch.arange(s["history"].numel(), device=DEV)
    row = torch.bucketize(at, start[1:], right=True)
    token = row * v + s["history"].long()
    answered = (at - start[row] >= s["prompt_len"].long()[row]).float()
    seen = torch.zeros(b * v, device=DEV).index_fill_(0, token, 1.0).view(b, v)
    count = torch.zeros(b * v, device=DEV).index_add_(0, token, answered).view(b, v)
    r = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0).float()
    if s["bias_ids"] is not None:
        start = s["bias_start"].long()
        row = torch.bucketize(torch.arange(s["bias_ids"].numel(), device=DEV), start[1:], right=True)
        x.view(-1)[row * v + s["bias_ids"].long()] += s["bias_values"]
    if s["mask"] is not None:
        j = torch.arange(v, device=DEV)
        x = torch.where((s["mask"][:, j // 32] >> (j % 32)) & 1 != 0, x, -math.inf)
    return x.to(s["logits"].dtype)


def run(state):
    s, c = state, state["c"]
    if not own:
        return {"linear": _plain_linear, "moe": _plain_moe, "adjust": _plain_adjust}[c["op"]](s)
    import w4_dequant_gemm_amd as w4
    if c["op"] == "linear":
        args = (s["x"], s["w"]["wq"], s["w"]["sz"], c["group"])
        more = {"bias": s["bias"], "act": c["act"], "residual": s["residual"]}
        if c["kind"] == "a8":
            y, xq, xscale = w4.w4a8_linear(*args, **more)
            return y, xq.view(torch.float8_e4m3fn), xscale
        return w4.w4a16_linear(*args, **more)
    if c["op"] == "moe":
        ids, weights = w4.w4_route(s["x"], s["router"], c["top_k"], score=c["score"], bias=s["pick"])
        y = w4.w4a16_moe(s["x"], ids, weights, s["gate"], s["up"], s["down"], c["group"], c["act"],
                         residual=s["residual"])
        return y, ids, weights
    return w4.w4_adjust_logits(s["logits"], history=s["history"], history_start=s["history_start"],
                               prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
                               frequency=s["frequency"], bias_start=s["bias_start"], bias_ids=s["bias_ids"],
                               bias_values=s["bias_values"], mask=s["mask"])


# -------------------------------------------------------------------- exact

def _weight64(w):
    n = w["packed"].shape[0]
    u = torch.empty(n, 2 * w["packed"].shape[1], dtype=torch.float64, device=DEV)
    u[:, 0::2] = (w["packed"] % 16).double()
    u[:, 1::2] = (w["packed"] // 16).double()
    times = u.shape[1] // w["scale"].shape[1]
    return (u - w["zero"].double().repeat_interleave(times, 1)) * w["scale"].double().repeat_interleave(times, 1)


def _act64(x, act):
    f = torch.nn.functional
    return {"none": lambda: x, "silu": lambda: f.silu(x), "gelu_tanh": lambda: f.gelu(x, approximate="tanh"),
            "gelu": lambda: f.gelu(x), "relu": lambda: f.relu(x)}[act]()


def _exact_linear(s):
    c = s["c"]
    x = s["x"].double()
    if c["kind"] == "a8":
        # the rows' scales and codes are whole results of 32 and 8 bits by definition
        scale = torch.maximum(s["x"].abs().max(1).values.float() / 448.0, torch.tensor(1e-8, device=DEV))
        codes = torch.clamp((x / scale.double().unsqueeze(1)).float(), -448.0, 448.0).to(torch.float8_e4m3fn)
        x = codes.double() * scale.double().unsqueeze(1)
    y = torch.empty(c["rows"], c["n"], dtype=torch.float64, device=DEV)
    for i in range(0, c["rows"], 256):
        y[i:i + 256] = torch.matmul(x[i:i + 256], _weight64(s["w"]).t())
    if c["bias"]:
        y += s["bias"].double().unsqueeze(0)
    y = _act64(y, c["act"])
    if c["residual"]:
        y += s["residual"].double()
    return (y, codes.double(), scale.double()) if c["kind"] == "a8" else y


def _exact_moe(s):
    c = s["c"]
    x = s["x"].double()
    logits = torch.matmul(x, s["router"].double().t())
    if c["score"] == "sigmoid":
        score = torch.sigmoid(logits)
        rank = score + s["pick"].double().unsqueeze(0)
    else:
        score = torch.softmax(logits, 1)
        rank = logits
    ids = torch.topk(rank, c["top_k"], dim=1, sorted=True).indices
    weights = torch.gather(score, 1, ids)
    weights /= weights.sum(1, keepdim=True)
    y = s["residual"].double() if c["residual"] else torch.zeros_like(x)
    for e in range(c["experts"]):
        token, place = torch.nonzero(ids == e, as_tuple=True)
        if token.numel():
            gate, up, down = (_weight64({key: v[e] for key, v in s[n].items()}) for n in ("gate", "up", "down"))
            rows = x[token]
            h = _act64(rows @ gate.t(), c["act"]) * (rows @ up.t())
            y.index_add_(0, token, (h @ down.t()) * weights[token, place].unsqueeze(1))
    return y, ids.int(), weights


def _exact_adjust(s):
    out = s["logits"].double()
    b, v = out.shape
    history, start, prompt = s["history"].cpu().numpy(), s["history_start"].tolist(), s["prompt_len"].tolist()
    for r in range(b):
        tokens = history[start[r]:start[r + 1]]
        all_ = torch.from_numpy(np.bincount(tokens, minlength=v)).to(DEV)
        later = torch.from_numpy(np.bincount(tokens[prompt[r]:], minlength=v)).to(DEV).double()
        p = s["repetition"][r].double()
        x = out[r]
        x = torch.where(all_ != 0, torch.where(x > 0, x / p, x * p), x)
        x = x - s["frequency"][r].double() * later - s["presence"][r].double() * later.clamp(max=1)
        if s["bias_start"] is not None:
            lo, hi = s["bias_start"][r:r + 2].tolist()
            x = x.index_add(0, s["bias_ids"][lo:hi].long(), s["bias_values"][lo:hi].double())
        if s["mask"] is not None:
            bits = np.unpackbits(s["mask"][r].cpu().numpy().view(np.uint8), bitorder="little")[:v]
            x = x.masked_fill(torch.from_numpy(bits == 0).to(DEV), -math.inf)
        out[r] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "moe": _exact_moe, "adjust": _exact_adjust}[case["op"]](s)
