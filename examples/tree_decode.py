"""Decoding with drafted trees on 4-bit weights: a small random transformer whose
products are W4A16 and whose decode loop is the library's calls.

A step appends the drafted nodes' keys and values to the paged cache
(``w4_kv_append``), lets every node attend to its context and its ancestors
(``w4_tree_attention``), draws a token after every node (``w4_sample``) and keeps
the path of the nodes that were drawn (``w4_kv_move``).  The uniform number of a
draw belongs to the sequence and the position, so a drafted node is accepted
exactly if plain decoding would have drawn it there, and trees change the speed
but not the text (up to the products' rounding, which differs with the number of
rows).

Drafts come from the text itself: what followed earlier occurrences of the last
token.  (The random model is made to favour one successor of every token, in
rings of 32, so that its text repeats itself as real text does.)

    python examples/tree_decode.py [--batch 4] [--tokens 200] [--e4m3] [--temperature 0.7]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4_dequant_gemm_amd as w4  # noqa: E402


class Linear:
    """A random [N, K] weight in 4-bit groups of G."""

    def __init__(self, gen, N, K, G, device, add=0.0):
        W = torch.randn((N, K), generator=gen, device=device) * K ** -0.5 + add
        self.G, self.codes = G, w4.w4_quantize_blockwise(W, G, "asym")
        self.packed = w4.w4_prepack(self.codes["packed"], self.codes["scale"], self.codes["zero"], G, "asym")

    def __call__(self, x):
        return w4.w4a16_gemm(x, self.packed["wq"], self.packed["sz"], self.G)


def rms_norm(x):
    return torch.nn.functional.rms_norm(x, x.shape[-1:], eps=1e-6)


class Model:
    """``layers`` pre-norm layers with normed and rotated queries and keys, a gated SiLU MLP, and an output product."""

    def __init__(self, layers=4, hidden=576, heads=9, kv_heads=3, head_dim=64, mlp=1536, vocab=2048, group=64,
                 context=2048, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim, self.device = heads, kv_heads, head_dim, device
        lin = lambda n, k: Linear(gen, n, k, group, device)  # noqa: E731
        self.embed = torch.randn((vocab, hidden), generator=gen, device=device).to(torch.bfloat16)
        self.layers = [{"qkv": lin((heads + 2 * kv_heads) * head_dim, hidden), "o": lin(hidden, heads * head_dim),
                        "gate": lin(mlp, hidden), "up": lin(mlp, hidden), "down": lin(hidden, mlp)} for _ in range(layers)]
        ring = torch.arange(vocab, device=device)
        before = ring // 32 * 32 + (ring - 1) % 32           # a token's logit grows with the one before it in its ring
        self.out = Linear(gen, vocab, hidden, group, device, add=20 / hidden * self.embed[before].float())
        self.norm = torch.ones(head_dim, device=device)      # weights of the queries' and keys' norms
        angle = torch.arange(context, device=device)[:, None] * 10000.0 ** (-torch.arange(head_dim // 2, device=device) / (head_dim / 2))
        self.rope = torch.cat([angle.cos(), angle.sin()], 1)

    def cache(self, pages, page_size, e4m3=False):
        """A cache for all layers, and the scales of its codes (normed keys are at most sqrt(head_dim))."""
        k, v = w4.w4_kv_cache(pages, self.kv_heads, self.head_dim, page_size, e4m3=e4m3, layers=len(self.layers), device=self.device)
        one = torch.ones(self.kv_heads, device=self.device)
        return k, v, {"k_scale": one * self.head_dim ** 0.5 / 448, "v_scale": one * 16 / 448} if e4m3 else {}

    def __call__(self, tokens, slots, positions, cache, page_table, kv_len, q_start, max_q, max_kv, tree=None):
        """Logits [T, vocab] of the rows ``tokens`` (int32 [T]), whose keys and values go to ``slots``."""
        k, v, scales = cache
        hq, hk = self.heads, self.kv_heads
        x = self.embed[tokens]
        for i, layer in enumerate(self.layers):
            qkv = layer["qkv"](rms_norm(x)).unflatten(1, (hq + 2 * hk, self.head_dim))
            q = w4.w4_kv_append(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, k[i], v[i], rope=self.rope,
                                positions=positions, q_norm=self.norm, k_norm=self.norm, **scales)
            o = w4.w4_tree_attention(q, k[i], v[i], page_table, kv_len, q_start, max_q, max_kv, tree=tree, **scales)
            x = x + layer["o"](o.flatten(1))
            h = w4.w4a16_gate_up(rms_norm(x), layer["gate"].packed, layer["up"].packed, layer["gate"].G)
            x = x + layer["down"](h)
        return self.out(rms_norm(x))


def draft(text, nodes, depth):
    """A tree of at most ``nodes`` tokens below text[-1]: what followed its latest occurrences, ``depth`` tokens each.
    Returns tokens, parents and depths, the root (text[-1] itself) first."""
    tokens, parents, depths = [text[-1]], [-1], [0]
    child = {}
    for at in range(len(text) - 2, -1, -1):
        if len(tokens) >= nodes:
            break
        if text[at] != text[-1]:
            continue
        node = 0
        for t in text[at + 1:at + 1 + depth]:
            if (node, t) not in child:
                if len(tokens) >= nodes:
                    break
                child[node, t] = len(tokens)
                tokens.append(t)
                parents.append(node)
                depths.append(depths[node] + 1)
            node = child[node, t]
    return tokens, parents, depths


def decode(model, prompts, count, *, nodes=16, depth=8, page_size=32, e4m3=False, temperature=0.0, top_p=1.0, seed=1):
    """``count`` tokens after every prompt (lists of ints; all of the prompt is given).  ``nodes`` 1: plain decoding.
    Returns the texts, the number of steps after the prompt, and their seconds."""
    dev, B = model.device, len(prompts)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    longest = max(map(len, prompts)) + count + nodes
    per = -(-longest // page_size)
    cache = model.cache(B * per, page_size, e4m3)
    gen = torch.Generator(device=dev).manual_seed(seed)
    table = torch.randperm(B * per, generator=gen, device=dev).to(torch.int32).view(B, per)
    host_table = table.tolist()
    last = max(map(len, prompts)) + count    # no draw that is kept is behind it
    uniform = torch.rand((B, last + 1), generator=torch.Generator(device=dev).manual_seed(seed), device=dev)
    slot = lambda b, t: host_table[b][t // page_size] * page_size + t % page_size  # noqa: E731
    texts = [list(p) for p in prompts]
    cached = [0] * B

    def step(trees, chain):
        """Appends every sequence's nodes, draws a token after each, and keeps the drawn path."""
        n = [len(t[0]) for t in trees]
        start = [0]
        for c in n:
            start.append(start[-1] + c)
        tokens, slots, positions, where, masks = [], [], [], [], []
        words = -(-max(n) // 64)
        for b, (toks, parents, depths) in enumerate(trees):
            tokens += toks
            slots += [slot(b, cached[b] + i) for i in range(len(toks))]
            positions += [cached[b] + d for d in depths]
            where += [b * (last + 1) + min(cached[b] + d + 1, last) for d in depths]
            sees = []
            for i, p in enumerate(parents):
                sees.append((sees[p] if p >= 0 else 0) | 1 << i)
            if not chain:
                masks += [[(s >> 64 * w & (1 << 64) - 1) - (1 << 64 if s >> 64 * w + 63 & 1 else 0) for w in range(words)] for s in sees]
        lengths = [c + m for c, m in zip(cached, n)]
        logits = model(i32(tokens), i32(slots), i32(positions), cache, table, i32(lengths), i32(start), max(n), max(lengths),
                       None if chain else torch.tensor(masks, dtype=torch.int64, device=dev))
        u = uniform.view(-1)[torch.tensor(where, device=dev)]
        full = lambda x: torch.full((len(tokens),), x, device=dev)  # noqa: E731
        drawn, _ = w4.w4_sample(logits, u, temperature=full(temperature), top_p=full(top_p) if top_p < 1 else None)
        drawn = drawn.tolist()
        paths, new = [], []
        for b, (toks, parents, _) in enumerate(trees):
            at, path, out = (len(toks) - 1, list(range(len(toks))), []) if chain else (0, [0], [])
            while True:
                out.append(drawn[start[b] + at])
                child = next((i for i in range(at + 1, len(toks)) if parents[i] == at and toks[i] == out[-1]), None)
                if child is None:
                    break
                at = child
                path.append(at)
            paths.append(path)
            new.append(out)
        if any(p[-1] != len(p) - 1 for p in paths):
            width = max(map(len, paths))
            w4.w4_kv_move(cache[0], cache[1], table, i32(cached), i32([p + [0] * (width - len(p)) for p in paths]), i32([len(p) for p in paths]))
        for b in range(B):
            cached[b] += len(paths[b])
            texts[b] += new[b]

    step([(p, list(range(-1, len(p) - 1)), list(range(len(p)))) for p in prompts], True)
    torch.cuda.synchronize()
    began, steps = time.perf_counter(), 0
    while min(len(t) - len(p) for t, p in zip(texts, prompts)) < count:
        # (sequences that are through draft nothing more and wait for the others)
        done = [len(t) - len(p) >= count for t, p in zip(texts, prompts)]
        trees = [draft(t, 1 if d else nodes, depth) for t, d in zip(texts, done)]
        before = [len(t) for t in texts]
        step(trees, nodes == 1)
        for b in range(B):
            if done[b]:
                del texts[b][before[b]:]
                cached[b] = before[b] - 1
        steps += 1
    torch.cuda.synchronize()
    return [t[:len(p) + count] for t, p in zip(texts, prompts)], steps, time.perf_counter() - began


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--batch", type=int, default=4)
    a.add_argument("--prompt", type=int, default=60, help="longest prompt")
    a.add_argument("--tokens", type=int, default=200)
    a.add_argument("--nodes", type=int, default=16)
    a.add_argument("--e4m3", action="store_true", help="8-bit cache")
    a.add_argument("--temperature", type=float, default=0.0)
    a.add_argument("--top-p", type=float, default=1.0)
    a = a.parse_args()
    model = Model()
    gen = torch.Generator().manual_seed(0)
    prompts = [torch.randint(0, model.embed.shape[0], (max(1, a.prompt - 7 * b),), generator=gen).tolist() for b in range(a.batch)]
    results = []
    for nodes in (1, a.nodes):
        run = lambda: decode(model, prompts, a.tokens, nodes=nodes, e4m3=a.e4m3, temperature=a.temperature, top_p=a.top_p)  # noqa: E731,B023
        run()
        texts, steps, seconds = run()
        results.append(texts)
        print(f"{nodes:3d} nodes a step: {a.batch * a.tokens / seconds:8.0f} tokens/s, {steps} steps, "
              f"{(a.tokens - 1) / steps:.2f} tokens a step and sequence", flush=True)
    same = [next((i for i, (x, y) in enumerate(zip(*t)) if x != y), len(t[0])) - len(p) for t, p in zip(zip(*results), prompts)]
    print(f"equal tokens before the first difference, of {a.tokens}: {same}", flush=True)


if __name__ == "__main__":
    main()
