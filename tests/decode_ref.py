"""64-bit references of the decoding calls, written from their formulas in plain
NumPy loops, and random cache contents in the library's layout."""
import math

import numpy as np
import torch

E4M3_MAX = 448.0


def cache_shapes(pages, hk, d, page, e4m3):
    c = 16 if e4m3 else 8
    return (pages, hk, page // 16, d // c, 16, c), (pages, hk, page // 16, 16 // c, d, c)


def to_tokens(k, v):
    """Cache arrays [pages, hk, blocks, ...] -> [pages * page_size, hk, d] values in slot order (float64)."""
    if k.dtype == torch.uint8:
        k, v = k.view(torch.float8_e4m3fn).float(), v.view(torch.float8_e4m3fn).float()
    k, v = k.double().cpu(), v.double().cpu()
    pages, hk, nb, nc, _, c = k.shape
    d = nc * c
    kt = k.permute(0, 2, 4, 1, 3, 5).reshape(pages * nb * 16, hk, d)
    vt = v.permute(0, 2, 3, 5, 1, 4).reshape(pages * nb * 16, hk, d)
    return kt.numpy(), vt.numpy()


def random_cache(rng, pages, hk, d, page, e4m3, device):
    ks, vs = cache_shapes(pages, hk, d, page, e4m3)
    out = []
    for s in (ks, vs):
        x = torch.from_numpy(rng.standard_normal(s).astype(np.float32))
        out.append((40 * x).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8).to(device) if e4m3
                   else x.to(torch.bfloat16).to(device))
    return out


def page_table(rng, lengths, page, spare=2):
    need = [max(1, -(-n // page)) for n in lengths]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lengths), max(need)), 0, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pages, table


def random_tree(rng, n):
    """Ancestor sets (each node's own bit included) and depths of a random tree."""
    sees, depth = [], []
    for i in range(n):
        p = int(rng.integers(max(0, i - 5), i)) if i else -1
        sees.append((sees[p] if i else 0) | 1 << i)
        depth.append(depth[p] + 1 if i else 0)
    return sees, depth


def pack_tree(all_sees, words):
    rows = [[(s >> 64 * w) & (1 << 64) - 1 for w in range(words)] for s in all_sees]
    return torch.from_numpy(np.array(rows, dtype=np.uint64).view(np.int64).reshape(len(all_sees), words))


def attention(q, keys, values, past, scale, sees=None, positions=None, window=0):
    """One sequence: q [n, hq, d], keys/values [len, hk, d] (float64).  Returns the outputs and, per output, a
    bound of |bf16 kernel - this|: the output's rounding to bf16 (8 bits: 2^-8 |o|), plus, in units of A = sum p
    |v| / sum p, p's rounding to bf16 (2^-8), the scores' fp32 errors twice (numerator and sum; (d + 2) 2^-24 of the
    largest sum |q k| scale, and the exponent's own, 2^-21) and the sums' (length 2^-24 twice)."""
    n, hq, d = q.shape
    length, hk = keys.shape[:2]
    out, tol = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    at = [past + i if positions is None else int(positions[i]) for i in range(n)]
    for i in range(n):
        see = np.zeros(length, bool)
        for j in range(length):
            if j < past:
                see[j] = not window or j > at[i] - window
            else:
                node = j - past
                see[j] = (bool(sees[i] >> node & 1) if sees is not None else node <= i) and \
                    (not window or at[node] > at[i] - window)
        if not see.any():
            continue
        for h in range(hq):
            kh, vh = keys[see, h // (hq // hk)], values[see, h // (hq // hk)]
            s = scale * (kh @ q[i, h])
            p = np.exp(s - s.max())
            out[i, h] = p @ vh / p.sum()
            spread = (d + 2) * 2.0 ** -24 * np.max(np.abs(kh) @ np.abs(q[i, h])) * abs(scale) + 2.0 ** -21
            big = p @ np.abs(vh) / p.sum()
            tol[i, h] = 2.0 ** -8 * np.abs(out[i, h]) + big * (2.0 ** -8 + 2 * spread + 2 * length * 2.0 ** -24)
    return out, 1.02 * tol + 1e-30


def head_rows(x, norm, eps, rope, positions, rot, interleaved):
    """Norm and rotation of [T, heads, d] in float64, and a bound of the fp32 error before the last rounding:
    the sum of squares and the products, (d + 16) 2^-24 of |a| + |b| of a pair."""
    x = x.astype(np.float64)
    d = x.shape[-1]
    y = x if norm is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * norm.astype(np.float64)
    z, size = y.copy(), np.abs(y)
    if rope is not None:
        for j in range(rot // 2):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
            co = rope[positions, j].astype(np.float64)[:, None]
            si = rope[positions, rot // 2 + j].astype(np.float64)[:, None]
            z[..., a] = y[..., a] * co - y[..., b] * si
            z[..., b] = y[..., b] * co + y[..., a] * si
            size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return z, (d + 16) * 2.0 ** -24 * size


def rope_table(rows, rot):
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot / 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def kept_weights(x, temperature, top_k, top_p, min_p):
    """Real weights exp((x - max) / T) of the kept tokens (0 elsewhere), float64."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    order = np.lexsort((np.arange(len(x)), -x))
    if temperature == 0:
        w = np.zeros(len(x))
        w[order[0]] = 1
        return w
    w = np.exp((x - x.max()) / temperature)[order]
    if top_k and top_k > 0:
        w[top_k:] = 0
    keep = np.ones(len(x), bool)
    if top_p is not None:
        before = np.cumsum(w) - w
        keep &= before < max(math.floor(np.float32(top_p) * 2.0 ** 24) / 2.0 ** 24 * w.sum(), 1e-300)
    if min_p is not None:
        keep &= w >= min_p
    out = np.zeros(len(x))
    out[order] = np.where(keep, w, 0)
    return out
