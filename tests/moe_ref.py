"""64-bit references of the mixture-of-experts calls and bounds on how far fp32 arithmetic may be from them.

A rounding to fp32 is off by at most U = 2^-24 of the value, one to bf16 by 2^-8 of it (half a step)."""
import numpy as np
import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8


def experts(gen, E, N, K, G, device, zeros="asym"):
    """E random weights [N, K] in 4-bit groups: the canonical arrays, the stacked GPU layout (w4_prepack), and W' with
    s (256 + 2 |z|) of every weight (what a product with 128 + u passes through) in 64 bits."""
    import w4_dequant_gemm_amd as w4
    out = {"wq": [], "sz": [], "W": [], "size": []}
    for _ in range(E):
        u = torch.randint(0, 16, (N, K), generator=gen, device=device, dtype=torch.int32)
        s = (0.01 + 0.05 * torch.rand((N, K // G), generator=gen, device=device)).half()
        z = torch.randint(0, 16, (N, K // G), generator=gen, device=device).half()
        if zeros == "far":                    # zero points outside the codes' range
            z = torch.randint(-40, 60, (N, K // G), generator=gen, device=device).half()
        packed = (u[:, 0::2] | u[:, 1::2] << 4).to(torch.uint8)
        p = w4.w4_prepack(packed, s, z, G, "asym")
        out["wq"].append(p["wq"])
        out["sz"].append(p["sz"])
        wide = lambda x: x.double().repeat_interleave(G, 1)  # noqa: E731
        out["W"].append((u.double() - wide(z)) * wide(s))
        out["size"].append(wide(s) * (256 + 2 * wide(z).abs()))
    return {k: torch.stack(v) for k, v in out.items()}


def activation(x, act):
    f = torch.nn.functional
    return f.silu(x) if act == "silu" else f.gelu(x, approximate="tanh")


def product(x, dx, w, e):
    """x . W'[e]^T and a bound on its error for operands known to dx.  Sums run over at most 160 additions a group and
    the groups' (fewer than 160 of K / 32 groups and 8 waves together in any chain of these tests), each off by U of a
    partial sum, which is at most what passes through it: s (128 + u + 128 + |z|) |x|, below `size` |x|."""
    y = x @ w["W"][e].T
    return y, dx @ w["W"][e].abs().T + 320 * U * (x.abs() @ w["size"][e].T)


def moe(x, ids, weights, gate, up, down, act, residual=None):
    """(Y, bound): Y in 64 bits, the bound for the kernels' bf16 result."""
    x, weights = x.double(), weights.double()
    E = gate["W"].shape[0]
    y = torch.zeros_like(x) if residual is None else residual.double()
    bound = torch.zeros_like(x)
    zero = torch.zeros_like(x)
    for e in range(E):
        share = torch.where(ids == e, weights, torch.zeros_like(weights))
        if not bool((ids == e).any()):
            continue
        g, dg = product(x, zero, gate, e)
        u, du = product(x, zero, up, e)
        a = activation(g, act)
        # |act'| < 1.13; the activation itself: eight roundings of at most |g|
        h = a * u
        dh = 1.13 * u.abs() * dg + a.abs() * du + 1.13 * dg * du + 8 * U * g.abs() * u.abs() + 3 * U * h.abs()
        # h is kept as hi + lo, the rest of a rounding to bf16 rounded to bf16, or, from 16 rows an expert on, as bf16
        dh = dh + (BF16 if ids.numel() > 64 and ids.numel() >= 16 * E else 2.0 ** -16) * (h.abs() + dh)
        for j in range(ids.shape[1]):
            w = share[:, j:j + 1]
            o, do = product(w * h, w.abs() * dh, down, e)
            y = y + o
            bound = bound + do + 8 * U * o.abs()
    bound = bound + 40 * U * y.abs()
    return y, bound + BF16 * (y.abs() + bound)


def route(x, router, top_k, score="softmax", bias=None, renormalize=True, scale=1.0):
    """ids, weights (64 bits), the logits' error bound [T, 1], and which places [T, top_k] no error of that size can
    give to another expert: those farther from their neighbours' values than both can move."""
    x, r = x.double(), router.double()
    l = x @ r.T
    # at most H / 32 + 32 + 16 additions in a chain, products of bf16 numbers exact in fp32
    dl = ((x.shape[1] // 32 + 48) * U * (x.abs() @ r.abs().T)).amax(1, keepdim=True)
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    rank, move = l, dl
    if bias is not None:
        rank = s + bias.double()
        # d softmax = s (dl_e - sum s dl) <= 2 s dl, d sigmoid <= dl / 4; and sixteen roundings of numbers up to 1 + |bias|
        move = (2 * dl * s.amax(1, keepdim=True) if score == "softmax" else dl / 4) + 16 * U * (1 + bias.abs().max())
    order = torch.sort(rank, dim=1, descending=True, stable=True)
    ids = order.indices[:, :top_k]
    inf = torch.full((x.shape[0], 1), np.inf, dtype=torch.float64, device=x.device)
    gaps = torch.cat([inf, order.values[:, :-1] - order.values[:, 1:], inf], 1)
    sure = (torch.minimum(gaps[:, :-1], gaps[:, 1:]) > 2 * move)[:, :top_k]
    w = s.gather(1, ids)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    return ids, w * scale, dl, sure
