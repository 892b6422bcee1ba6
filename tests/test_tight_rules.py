"""The limits of ``tight`` on the CPU: the calls' own roundings stay within them for every shape, and results with a part
left out or computed otherwise do not."""
import pytest
import torch

import tight


def _inputs(T, k, E, H, I, G):
    g = torch.Generator().manual_seed(T * 1000 + E)

    def weights(n, kk):
        u = torch.randint(0, 16, (n, kk), generator=g).double()
        s = (0.01 + 0.05 * torch.rand((n, kk // G), generator=g)).half().double().repeat_interleave(G, 1)
        z = torch.randint(0, 16, (n, kk // G), generator=g).double().repeat_interleave(G, 1)
        return (u - z) * s
    x = tight.bf16(torch.randn((T, H), generator=g) / H ** 0.5)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    w = torch.rand((T, k), generator=g).double()
    return x, ids, w, {e: (weights(I, H), weights(I, H), weights(H, I)) for e in sorted(set(ids.flatten().tolist()))}


def _twice(h):
    hi = tight.bf16(h)
    return hi + tight.bf16(h - hi)


def _layer(given, rounding, no_choice=False, no_tile=False, act=torch.nn.functional.silu):
    x, ids, w, experts = given
    y = torch.zeros_like(x)
    for e, (gate, up, down) in experts.items():
        for j in range(ids.shape[1] - int(no_choice)):
            t = (ids[:, j] == e).nonzero()[:, 0]
            h = rounding(act(x[t] @ gate.T) * (x[t] @ up.T) * w[t, j:j + 1])
            if no_tile:
                h[:, -32:] = 0
            y.index_add_(0, t, h @ down.T)
    return y


@pytest.mark.parametrize("shape", tight.MOE)
def test_experts(shape):
    given = _inputs(*shape)
    want = _layer(given, lambda h: h)
    limit = tight.moe_limit(shape)

    def error(y):
        first = tight.bf16(y)
        return tight.moe_error(first, tight.bf16(y - first), want)

    own = tight.bf16 if tight.tiled(*shape) else _twice
    assert error(_layer(given, own)) < limit
    faults = {"nothing": torch.zeros_like(want), "a choice": _layer(given, own, no_choice=True),
              "the last tile of h": _layer(given, own, no_tile=True),
              "another activation": _layer(given, own, act=lambda v: torch.nn.functional.gelu(v, approximate="tanh"))}
    if not tight.tiled(*shape):
        faults["h rounded once"] = _layer(given, tight.bf16)
    for name, y in faults.items():
        assert error(y) > 3 * limit, name


@pytest.mark.parametrize("M,K,N,G", [(1, 576, 500, 32), (5, 8192, 300, 128), (16, 14336, 130, 128), (1, 49152, 33, 128), (100, 4096, 64, 128),
                                     (200, 96, 250, 32)])
@pytest.mark.parametrize("exact", [True, False])
def test_products(M, K, N, G, exact):
    g = torch.Generator().manual_seed(K)
    f = torch.nn.functional
    acts = {"none": (lambda v: v, 1.0), "silu": (f.silu, 1.1), "gelu_tanh": (lambda v: f.gelu(v, approximate="tanh"), 1.13),
            "gelu": (f.gelu, 1.13), "relu": (f.relu, 1.0)}
    u = torch.randint(0, 16, (N, K), generator=g).double()
    s = (0.01 + 0.05 * torch.rand((N, K // G), generator=g)).half().double().repeat_interleave(G, 1)
    z = torch.randint(0, 16, (N, K // G), generator=g).double().repeat_interleave(G, 1)
    W, size = (u - z) * s, s * (256 + 2 * z)
    x = tight.bf16(torch.randn((M, K), generator=g) / K ** 0.5)
    bias = 2 * torch.randn(N, generator=g).double()
    sums, own = x @ W.T, x @ (W if exact else tight.bf16(W)).T
    for name, (act, slope) in acts.items():
        want = act(sums + bias)
        first = tight.bf16(want)
        limit = tight.linear_limit(exact, K, x, size, slope, tight.rms(sums), want)

        def error(y):
            return tight.rms(tight.bf16(y - first) - (want - first))

        assert error(act(own + bias)) < limit, name
        faults = {"no bias": act(own), "the bias behind the activation": act(own) + bias if name != "none" else act(own),
                  "the last 32 k": act(own - x[:, -32:] @ W[:, -32:].T + bias)}
        for other, (a, _) in acts.items():
            # (GELU's two forms are 2e-4 apart: seen where the weights are exact)
            if other != name and (exact or {name, other} != {"gelu", "gelu_tanh"}):
                faults[other] = a(own + bias)
        for fault, y in faults.items():
            assert error(y) > 1.5 * limit, (name, fault, error(y) / limit)
