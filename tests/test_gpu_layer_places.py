"""Results beside their inputs in one array: what lies next to each other without sharing a byte is taken, and gives
what arrays of their own give."""
import pytest

import moe_ref as ref
from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu


def _beside(*tensors):
    """The tensors one right behind the other in one array, as views of it."""
    import torch
    assert all(t.nbytes % 16 == 0 for t in tensors)
    whole = torch.empty(sum(t.nbytes for t in tensors), dtype=torch.uint8, device=dev())
    out, at = [], 0
    for t in tensors:
        v = whole[at:at + t.nbytes].view(t.dtype).view(t.shape)
        v.copy_(t)
        out.append(v)
        at += t.nbytes
    return out


@pytest.mark.parametrize("M", [1, 4, 48, 200])
def test_linear_beside_its_inputs(M):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    g = torch.Generator(device=dev()).manual_seed(M)
    K, N, G = 512, 320, 128
    w = ref.experts(g, 1, N, K, G, dev())
    wq, sz = w["wq"][0], w["sz"][0]
    x = torch.randn((M, K), generator=g, device=dev()).to(torch.bfloat16)
    res, bias = torch.randn((M, N), generator=g, device=dev()).to(torch.bfloat16), torch.randn(N, generator=g, device=dev())
    want = w4.w4a16_linear(x, wq, sz, G, bias=bias, act="silu", residual=res)
    for order in ("xyrb", "bryx", "ryxb"):
        v = dict(zip(order, _beside(*({"x": x, "y": torch.zeros_like(res), "r": res, "b": bias}[c] for c in order))))
        assert torch.equal(w4.w4a16_linear(v["x"], wq, sz, G, bias=v["b"], act="silu", residual=v["r"], Y=v["y"]), want)
        assert torch.equal(v["x"], x) and torch.equal(v["r"], res) and torch.equal(v["b"], bias)
    y, q, s = w4.w4a8_linear(x, wq, sz, G, bias=bias, act="silu", residual=res)
    s4 = torch.zeros((M + 3) // 4 * 4, device=dev())
    for order in ("xqyrs", "sqryx"):
        v = dict(zip(order, _beside(*({"x": x, "y": torch.zeros_like(res), "r": res, "q": torch.zeros_like(q), "s": s4}[c]
                                      for c in order))))
        got = w4.w4a8_linear(v["x"], wq, sz, G, bias=bias, act="silu", residual=v["r"], Y=v["y"], xq=v["q"], xscale=v["s"][:M])
        assert torch.equal(got[0], y) and torch.equal(got[1], q) and torch.equal(got[2], s)
    # in place of the residual, which is the activations' neighbour
    a, b = _beside(x, res)
    assert torch.equal(w4.w4a16_linear(a, wq, sz, G, bias=bias, act="silu", residual=b, Y=b), want)


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_experts_beside_their_inputs(T):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    g = torch.Generator(device=dev()).manual_seed(T)
    k, E, H, I, G = 4, 6, 256, 128, 64
    w = [ref.experts(g, E, n, kk, G, dev()) for n, kk in ((I, H), (I, H), (H, I))]
    x, res = (torch.randn((T, H), generator=g, device=dev()).to(torch.bfloat16) for _ in range(2))
    ids = torch.randint(0, E, (T, k), generator=g, device=dev(), dtype=torch.int32)
    weights = torch.rand((T, k), generator=g, device=dev())
    want = w4.w4a16_moe(x, ids, weights, *w, G, residual=res)
    need = (w4.w4a16_moe_workspace_bytes(T, k, E, H, I, G) + 15) // 16 * 16
    for order in ("xyriws", "swiryx", "iysxwr"):
        made = {"x": x, "y": torch.zeros_like(x), "r": res, "i": ids, "w": weights,
                "s": torch.zeros(need, dtype=torch.uint8, device=dev())}
        v = dict(zip(order, _beside(*(made[c] for c in order))))
        got = w4.w4a16_moe(v["x"], v["i"], v["w"], *w, G, residual=v["r"], Y=v["y"], workspace=v["s"])
        assert torch.equal(got, want) and torch.equal(v["x"], x) and torch.equal(v["i"], ids) and torch.equal(v["r"], res)
    a, b = _beside(x, res)
    assert torch.equal(w4.w4a16_moe(a, ids, weights, *w, G, residual=b, Y=b), want)
