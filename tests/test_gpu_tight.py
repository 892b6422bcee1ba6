"""The experts' call and the products with an epilogue against 64 bits on the whole, with the limits of ``tight``."""
import pytest

import moe_ref as ref
import tight
from helpers import dev, require_gpu
from test_gpu_linear import SHAPES, _act
from test_gpu_moe import _layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", tight.MOE)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_experts(shape, act):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    T, k, E, H, I, G = shape
    x, ids, weights, gate, up, down, _ = _layer(T + E, *shape)
    first = w4.w4a16_moe(x, ids, weights, gate, up, down, G, act)
    left = w4.w4a16_moe(x, ids, weights, gate, up, down, G, act, residual=-first)
    want = ref.moe(x, ids, weights, gate, up, down, act)[0]
    torch.cuda.synchronize()
    off, limit = tight.moe_error(first, left, want), tight.moe_limit(shape)
    print(f"{shape} {act}: {off:.2e} of at most {limit:.2e}")
    assert off <= limit
    # and the result itself, a rounding of the same
    assert tight.rms(first.double() - want) <= (limit ** 2 + tight.STEP ** 2) ** 0.5 * 1.05 * tight.rms(want)


@pytest.mark.parametrize("kind", ["a16", "a8"])
@pytest.mark.parametrize("M,K,N,G", SHAPES)
def test_products(M, K, N, G, kind):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    g = torch.Generator(device=dev()).manual_seed(M + K + N)
    group = K if G == "row" else G
    w = ref.experts(g, 1, N, K, group, dev())
    wq, sz = w["wq"][0], w["sz"][0]
    x = (torch.randn((M, K), generator=g, device=dev()) / K ** 0.5).to(torch.bfloat16)
    bias = 2 * torch.randn(N, generator=g, device=dev())
    if kind == "a16":
        run, xd = (lambda **kw: w4.w4a16_linear(x, wq, sz, group, **kw)), x.double()
    else:
        _, q, s = w4.w4a8_linear(x, wq, sz, group)
        run, xd = (lambda **kw: w4.w4a8_linear(x, wq, sz, group, **kw)[0]), q.view(torch.float8_e4m3fn).double() * s.double()[:, None]
    # up to 32 rows, groups of 128 and more multiply the whole codes; other kernels weights rounded to bf16
    exact = M <= 32 and group % 128 == 0
    sums = xd @ w["W"][0].T
    for act, slope in ((None, 1.0), ("silu", 1.1), ("gelu_tanh", 1.13), ("relu", 1.0), ("gelu", 1.13)):
        want = _act(sums + bias.double(), act)
        first = want.to(torch.bfloat16)
        left = run(bias=bias, act=act, residual=-first)
        off = tight.rms(left.double() - (want - first.double()))
        limit = tight.linear_limit(exact, K, xd, w["size"][0], slope, tight.rms(sums), want)
        print(f"{act}: {off:.2e} of at most {limit:.2e}")
        assert off <= limit, act
