"""Products of millions of short rows: every row is computed, as in a call with few."""
import pytest

import moe_ref as ref
from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,M,K", [("a8", (1 << 24) + 300, 64), ("a8", (1 << 24) + 300, 32), ("a16", (1 << 24) + 300, 64),
                                      ("a16", (1 << 23) + 300, 32), ("a8", (1 << 22) + 300, 12288)])
def test_many_rows(kind, M, K):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    if M * K > 1 << 34 and torch.cuda.get_device_properties(0).total_memory < 240 << 30:
        pytest.skip("needs 190 GB of memory")
    N, G = 16, 32
    g = torch.Generator(device=dev()).manual_seed(K)
    w = ref.experts(g, 1, N, K, G, dev())
    wq, sz = w["wq"][0], w["sz"][0]
    bias = torch.randn(N, generator=g, device=dev())
    rows = [0, 1, 255, 65535 * 128, 65535 * 128 + 1, M // 2, M - 300, M - 45, M - 44, M - 1]
    rows = [r for r in rows if r < M]
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=dev())
    some = (torch.randn((len(rows), K), generator=g, device=dev()) / K ** 0.5).to(torch.bfloat16)
    x[rows] = some
    if kind == "a8":
        y, xq, xs = w4.w4a8_linear(x, wq, sz, G, bias=bias)
        few, q, s = w4.w4a8_linear(some, wq, sz, G, bias=bias)
        assert torch.equal(xq[rows], q) and torch.equal(xs[rows], s)
        xd = q.view(torch.float8_e4m3fn).double() * s.double()[:, None]
    else:
        y, xd = w4.w4a16_linear(x, wq, sz, G, bias=bias), some.double()
    want = xd @ w["W"][0].T + bias.double()
    # sums of at most K terms in fp32, weights rounded to bf16, one rounding of the result
    bound = ref.BF16 * (want.abs() + xd.abs() @ w["W"][0].abs().T) + (K + 160) * ref.U * (xd.abs() @ w["size"][0].T) + 1e-6
    worst = ((y[rows].double() - want).abs() / bound).amax(1)
    assert (worst <= 1).all(), list(zip(rows, worst.tolist()))
    # rows of zeros leave the bias
    y[rows] = bias.to(torch.bfloat16)
    for i in range(0, M, 1 << 22):
        assert (y[i:i + (1 << 22)] == bias.to(torch.bfloat16)).all(), i
    del x, y
    torch.cuda.empty_cache()
