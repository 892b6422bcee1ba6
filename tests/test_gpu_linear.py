"""w4a16_linear and w4a8_linear on the GPU: every kernel that a product can run on, against its own product followed by
the epilogue in 64 bits, and against the whole formula in 64 bits."""
import pytest

import moe_ref as ref
from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu

ACTS = [None, "silu", "gelu_tanh", "relu", "gelu"]


def _act(x, act):
    import torch
    f = torch.nn.functional
    return {None: lambda: x, "silu": lambda: f.silu(x), "gelu_tanh": lambda: f.gelu(x, approximate="tanh"),
            "relu": lambda: f.relu(x), "gelu": lambda: f.gelu(x)}[act]()


def _inputs(M, K, N, G):
    import torch
    g = torch.Generator(device=dev()).manual_seed(M + K + N)
    w = ref.experts(g, 1, N, K, K if G == "row" else G, dev())
    x = (torch.randn((M, K), generator=g, device=dev()) / K ** 0.5).to(torch.bfloat16)
    return w, x, 0.5 * torch.randn(N, generator=g, device=dev()), torch.randn((M, N), generator=g, device=dev()).to(torch.bfloat16)


# (M, K, N, G): every kernel, whole and split along K
SHAPES = [
    (1, 576, 1000, 32), (1, 1024, 48, 128), (1, 256, 5, 64), (2, 512, 777, 128), (2, 16384, 130, 128), (1, 49152, 33, 128),
    (3, 576, 100, 32), (4, 2048, 4100, 128), (5, 8192, 300, 128), (16, 14336, 520, 128), (17, 1536, 576, 32),
    (32, 1024, 1000, 64), (30, 4096, 64, "row"),
    (33, 512, 130, 128), (40, 96, 300, 32), (48, 4096, 1000, 64), (64, 8192, 256, 128), (64, 3840, 1920, 32),
    (65, 256, 129, 128), (100, 4096, 512, 128), (128, 576, 130, 64), (97, 1024, 65, "row"),
    (129, 256, 300, 128), (200, 96, 250, 32), (256, 4096, 1000, 128), (300, 2048, 515, 64), (513, 1024, 1030, 128),
    (1056, 2048, 8200, 32),
]


@pytest.mark.parametrize("kind", ["a16", "a8"])
@pytest.mark.parametrize("M,K,N,G", SHAPES)
def test_linear(M, K, N, G, kind):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    w, x, bias, res = _inputs(M, K, N, G)
    g = K if G == "row" else G
    wq, sz = w["wq"][0], w["sz"][0]
    if kind == "a16":
        y, plain, xd = (lambda **kw: w4.w4a16_linear(x, wq, sz, g, **kw)), w4.w4a16_gemm(x, wq, sz, g), x.double()
    else:
        plain, xq, xs = w4.w4a8_gemm(x, wq, sz, g)
        xd = xq.view(torch.float8_e4m3fn).double() * xs.double()[:, None]

        def y(**kw):
            out, q, s = w4.w4a8_linear(x, wq, sz, g, **kw)
            assert torch.equal(q, xq) and torch.equal(s, xs)
            if K % 16 == 0:                   # (on the codes of the rows, the same; up to two rows another kernel's sums)
                same = w4.w4a8_linear_e4m3(xq, xs, wq, sz, g, **kw)
                assert M <= 2 or torch.equal(same, out)
                check(same, kw) if M <= 2 else None
            return out

        def check(out, kw):
            again = w4.w4a8_gemm_e4m3(xq, xs, wq, sz, g)
            assert torch.equal(again, w4.w4a8_linear_e4m3(xq, xs, wq, sz, g))
            left = w4.w4a8_linear_e4m3(xq, xs, wq, sz, g, residual=-again).double().abs()
            assert (left <= (ref.BF16 + 4 * ref.U) * again.double().abs() + 1e-37).all()
    # nothing to add: the product's own bits
    assert torch.equal(y(), plain) and torch.equal(y(act="none"), plain)
    # the whole formula.  The sums: at most K / 32 + 160 roundings in a chain, each of what passes through it (s (256 +
    # 2 |z|) |x| at most), and, with weights rounded to bf16 (groups below 128, tiles above 128 rows), 2^-8 of each
    exact = xd @ w["W"][0].T
    off = (K / 32 + 160) * ref.U * (xd.abs() @ w["size"][0].T) + 2.0 ** -8 * (xd.abs() @ w["W"][0].abs().T)
    for i, act in enumerate(ACTS):
        for b, r in (((bias, res), (None, None))[i % 2], (bias, None), (None, res)):
            if b is None and r is None and act is None:
                continue
            z = exact + (0 if b is None else b.double())
            want = _act(z, act) + (0 if r is None else r.double())
            # |act'| < 1.13; twelve roundings of at most |z| and the residual; the last one to bf16
            bound = 1.13 * off + 12 * ref.U * (z.abs() + want.abs() + (0 if r is None else r.double().abs()))
            bound = bound + ref.BF16 * (want.abs() + bound)
            got = y(bias=b, act=act, residual=r)
            worst = ((got.double() - want).abs() / bound.clamp(min=1e-30)).max().item()
            assert worst <= 1, (act, b is not None, r is not None, worst)
    # the epilogue by itself, on the sums that the product rounds: with a residual that is its negative, what is left
    # is the rounding of the product, half a step of bf16, and the roundings of the two sums
    left = y(residual=-plain).double().abs()
    assert (left <= (ref.BF16 + 4 * ref.U) * plain.double().abs() + 1e-37).all()


@pytest.mark.parametrize("M", [1, 8, 50, 100, 300])
@pytest.mark.parametrize("kind", ["a16", "a8"])
def test_linear_in_place_of_the_residual(M, kind):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    w, x, bias, res = _inputs(M, 4096, 384, 128)
    f = w4.w4a16_linear if kind == "a16" else (lambda *a, **kw: w4.w4a8_linear(*a, **kw)[0])
    want = f(x, w["wq"][0], w["sz"][0], 128, bias=bias, act="gelu", residual=res)
    assert f(x, w["wq"][0], w["sz"][0], 128, bias=bias, act="gelu", residual=res, Y=res) is res
    assert torch.equal(res, want)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_linear_without_workspace_and_special_values(M):
    """Infinite and NaN residuals and biases reach their own outputs only; activations at the ends of the range."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    w, x, bias, res = _inputs(M, 256, 200, 64)
    args = (x, w["wq"][0], w["sz"][0], 64)
    want = w4.w4a16_linear(*args, bias=bias, act="silu", residual=res)
    b2, r2 = bias.clone(), res.clone()
    b2[7], b2[9] = float("nan"), float("inf")
    r2[M - 1, 100] = float("-inf")
    got = w4.w4a16_linear(*args, bias=b2, act="silu", residual=r2)
    assert got[:, 7].isnan().all() and (got[:, 9] == float("inf")).all() and got[M - 1, 100] == float("-inf")
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[:, [7, 9]] = False
    keep[M - 1, 100] = False
    assert torch.equal(got[keep], want[keep])
    for big in (3e19, 1e25, 3e38):
        for act in ACTS[1:]:
            b2 = torch.full_like(bias, big)
            assert torch.equal(w4.w4a16_linear(*args, bias=b2, act=act), b2.to(torch.bfloat16).expand(M, -1))
            assert not w4.w4a16_linear(*args, bias=-b2, act=act).any()
