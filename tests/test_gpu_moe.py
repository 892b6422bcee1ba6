"""w4_route and w4a16_moe on the GPU against references in 64 bits."""
import pytest

import moe_ref as ref
from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch
    return torch.Generator(device=dev()).manual_seed(seed)


def _layer(seed, T, k, E, H, I, G, zeros="asym"):
    import torch
    g = _gen(seed)
    gate, up, down = (ref.experts(g, E, n, kk, G, dev(), zeros) for n, kk in ((I, H), (I, H), (H, I)))
    x = (torch.randn((T, H), generator=g, device=dev()) / H ** 0.5).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g, device=dev())[:k] for _ in range(T)]).to(torch.int32)
    weights = torch.rand((T, k), generator=g, device=dev())
    res = torch.randn((T, H), generator=g, device=dev()).to(torch.bfloat16)
    return x, ids, weights, gate, up, down, res


def _check(got, want, bound, what):
    off = (got.double() - want).abs()
    worst = (off / bound).max().item()
    assert worst <= 1, f"{what}: {worst} of the bound"


@pytest.mark.parametrize("T,k,E,H,I,G", [
    (1, 2, 4, 64, 32, 32), (1, 8, 8, 256, 128, 128), (3, 1, 2, 128, 128, 64), (5, 4, 16, 576, 1536, 32),
    (7, 2, 4, 192, 320, 64), (16, 2, 4, 256, 384, 128), (17, 3, 5, 288, 96, 32), (33, 8, 40, 512, 256, 128),
    (40, 4, 4, 256, 256, 128), (70, 2, 3, 320, 192, 64), (129, 3, 7, 256, 640, 128), (300, 1, 1, 128, 128, 128),
    (500, 6, 16, 384, 256, 128), (2, 32, 32, 128, 128, 128), (1, 1, 1, 32, 32, 32), (64, 1, 64, 256, 128, 64),
    (16, 8, 40, 256, 256, 128), (9, 8, 16, 160, 224, 32), (2, 8, 64, 512, 320, 64), (1, 2, 4, 256, 14336, 128), (2, 4, 9, 8192, 96, 32),
    (32, 2, 70, 256, 128, 128),
    # 32 rows at a time (many columns), and 16 in turn or beside each other
    (52, 2, 8, 64, 4352, 32), (52, 2, 8, 64, 4352, 64), (52, 2, 8, 128, 4352, 128), (14, 4, 4, 64, 8320, 32),
    (40, 2, 8, 128, 4352, 128), (14, 4, 4, 96, 160, 32), (60, 2, 9, 256, 384, 128), (45, 3, 10, 288, 320, 32), (42, 2, 6, 320, 192, 64),
    # rows in tiles: ragged, one tile and several an expert, columns past the last tile's, long inner sums
    (100, 2, 4, 128, 128, 128), (200, 6, 16, 384, 640, 128), (700, 4, 32, 640, 256, 128), (90, 3, 3, 256, 4096, 128),
    (65, 1, 1, 4096, 256, 128), (1000, 8, 64, 256, 384, 128),
    (100, 2, 4, 64, 192, 64), (300, 4, 8, 320, 448, 64), (130, 1, 2, 576, 1536, 64), (200, 3, 5, 96, 160, 32),
    (90, 2, 2, 576, 1536, 32), (150, 2, 3, 288, 32, 32), (77, 1, 1, 2048, 4096, 32), (100, 2, 4, 128, 14336, 64),
])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_moe(T, k, E, H, I, G, act):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    x, ids, weights, gate, up, down, res = _layer(T + E, T, k, E, H, I, G)
    for r in (None, res):
        got = w4.w4a16_moe(x, ids, weights, gate, up, down, G, act, residual=r)
        want, bound = ref.moe(x, ids, weights, gate, up, down, act, r)
        torch.cuda.synchronize()
        _check(got, want, bound, f"residual {r is not None}")


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 9, 50])
def test_moe_far_zero_points(G, T):
    require_gpu()
    import w4_dequant_gemm_amd as w4
    x, ids, weights, gate, up, down, res = _layer(5, T, 2, 4, 256, 384, G, "far")
    got = w4.w4a16_moe(x, ids, weights, gate, up, down, G, residual=res)
    _check(got, *ref.moe(x, ids, weights, gate, up, down, "silu", res), "far zero points")


@pytest.mark.parametrize("T", [1, 2, 12, 40, 200])
def test_moe_choices_that_are_no_expert_or_come_twice(T):
    """Ids outside the experts add nothing, a token may choose an expert twice, and a token without any keeps its
    residual, bit for bit."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    E, H, I, G, k = 6, 256, 128, 64, 4
    x, ids, weights, gate, up, down, res = _layer(11, T, k, E, H, I, G)
    ids[:, 1] = ids[:, 0]                                    # twice
    ids[::2, 2] = torch.tensor([-1, E, 1 << 30, -(1 << 31)], dtype=torch.int32, device=dev()).repeat(T)[:(T + 1) // 2]
    ids[T // 2] = -1                                         # none at all
    got = w4.w4a16_moe(x, ids, weights, gate, up, down, G, residual=res)
    _check(got, *ref.moe(x, ids, weights, gate, up, down, "silu", res), "repeated and absent choices")
    assert torch.equal(got[T // 2], res[T // 2])
    got = w4.w4a16_moe(x, torch.full_like(ids, -1), weights, gate, up, down, G)
    assert not got.any()


@pytest.mark.parametrize("T,E", [(20, 3), (150, 3)])
def test_moe_one_expert_has_all_the_tokens(T, E):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    x, ids, weights, gate, up, down, res = _layer(3, T, 1, E, 256, 256, 128)
    ids[:] = E - 1
    got = w4.w4a16_moe(x, ids, weights, gate, up, down, 128, residual=res)
    _check(got, *ref.moe(x, ids, weights, gate, up, down, "silu", res), "one expert")
    # in place of its residual
    again = res.clone()
    assert w4.w4a16_moe(x, ids, weights, gate, up, down, 128, residual=again, Y=again) is again
    assert torch.equal(again, got)


@pytest.mark.parametrize("T", [3, 30, 300])
def test_moe_rows_do_not_reach_each_other(T):
    """An infinity or NaN in one token leaves the others' results as they are, and unused experts' weights (scales of
    NaN) reach nothing."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    x, ids, weights, gate, up, down, res = _layer(8, T, 2, 5, 256, 128, 128)
    ids = ids % 4                                            # expert 4 is never chosen
    want = w4.w4a16_moe(x, ids, weights, gate, up, down, 128, residual=res)
    for w in (gate, up, down):
        w["sz"][4] = 0x7E007E00                              # NaN scale and zero point
    x2 = x.clone()
    x2[1, 5], x2[1, 77] = float("inf"), float("nan")
    got = w4.w4a16_moe(x2, ids, weights, gate, up, down, 128, residual=res)
    keep = torch.arange(T, device=dev()) != 1
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[1].float()).any()


def test_moe_large_and_small_values():
    """h beyond bf16's range of small numbers, and results that are infinite in bf16."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    x, ids, weights, gate, up, down, _ = _layer(21, 4, 2, 4, 128, 128, 128)
    for scale in (1e-20, 1e-3, 1e3, 1e9):
        xs = (x.float() * scale).to(torch.bfloat16)
        got = w4.w4a16_moe(xs, ids, weights, gate, up, down, 128)
        want, bound = ref.moe(xs, ids, weights, gate, up, down, "silu")
        _check(got, want, bound + 2.0 ** -120, f"scale {scale}")


@pytest.mark.parametrize("T,H,E,k", [(1, 8, 1, 1), (1, 64, 8, 2), (3, 72, 5, 5), (16, 256, 64, 8), (17, 1000, 65, 3),
                                     (50, 2048, 128, 8), (200, 576, 130, 32), (5, 4096, 256, 6), (9, 128, 1000, 4),
                                     (1, 7168, 1024, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(T, H, E, k, score):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    g = _gen(T + H + E)
    x = torch.randn((T, H), generator=g, device=dev()).to(torch.bfloat16)
    r = (2 / H ** 0.5 * torch.randn((E, H), generator=g, device=dev())).to(torch.bfloat16)
    bias = 0.1 * torch.randn(E, generator=g, device=dev())
    for b in (None, bias):
        for renorm, scale in ((True, 1.0), (False, 2.5)):
            ids, weights = w4.w4_route(x, r, k, score=score, bias=b, renormalize=renorm, scale=scale)
            want, w64, dl, sure = ref.route(x, r, k, score, b, renorm, scale)
            torch.cuda.synchronize()
            assert ids.dtype == torch.int32 and ids.min() >= 0 and ids.max() < E
            assert all(len(set(row)) == k for row in ids.tolist())
            assert sure.double().mean() >= 0.25                # (enough places have one answer)
            assert torch.equal(ids.long()[sure], want[sure])
            # a weight moves by at most 2 dl of itself, divided by a sum that does by 4 dl; its own roundings
            tol = (4 * dl + (64 + E) * ref.U) * w64
            whole = sure.all(1)
            assert ((weights.double() - w64).abs() <= tol)[whole].all()


def test_route_ties_and_what_is_no_number():
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    E, H, k = 70, 64, 5
    x = torch.ones((3, H), device=dev()).to(torch.bfloat16)
    r = torch.zeros((E, H), device=dev()).to(torch.bfloat16)
    r[[3, 66, 10, 40]] = 1.0                                 # four even logits, then zeros
    ids, weights = w4.w4_route(x, r, k)
    assert ids.tolist() == [[3, 10, 40, 66, 0]] * 3
    assert torch.allclose(weights[:, :4], weights[:, :1].expand(3, 4))
    r[10] = float("nan")
    r[40] = float("inf")
    ids, weights = w4.w4_route(x, r, k)
    assert ids.tolist() == [[40, 3, 66, 0, 1]] * 3           # NaN counts as -inf
    assert weights.tolist() == [[1.0, 0, 0, 0, 0]] * 3
    x[1] = float("nan")                                      # nothing but NaN: the lowest indexes, no weight
    ids, weights = w4.w4_route(x, r, k)
    assert ids[1].tolist() == [0, 1, 2, 3, 4] and not weights[1].any()
    assert ids[0].tolist() == [40, 3, 66, 0, 1]


def test_route_then_moe_as_a_layer():
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    x, _, _, gate, up, down, res = _layer(2, 21, 2, 8, 256, 128, 64)
    g = _gen(9)
    r = (8 * torch.randn((8, 256), generator=g, device=dev())).to(torch.bfloat16)
    ids, weights = w4.w4_route(x, r, 3, score="sigmoid")
    got = w4.w4a16_moe(x, ids, weights, gate, up, down, 64, residual=res)
    _check(got, *ref.moe(x, ids, weights, gate, up, down, "silu", res), "layer")
