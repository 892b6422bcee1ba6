"""w4a16_moe at the ends of its range of sizes."""
import pytest

import moe_ref as ref
import tight
from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu


def test_a_million_tokens_of_wide_rows():
    """More than 2^34 results (2^32 groups of four, one a thread): a million tokens of which a few have an expert."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    T, H, I, G = 1000000, 17184, 32, 32
    assert T * H // 4 > 1 << 32
    if torch.cuda.get_device_properties(0).total_memory < 200 << 30:
        pytest.skip("needs 150 GB of memory")
    g = torch.Generator(device=dev()).manual_seed(4)
    gate, up, down = (ref.experts(g, 1, n, k, G, dev()) for n, k in ((I, H), (I, H), (H, I)))
    some = [0, 1, 77777, 999998, 999999]
    x = torch.empty((T, H), dtype=torch.bfloat16, device=dev())          # (rows without an expert are not read)
    x[some] = (torch.randn((len(some), H), generator=g, device=dev()) / H ** 0.5).to(torch.bfloat16)
    ids = torch.full((T, 1), -1, dtype=torch.int32, device=dev())
    ids[some] = 0
    weights = torch.rand((T, 1), generator=g, device=dev())
    y = w4.w4a16_moe(x, ids, weights, gate, up, down, G)
    want, bound = ref.moe(x[some], ids[some], weights[some], gate, up, down, "silu")
    assert ((y[some].double() - want).abs() <= bound).all() and y[some].any(1).all()
    y[some] = 0
    for i in range(0, T, 50000):
        assert not y[i:i + 50000].any(), i
    del x, y
    torch.cuda.empty_cache()


# many rows an expert: wider than the tiles' row sums may be (groups of 32 above 8192, of 64 above 16384) they are
# streamed, 32 rows at a time or, with few columns, 16; at those widths they are the tiles' own
@pytest.mark.parametrize("T,k,E,H,I,G", [(500, 2, 2, 64, 8224, 32), (700, 2, 4, 128, 14336, 32), (600, 1, 1, 64, 16448, 64),
                                         (300, 2, 2, 8224, 64, 32), (300, 2, 2, 16448, 64, 64), (400, 2, 2, 64, 8192, 32),
                                         (300, 2, 2, 8192, 64, 32), (400, 1, 1, 64, 16384, 64), (500, 2, 2, 128, 14336, 128)])
def test_many_rows_of_wide_experts(T, k, E, H, I, G):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    g = torch.Generator(device=dev()).manual_seed(I + H)
    gate, up, down = (ref.experts(g, E, n, kk, G, dev()) for n, kk in ((I, H), (I, H), (H, I)))
    x = (torch.randn((T, H), generator=g, device=dev()) / H ** 0.5).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g, device=dev())[:k] for _ in range(T)]).to(torch.int32)
    weights = torch.rand((T, k), generator=g, device=dev())
    first = w4.w4a16_moe(x, ids, weights, gate, up, down, G)
    left = w4.w4a16_moe(x, ids, weights, gate, up, down, G, residual=-first)
    want, bound = ref.moe(x, ids, weights, gate, up, down, "silu")
    assert ((first.double() - want).abs() <= bound).all()
    assert tight.tiled(T, k, E, H, I, G) == (max(H, I) <= {32: 8192, 64: 16384, 128: 1 << 20}[G])
    off = tight.moe_error(first, left, want)
    assert off <= tight.moe_limit(None, once=True), off


def test_rows_beyond_the_tiles_offsets():
    """65536 tokens with eight choices each, 4096 rows an expert: more than the tiles' 31-bit offsets reach."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    T, k, E, H, I, G = 65536, 8, 128, 2080, 64, 32
    assert not tight.tiled(T, k, E, H, I, G) and tight.tiled(T, k, E, 2016, I, G)
    g = torch.Generator(device=dev()).manual_seed(2)
    gate, up, down = (ref.experts(g, E, n, kk, G, dev()) for n, kk in ((I, H), (I, H), (H, I)))
    x = torch.randn((T, H), generator=g, device=dev()).to(torch.bfloat16)
    x *= H ** -0.5
    ids = torch.randint(0, E, (T, k), generator=g, device=dev(), dtype=torch.int32)
    weights = torch.rand((T, k), generator=g, device=dev())
    y = w4.w4a16_moe(x, ids, weights, gate, up, down, G)
    some = torch.tensor([0, 1, 4095, 32767, 32768, 50001, 65534, 65535], device=dev())
    want, bound = ref.moe(x[some], ids[some], weights[some], gate, up, down, "silu")
    assert ((y[some].double() - want).abs() <= bound).all()
    assert tight.rms(y[some].double() - want) <= 1.05 * 2 ** 0.5 * tight.STEP * tight.rms(want)
