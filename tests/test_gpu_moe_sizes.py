"""w4a16_moe at the ends of its range of sizes."""
import pytest

import moe_ref as ref
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
