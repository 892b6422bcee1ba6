"""w4_sample on numbers of unusual size: what is kept and drawn follows from whole numbers alone, so tokens are equal
to the reference's, on every path of the kernel and in both types."""
import numpy as np
import pytest

from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu


def _full(n, x):
    import torch
    return torch.full((n,), x, device=dev())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [50, 5003, 60000])
def test_infinite_logits_share_everything(V, f32):
    # whatever the temperature, an infinite one included: of n infinite logits the kept ones have equal weights
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(V)
    B, n = 16, 11
    x = torch.randn((B, V), device=dev())
    x[:, 3] = -float("inf")
    at = np.stack([np.sort(rng.choice(np.arange(4, V), n, replace=False)) for _ in range(B)])
    x.scatter_(1, torch.from_numpy(at).to(dev()), float("inf"))
    x = x if f32 else x.to(torch.bfloat16)
    u = rng.random(B).astype(np.float32)
    units = np.floor(u.astype(np.float64) * 2 ** 24).astype(np.int64)
    uu = torch.from_numpy(u).to(dev())
    k = torch.full((B,), 4, dtype=torch.int32, device=dev())
    for t in (0.5, 1.0, 2e37, float("inf")):
        for kept, kw in ((n, {}), (6, {"top_p": _full(B, 0.5)}), (4, {"top_k": k}), (2, {"top_k": k, "top_p": _full(B, 0.5)}),
                         (n, {"min_p": _full(B, 0.25)}), (6, {"top_p": _full(B, 0.5), "min_p": _full(B, 1.0)})):
            tokens, probs = w4.w4_sample(x, uu, temperature=_full(B, t), **kw)
            assert np.array_equal(tokens.cpu().numpy(), at[np.arange(B), units * kept >> 24]), (t, kept)
            assert np.all(np.abs(probs.cpu().numpy() - 1 / kept) <= 2.0 ** -24), (t, kept)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V,tail", [(1500, 600), (50000, 600), (50000, 5000)])
@pytest.mark.parametrize("min_p,x,t", [(9e-10, -21.0, 1.0), (2.3e-9, -19.875, 19.875 / 19.95)])
def test_small_min_p_keeps_weights_that_round_up(V, tail, f32, min_p, x, t):
    # weights are whole numbers: one of 1.63 is 2 and passes a threshold of 1.93, which is 2 too
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(V + tail)
    logits = np.full(V, -400.0)
    logits[0] = 0.0
    at = np.sort(rng.choice(np.arange(1, V), tail, replace=False))
    logits[at] = x
    real = 2.0 ** 31 * np.exp(x / np.float32(t))
    least = int(np.ceil(np.float32(min_p) * 2.0 ** 31))
    weight = int(np.rint(real))
    assert real < np.float32(min_p) * 2.0 ** 31 and weight >= least and abs(abs(real - weight) - 0.5) > 0.05
    total = 2 ** 31 + weight * tail
    units = 2 ** 24 - 1 - np.arange(12)
    upto = np.concatenate([[2 ** 31], 2 ** 31 + weight * np.arange(1, tail + 1)])
    want = np.concatenate([[0], at])[np.searchsorted(upto, units * total >> 24, side="right")]
    assert np.count_nonzero(want) >= 3
    B = len(units)
    row = torch.from_numpy(logits.astype(np.float32)).to(torch.float32 if f32 else torch.bfloat16).to(dev())
    u = torch.from_numpy((units / 2.0 ** 24).astype(np.float32)).to(dev())
    many = torch.full((B,), tail + 100, dtype=torch.int32, device=dev())
    for kw in ({}, {"top_k": many}):
        tokens, probs = w4.w4_sample(row.expand(B, V), u, temperature=_full(B, t), min_p=_full(B, min_p), **kw)
        assert np.array_equal(tokens.cpu().numpy(), want), kw
        share = np.where(want == 0, 2.0 ** 31, weight) / total
        assert np.all(np.abs(probs.cpu().numpy() - share) <= 2.0 ** -23 * share), kw


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [40, 5003, 20000, 131072])
def test_signalling_nan_count_as_nothing(V, f32):
    # bit patterns of memory nobody wrote (a padded vocabulary): like -inf, wherever they stand beside the maximum
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(V)
    B = 24
    x = torch.randn((B, V), device=dev())
    for r in range(B):
        x[r, r % V] = 6.0 + r / 8            # the maximum, in every place of a vector
    bits = x.view(torch.int32) if f32 else (x := x.to(torch.bfloat16)).view(torch.int16)
    patterns = [0x7F800001, 0x7FBFFFFF, -0x7FFFFF, -0x400001] if f32 else [0x7F81, 0x7FBF, -0x7F, -0x41]
    spots = [s for s in range(0, V, 3)] + [s for s in range(V // 2, V)]
    clean = x.clone()
    for i, p in enumerate(patterns):
        at = torch.tensor(spots[i::4], device=dev())
        keep = bits[torch.arange(B), torch.arange(B) % V].clone()
        bits[:, at] = p
        clean[:, at] = -float("inf")
        bits[torch.arange(B), torch.arange(B) % V] = keep
        clean[torch.arange(B), torch.arange(B) % V] = x[torch.arange(B), torch.arange(B) % V]
    assert bool(x.isnan().any())
    u = torch.from_numpy(rng.random(B).astype(np.float32)).to(dev())
    k = torch.full((B,), 7, dtype=torch.int32, device=dev())
    tokens, _ = w4.w4_sample(x, u, temperature=_full(B, 0.0))
    assert tokens.tolist() == [r % V for r in range(B)]
    for kw in ({}, {"top_k": k}, {"top_p": _full(B, 0.8)}, {"min_p": _full(B, 0.05)}, {"top_k": k, "top_p": _full(B, 0.6)}):
        got, want = w4.w4_sample(x, u, **kw), w4.w4_sample(clean, u, **kw)
        for a, b in zip(got, want):
            assert torch.equal(a, b), kw
