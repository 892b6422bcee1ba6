"""w4_tree_attention on values and scales of unusual size, in each of its forms: up to 16 and 32 rows a KV head, up
to 64, more, and heads of 256 dims."""
import numpy as np
import pytest

from helpers import dev, require_gpu
from test_gpu_decode import _attend, _f64

pytestmark = pytest.mark.gpu

# n nodes, hq, hk, d: rows a KV head n hq / hk
FORMS = [(6, 4, 2, 64), (6, 4, 2, 128), (12, 4, 2, 128), (12, 4, 2, 64), (25, 4, 2, 64), (25, 4, 2, 128), (45, 4, 2, 64),
         (70, 4, 2, 128), (12, 8, 2, 256)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("tree,window", [(True, 0), (False, 0), (False, 90), (True, 150)])
@pytest.mark.parametrize("past", [401, 424])   # the context ends in the first and in the second half of 64 tokens
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_infinities_and_nan_reach_the_rows_that_see_them(form, past, tree, window, e4m3):
    """Values of one token in two dims are infinite or NaN: these dims of the rows that see the token show it, and
    nothing else does, wherever the token lies beside the edges of what the rows see."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    n, hq, hk, d = form
    rng = np.random.default_rng(n + d + window)
    args, kw, want, tol = _attend(rng, [n], [past + n], hq, hk, d, 16, e4m3, tree, window)
    v_cache, table = args[2], args[3].cpu().numpy()[0]
    c = 16 if e4m3 else 8
    if tree:
        words = kw["tree"].cpu().numpy().view(np.uint64)
        bits = lambda i, j: bool(int(words[i, j // 64]) >> (j % 64) & 1)  # noqa: E731
    else:
        bits = lambda i, j: j <= i  # noqa: E731
    at = kw["positions"].cpu().numpy() if "positions" in kw else past + np.arange(n)
    position = lambda j: j if j < past else at[j - past]  # noqa: E731
    low = past - window if window else 0
    spots = {past - 1, past - 10, past - 20, past - 30, past - 45, past, past + n - 1, low + 1, low + 10, low + 30, low + 50,
             low + n, low + n + 20, low + n + 40}
    for j in sorted(s for s in spots if 0 <= s < past + n):
        sees = np.array([(j < past or bits(i, j - past)) and (not window or position(j) > at[i] - window) for i in range(n)])
        pg, blk, s = int(table[j // 16]), 0, j % 16
        for value in ((0x7F,) if e4m3 else (float("nan"), float("inf"), -float("inf"))):
            old = v_cache[pg, :, blk, s // c, :, s % c].clone()
            v_cache[pg, :, blk, s // c, 3, s % c] = value
            v_cache[pg, :, blk, s // c, d - 5, s % c] = value
            got = _f64(w4.w4_tree_attention(*args, **kw))
            v_cache[pg, :, blk, s // c, :, s % c] = old
            special = np.zeros((n, hq, d), bool)
            special[sees[:, None] & np.ones((1, hq), bool)] = np.isin(np.arange(d), (3, d - 5))
            assert np.max(np.abs(got - want)[~special] / tol[~special]) <= 1, (j, value)
            show = got[special]
            assert np.all(np.isnan(show) if e4m3 or value != value else show == value), (j, value)


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_no_token_is_seen_where_the_bound_is_zero(form):
    # lengths are cut to max_kv, to 0 too: rows that see nothing are zeros
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    n, hq, hk, d = form
    args, kw, _, _ = _attend(np.random.default_rng(n), [n, n], [n + 40, n], hq, hk, d, 16, False, False)
    out = torch.full((2 * n, hq, d), 7.0, dtype=torch.bfloat16, device=dev())
    args[7] = 0
    assert bool((w4.w4_tree_attention(*args, **kw, O=out) == 0).all())


@pytest.mark.parametrize("stride", [1, 515, 1025])
def test_a_single_row_has_any_stride(stride):
    """The stride of a dimension of one row is arbitrary (of a slice, say): it is neither used nor checked."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(stride)
    args, kw, want, tol = _attend(rng, [1], [300], 8, 2, 64, 16, False, False)
    odd = lambda x: x.as_strided(x.shape, (stride, x.stride(1), 1))  # noqa: E731
    args[0] = odd(args[0])
    assert np.max(np.abs(_f64(w4.w4_tree_attention(*args, **kw)) - want) / tol) <= 1
    q, k = torch.randn((1, 8, 64), device=dev()).to(torch.bfloat16), torch.randn((1, 2, 64), device=dev()).to(torch.bfloat16)
    slot = torch.tensor([5], dtype=torch.int32, device=dev())
    caches = [w4.w4_kv_cache(1, 2, 64, 16, device=dev()) for _ in range(2)]
    a = w4.w4_kv_append(q, k, k, slot, *caches[0])
    b = w4.w4_kv_append(odd(q), odd(k), odd(k), slot, *caches[1])
    assert torch.equal(a, b) and torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [-0.11, 0.0, 1.5])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_scales(form, scale, e4m3):
    """Negative (the smallest product has the largest weight), zero (the mean of what a row sees), far above 1/sqrt(d)."""
    require_gpu()
    import w4_dequant_gemm_amd as w4
    n, hq, hk, d = form
    for tree, window in ((True, 0), (False, 150)):
        args, kw, want, tol = _attend(np.random.default_rng(n + d), [n, n // 2], [n + 390, n // 2 + 7], hq, hk, d, 16, e4m3, tree, window, scale)
        got = _f64(w4.w4_tree_attention(*args, **kw))
        assert np.isfinite(got).all() and np.max(np.abs(got - want) / tol) <= 1, (tree, window)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [1e4, -1e4, 3e9, -3e9, 1e20, 1e30, -1e30])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_scores_far_apart(form, scale, e4m3):
    """Products of small whole numbers are exact, so with a large scale a row's result is the mean of the values of its
    largest products: equal weights for them and none for the others, whatever the size of the scores."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    n, hq, hk, d = form
    rng = np.random.default_rng(n + d)
    past = 20000 if n < 8 else 390           # (the first forms with the tokens split over workgroups)
    args, kw, _, _ = _attend(rng, [n], [past + n], hq, hk, d, 16, False, False)
    q = torch.from_numpy(rng.integers(-2, 3, (n, hq, d)).astype(np.float32)).to(torch.bfloat16).to(dev())
    # one KV head's keys and values [tokens, d] in the cache's places
    keys, values = (rng.integers(-2, 3, (hk, past + n, d)).astype(np.float32) for _ in range(2))
    c = 16 if e4m3 else 8
    table = args[3].cpu().numpy()[0].astype(np.int64)
    k_cache, v_cache = w4.w4_kv_cache(int(table.max()) + 1, hk, d, 16, device="cpu")
    if e4m3:
        k_cache, v_cache = (x.to(torch.float8_e4m3fn) for x in w4.w4_kv_cache(int(table.max()) + 1, hk, d, 16, e4m3=True, device="cpu"))
        kw.update(k_scale=torch.full((hk,), 0.5, device=dev()), v_scale=torch.ones(hk, device=dev()))
    t = np.arange(past + n)
    for h in range(hk):
        k_cache[table[t // 16], h, 0, :, t % 16] = torch.from_numpy(keys[h].reshape(-1, d // c, c)).to(k_cache.dtype)
        v_cache[table[t // 16], h, 0, t % 16 // c, :, t % c] = torch.from_numpy(values[h]).to(v_cache.dtype)
    args[:3] = q, *(x.view(torch.uint8 if e4m3 else x.dtype).to(dev()) for x in (k_cache, v_cache))
    kw["scale"] = scale
    got = _f64(w4.w4_tree_attention(*args, **kw))
    qn = _f64(q)
    for i in range(n):
        for h in range(hq):
            s = np.sign(scale) * (keys[h // (hq // hk), :past + i + 1].astype(np.float64) @ qn[i, h])
            want = values[h // (hq // hk), :past + i + 1][s == s.max()].astype(np.float64).mean(0)
            # one rounding to bf16, and the division's and the sums' to fp32
            assert np.all(np.abs(got[i, h] - want) <= 1.01 * 2.0 ** -8 * np.abs(want) + 2.0 ** -20), (i, h)
