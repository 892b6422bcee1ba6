"""The decoding calls on the GPU against 64-bit references (``decode_ref``):
appending to the paged cache, attention over it, token choice, moving a path."""
import numpy as np
import pytest

import decode_ref as ref
from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev())


def _bf16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).to(dev())


def _f32(a):
    import torch
    return torch.tensor(np.asarray(a, np.float32), device=dev())


def _f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ append

APPEND = [
    # T, hq, hk, d, rot, page, e4m3, norm, interleaved
    (1, 9, 3, 64, 64, 16, False, False, False),
    (5, 9, 3, 64, 32, 16, True, True, False),
    (37, 8, 2, 128, 128, 48, False, True, True),
    (70, 28, 4, 128, 64, 64, True, False, True),
    (33, 4, 2, 256, 256, 32, False, True, False),
    (20, 8, 1, 256, 16, 1024, True, True, True),
    (130, 2, 2, 64, 0, 128, False, False, False),
]


@pytest.mark.parametrize("case", APPEND, ids=str)
@pytest.mark.parametrize("fused", [True, False])
def test_append(case, fused):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    T, hq, hk, d, rot, page, e4m3, norm, interleaved = case
    rng = np.random.default_rng(T + d)
    pages, _ = ref.page_table(rng, [T + 9], page)
    k_cache, v_cache = ref.random_cache(rng, pages, hk, d, page, e4m3, dev())
    before = [x.clone() for x in (k_cache, v_cache)]
    qkv = _bf16(rng.standard_normal((T, hq + 2 * hk, d)))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    if not fused:                            # rows of their own, the values' further apart
        q, k = q.contiguous(), k.contiguous()
        wide = torch.zeros((T, hk * d + 24), dtype=torch.bfloat16, device=dev())
        wide[:, :hk * d] = v.reshape(T, -1)
        v = wide[:, :hk * d].unflatten(1, (hk, d))
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    if T > 3:
        slots[1], slots[3] = -1, pages * page          # padding, and a slot behind the cache
    kw = {}
    rope = positions = nq = nk = None
    if rot:
        rope, positions = ref.rope_table(T + 40, rot), rng.integers(0, T + 40, T)
        kw.update(rope=torch.from_numpy(rope).to(dev()), positions=_i32(positions), interleaved=interleaved)
    if norm:
        nq, nk = (1 + 0.3 * rng.standard_normal(d) for _ in range(2))
        nq, nk = nq.astype(np.float32), nk.astype(np.float32)
        kw.update(q_norm=torch.from_numpy(nq).to(dev()), k_norm=torch.from_numpy(nk).to(dev()), eps=1e-5)
    ks = vs = np.ones(hk, np.float32)
    if e4m3:
        ks, vs = (rng.uniform(0.003, 0.05, hk).astype(np.float32) for _ in range(2))
        kw.update(k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev()))
    Q = w4.w4_kv_append(q, k, v, _i32(slots), k_cache, v_cache, **kw)
    want, err = ref.head_rows(_f64(q), nq, 1e-5, rope, positions, rot, interleaved)
    # one rounding to bf16: 2^-8 of the value at most (8 bits of significand, nearest)
    assert np.all(np.abs(_f64(Q) - want) <= 1.001 * (2.0 ** -8 * np.abs(want) + err) + 1e-38)
    kw64, kerr = ref.head_rows(_f64(k), nk, 1e-5, rope, positions, rot, interleaved)
    gk, gv = ref.to_tokens(k_cache, v_cache)
    ok, ov = ref.to_tokens(*before)
    stored = (slots >= 0) & (slots < pages * page)
    for got, old, want, err, s in ((gk, ok, kw64, kerr, ks), (gv, ov, _f64(v), 0 * kerr, vs)):
        untouched = np.ones(pages * page, bool)
        untouched[slots[stored]] = False
        assert np.array_equal(got[untouched], old[untouched], equal_nan=True)
        want, err, got = want[stored], err[stored], got[slots[stored]]
        if e4m3:
            # half a unit of E4M3 (4 bits; subnormal step 2^-9), saturating
            want, err = np.clip(want / s[:, None], -448, 448), err / s[:, None]
            assert np.all(np.abs(got - want) <= 1.001 * (np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 1.2 * err + 2.0 ** -23 * np.abs(want)))
        else:
            assert np.all(np.abs(got - want) <= 1.001 * (2.0 ** -8 * np.abs(want) + err) + 1e-38)


def test_append_in_place_without_queries_and_outside_the_table():
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(3)
    T, hq, hk, d, page = 6, 4, 2, 64, 16
    q, k, v = (_bf16(rng.standard_normal((T, h, d))) for h in (hq, hk, hk))
    rope = torch.from_numpy(ref.rope_table(50, d)).to(dev())
    caches = [w4.w4_kv_cache(3, hk, d, page, device=dev()) for _ in range(3)]
    slots, pos = _i32([0, 17, 30, 2, 47, 9]), _i32([0, 49, 3, 7, 50, -1])
    Q = w4.w4_kv_append(q, k, v, slots, *caches[0], rope=rope, positions=pos)
    # positions 50 and -1 lie outside the table: NaN, and only there
    assert torch.isnan(Q[4:]).all() and not torch.isnan(Q[:4]).any()
    q2 = q.clone()
    assert w4.w4_kv_append(q2, k, v, slots, *caches[1], rope=rope, positions=pos, Q=q2) is q2
    assert torch.equal(q2.view(torch.int16), Q.view(torch.int16))
    assert w4.w4_kv_append(None, k, v, slots, *caches[2], rope=rope, positions=pos) is None
    for c in caches[1:]:
        for a, b in zip(c, caches[0]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # nothing to append, and NaN through an E4M3 cache
    empty = torch.empty((0, hk, d), dtype=torch.bfloat16, device=dev())
    w4.w4_kv_append(None, empty, empty, _i32([]), *caches[2])
    c8 = w4.w4_kv_cache(1, hk, d, page, e4m3=True, device=dev())
    one = torch.ones(hk, device=dev())
    k[0, 0, 0], v[0, 1, 5], v[1, 0, 0], k[1, 1, 1] = float("nan"), float("nan"), float("inf"), -1e30
    w4.w4_kv_append(None, k[:2], v[:2], _i32([3, 4]), *c8, k_scale=one, v_scale=one)
    kt, vt = ref.to_tokens(*c8)
    assert np.isnan(kt[3, 0, 0]) and np.isnan(vt[3, 1, 5]) and vt[4, 0, 0] == 448 and kt[4, 1, 1] == -448
    assert np.isnan(kt).sum() == 1 and np.isnan(vt).sum() == 1


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hk,d", [(3, 64), (2, 128), (1, 256)])
def test_append_runs_of_slots(hk, d, e4m3):
    """Slots in runs that begin and end inside a block, inside 8 and 16 tokens of it, and at the tokens the kernel
    takes together; a prompt's padding between; runs backwards.  The cache is what storing token by token gives."""
    require_gpu()
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(d)
    page, pages = 48, 14
    slots = np.concatenate([np.arange(5, 42), [-1, -1], np.arange(200, 216), np.arange(112, 96, -1), [pages * page + 3],
                            np.arange(311, 343), [64, 65, 67, 68], np.arange(500, 507), [-5], np.arange(508, 531)]).astype(np.int32)
    T = len(slots)
    assert len(set(slots[slots >= 0])) == np.sum(slots >= 0)
    k, v = (_bf16(rng.standard_normal((T, hk, d))) for _ in range(2))
    scales = {"k_scale": _f32(np.full(hk, 0.01)), "v_scale": _f32(np.full(hk, 0.01))} if e4m3 else {}
    start = ref.random_cache(rng, pages, hk, d, page, e4m3, dev())
    got, want = [x.clone() for x in start], [x.clone() for x in start]
    w4.w4_kv_append(None, k, v, _i32(slots), *got, **scales)
    for t in range(T):
        w4.w4_kv_append(None, k[t:t + 1], v[t:t + 1], _i32(slots[t:t + 1]), *want, **scales)
    for a, b, c in zip(got, want, start):
        assert np.array_equal(_f64(a), _f64(b))
        assert not np.array_equal(_f64(a), _f64(c))
    gv = ref.to_tokens(*got)[1]
    stored = (slots >= 0) & (slots < pages * page)
    x = _f64(v)[stored]
    assert np.all(np.abs(gv[slots[stored]] * (np.float32(0.01) if e4m3 else 1) - x) <= (0.01 * np.maximum(2.0 ** -4 * np.abs(x) / 0.01, 2.0 ** -10) * 1.001 if e4m3 else 0))


# --------------------------------------------------------------- attention

def _attend(rng, nodes, lengths, hq, hk, d, page, e4m3, tree, window=0, scale=None, poison=True, out=None):
    """A random call; returns its arguments and the references of every row."""
    import torch
    pages, table = ref.page_table(rng, lengths, page)
    k_cache, v_cache = ref.random_cache(rng, pages, hk, d, page, e4m3, dev())
    ks = vs = np.ones(hk, np.float32)
    kw = {"window": window, "scale": scale}
    if e4m3:
        ks, vs = (rng.uniform(0.01, 0.04, hk).astype(np.float32) for _ in range(2))
        kw.update(k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev()))
    T = sum(nodes)
    q = _bf16(1.5 * rng.standard_normal((T, hq, d)))
    start = np.concatenate([[0], np.cumsum(nodes)])
    kt, vt = ref.to_tokens(k_cache, v_cache)
    kt, vt = kt * ks[:, None].astype(np.float64), vt * vs[:, None].astype(np.float64)
    sees, want, tol, positions = [], np.zeros((T, hq, d)), np.zeros((T, hq, d)), []
    used = np.zeros(pages * page, bool)
    for b, (n, length) in enumerate(zip(nodes, lengths)):
        s, depth = ref.random_tree(rng, n)
        if not tree:
            depth = list(range(n))
        sees += s
        pos = [length - n + x for x in depth]
        positions += pos
        at = table[b][np.arange(length) // page].astype(np.int64) * page + np.arange(length) % page
        used[at] = True
        w, t = ref.attention(_f64(q)[start[b]:start[b + 1]], kt[at], vt[at], length - n,
                             scale if scale is not None else d ** -0.5, s if tree else None, pos, window)
        want[start[b]:start[b + 1]], tol[start[b]:start[b + 1]] = w, t
    if poison:                               # what no sequence holds is NaN
        slots = torch.from_numpy(np.flatnonzero(~used)).to(dev())
        c = 16 if e4m3 else 8
        pg, blk, s = slots // page, slots % page // 16, slots % 16
        bad = 0x7F if e4m3 else float("nan")
        k_cache[pg, :, blk, :, s] = bad
        v_cache[pg, :, blk, s // c, :, s % c] = bad
    if tree:
        kw["tree"] = ref.pack_tree(sees, -(-max(nodes) // 64)).to(dev())
    if window and tree:
        kw["positions"] = _i32(positions)
    args = [q, k_cache, v_cache, _i32(table), _i32(lengths), _i32(start), max(nodes), max(lengths)]
    return args, kw, want, tol


ATTEND = [
    # nodes, lengths, hq, hk, d, page, e4m3, tree, window
    ([1], [1], 9, 3, 64, 16, False, False, 0),
    ([1], [517], 9, 3, 64, 16, False, False, 0),
    ([1, 1, 1], [64, 65, 2000], 32, 8, 128, 64, False, False, 0),
    ([1, 1], [33, 3001], 8, 1, 128, 48, True, False, 0),
    ([1, 1], [31, 700], 16, 8, 256, 32, False, False, 0),
    ([1], [1500], 8, 4, 256, 256, True, False, 0),
    ([7, 3, 1], [400, 3, 90], 9, 3, 64, 16, False, True, 0),
    ([12, 9], [300, 801], 28, 4, 128, 128, True, True, 0),
    ([60, 41, 1], [700, 41, 333], 16, 2, 128, 64, False, True, 0),
    ([130, 67], [600, 200], 4, 2, 64, 16, True, True, 0),
    ([17, 5], [900, 333], 16, 8, 256, 32, True, True, 100),
    ([20, 11], [500, 1100], 8, 2, 128, 64, False, True, 64),
    ([77], [200], 12, 12, 128, 48, False, False, 0),
    ([100, 5], [777, 5], 8, 2, 64, 16, True, False, 33),
    ([90, 33], [420, 33], 8, 4, 256, 16, False, False, 0),
    ([150], [150], 6, 1, 128, 32, False, False, 40),
    ([2, 2, 2, 2, 2], [2, 18, 34, 259, 515], 4, 4, 128, 16, False, True, 0),
    # windows that part a tree's nodes, and a chain's
    ([30, 9], [300, 9], 8, 2, 64, 16, False, True, 3),
    ([17, 5], [900, 20], 16, 8, 256, 32, True, True, 4),
    ([60, 2], [500, 70], 4, 2, 128, 64, True, True, 2),
    ([70], [70], 8, 4, 128, 16, True, False, 1),
    ([9], [600], 4, 2, 64, 32, True, True, 2),
    # 17 to 32 rows a KV head, and 33 to 64
    ([5, 4], [77, 1040], 20, 5, 64, 16, True, False, 0),
    ([8], [600], 16, 4, 128, 64, True, True, 0),
    ([12, 1], [700, 1], 8, 2, 64, 16, False, True, 0),
    ([16, 9], [1300, 9], 16, 4, 128, 32, True, True, 0),
    ([40, 33], [200, 97], 2, 2, 64, 1024, True, True, 0),
    ([33], [2500], 1, 1, 128, 128, False, False, 0),
    ([12, 7], [1500, 40], 16, 4, 128, 16, False, False, 50),
]


@pytest.mark.parametrize("case", ATTEND, ids=str)
def test_attention(case):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    nodes, lengths, hq, hk, d, page, e4m3, tree, window = case
    args, kw, want, tol = _attend(np.random.default_rng(sum(lengths) + d), *case[:8], window)
    print("[attention]", case, flush=True)
    O = w4.w4_tree_attention(*args, **kw)
    worst = np.max(np.abs(_f64(O) - want) / tol)
    assert np.isfinite(_f64(O)).all() and worst <= 1, worst
    # bounds above the true sizes change the launch, not what is computed; a workspace's contents do not matter
    args[6], args[7] = sum(nodes), args[3].shape[1] * page
    ws = torch.full((max(4, w4.w4_tree_attention_workspace_bytes(sum(nodes), len(nodes), hq, hk, d, e4m3, args[6], args[7], window) // 4),),
                    float("nan"), device=dev())
    if kw.get("tree") is not None:
        wide = torch.zeros((sum(nodes), -(-sum(nodes) // 64)), dtype=torch.int64, device=dev())
        wide[:, :kw["tree"].shape[1]] = kw["tree"]
        kw["tree"] = wide
    O2 = w4.w4_tree_attention(*args, **kw, workspace=ws)
    assert np.max(np.abs(_f64(O2) - want) / tol) <= 1
    # the same call gives the same bits
    assert torch.equal(O2.view(torch.int16), w4.w4_tree_attention(*args, **kw, workspace=ws).view(torch.int16))


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_long_context_split(e4m3):
    # tokens split over many workgroups, against the float64 products of torch
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(5)
    n, length, hq, hk, d, page = 3, 40009, 8, 2, 128, 64
    pages, table = ref.page_table(rng, [length], page)
    k_cache, v_cache = ref.random_cache(rng, pages, hk, d, page, e4m3, dev())
    scales = {"k_scale": torch.full((hk,), 0.02, device=dev()), "v_scale": torch.full((hk,), 0.03, device=dev())} if e4m3 else {}
    q = _bf16(2 * rng.standard_normal((n, hq, d)))
    O = w4.w4_tree_attention(q, k_cache, v_cache, _i32(table), _i32([length]), _i32([0, n]), n, length, **scales)
    kt, vt = ref.to_tokens(k_cache, v_cache)
    at = table[0][np.arange(length) // page].astype(np.int64) * page + np.arange(length) % page
    kt, vt = kt[at] * (0.02 if e4m3 else 1), vt[at] * (0.03 if e4m3 else 1)
    for i in range(n):
        m = length - n + i + 1
        for h in range(hq):
            k, v = kt[:m, h // 4], vt[:m, h // 4]
            x = _f64(q)[i, h]
            s = k @ x * d ** -0.5
            p = np.exp(s - s.max())
            o, big = p @ v / p.sum(), p @ np.abs(v) / p.sum()
            spread = (d + 2) * 2.0 ** -24 * np.max(np.abs(k) @ np.abs(x)) * d ** -0.5 + 2.0 ** -21
            tol = 2.0 ** -8 * np.abs(o) + big * (2.0 ** -8 + 2 * spread + 2 * m * 2.0 ** -24)
            assert np.all(np.abs(_f64(O)[i, h] - o) <= 1.02 * tol)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [64, 100])
def test_attention_long_context_of_many_heads(n, e4m3):
    # 150000 tokens in few splits: more of them than a workgroup looks up at a time; three heads checked on the device
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    length, hk, d, page = 150001, 64, 64, 64
    pages = -(-length // page)
    gen = torch.Generator(device=dev()).manual_seed(n)
    k_cache, v_cache = w4.w4_kv_cache(pages, hk, d, page, e4m3=e4m3, device=dev())
    for x in (k_cache, v_cache):
        for part in x.split(256):            # (a piece of the normal numbers at a time)
            r = torch.randn(part.shape, generator=gen, device=dev())
            part.copy_((40 * r).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else r)
    scales = {"k_scale": _f32(np.full(hk, 0.02)), "v_scale": _f32(np.full(hk, 0.03))} if e4m3 else {}
    table = torch.randperm(pages, generator=gen, device=dev()).to(torch.int32)
    q = torch.randn((n, hk, d), generator=gen, device=dev()).to(torch.bfloat16)
    O = w4.w4_tree_attention(q, k_cache, v_cache, table[None].contiguous(), _i32([length]), _i32([0, n]), n, length, **scales)
    mask = torch.arange(length, device=dev())[None] > length - n + torch.arange(n, device=dev())[:, None]
    for h in (0, 31, 63):
        def tokens(x, order):
            x = x[table.long(), h].contiguous()
            x = (x.view(torch.float8_e4m3fn) if e4m3 else x).double()
            return x.permute(order).reshape(pages * page, d)[:length]
        kt = tokens(k_cache, (0, 1, 3, 2, 4)) * (float(np.float32(0.02)) if e4m3 else 1)
        vt = tokens(v_cache, (0, 1, 2, 4, 3)) * (float(np.float32(0.03)) if e4m3 else 1)
        x = q[:, h].double()
        p = (x @ kt.T * d ** -0.5).masked_fill(mask, -float("inf")).softmax(1)
        o, big = p @ vt, p @ vt.abs()
        spread = (d + 2) * 2.0 ** -24 * (x.abs() @ kt.abs().T).amax(1, keepdim=True) * d ** -0.5 + 2.0 ** -21
        tol = 2.0 ** -8 * o.abs() + big * (2.0 ** -8 + 2 * spread + 2 * length * 2.0 ** -24)
        assert bool(((O[:, h].double() - o).abs() <= 1.02 * tol).all())


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_past_32_bits(e4m3):
    """Append, attention and move at the end of a cache whose arrays pass 2^32 elements and bytes."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    hk, hq, d, page, n = 8, 16, 128, 64, 5
    pages = 2 ** 32 // (hk * d * page) + 9
    k_cache, v_cache = w4.w4_kv_cache(pages, hk, d, page, e4m3=e4m3, device=dev())
    scales = {"k_scale": _f32(np.full(hk, 0.02)), "v_scale": _f32(np.full(hk, 0.02))} if e4m3 else {}
    rng = np.random.default_rng(1)
    length = 2 * page + 20
    table = np.array([[pages - 1, pages - 7, pages - 3]], np.int32)
    small = w4.w4_kv_cache(3, hk, d, page, e4m3=e4m3, device=dev())
    near = np.array([[0, 1, 2]], np.int32)
    q, k, v = (_bf16(rng.standard_normal((length, h, d))) for h in (hq, hk, hk))
    at = np.arange(length)
    out = []
    for cache, t in (((k_cache, v_cache), table), (small, near)):
        slots = t[0][at // page] * page + at % page
        w4.w4_kv_append(None, k, v, _i32(slots), *cache, **scales)
        first = w4.w4_tree_attention(q[-n:], *cache, _i32(t), _i32([length]), _i32([0, n]), n, length, **scales)
        many = w4.w4_tree_attention(q[-40:], *cache, _i32(t), _i32([length]), _i32([0, 40]), 40, length, **scales)
        w4.w4_kv_move(*cache, _i32(t), _i32([length - n]), _i32([[1, 3, 4]]), _i32([3]))
        out.append((first, many, [x[torch.from_numpy(t[0]).long().to(dev())] for x in cache]))
    (a, b, c), (x, y, z) = out
    assert torch.equal(a.view(torch.int16), x.view(torch.int16)) and torch.equal(b.view(torch.int16), y.view(torch.int16))
    assert float(a.float().abs().max()) > 0
    for l, r in zip(c, z):
        assert torch.equal(l, r) and bool((l != 0).any())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_unseen_infinities_and_nan(e4m3, d):
    """A node's own key and value are NaN or infinite: only the nodes that see it may show it."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(d)
    for n, length, hq in ((6, 75, 4), (40, 400, 8), (6, 75, 8), (12, 130, 8)):
        args, kw, want, tol = _attend(rng, [n], [length], hq, 2, d, 16, e4m3, True)
        q, k_cache, v_cache, table = args[:4]
        bad = n - 2
        words = kw["tree"].cpu().numpy().view(np.uint64)
        sees = np.array([bool(int(words[i, bad // 64]) >> (bad % 64) & 1) for i in range(n)])
        j = length - n + bad
        slot = int(table[0, j // 16]) * 16 + j % 16
        c = 16 if e4m3 else 8
        pg, s = slot // 16, slot % 16
        for value in ((0x7F,) if e4m3 else (float("nan"), float("inf"), -float("inf"))):
            v_cache[pg, :, 0, s // c, :, s % c] = value
            k_cache[pg, :, 0, :, s] = value
            got = _f64(w4.w4_tree_attention(*args, **kw))
            assert np.max(np.abs(got - want)[~sees] / tol[~sees]) <= 1
            assert not np.isfinite(got[sees]).any()


def test_attention_rows_that_see_nothing():
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(8)
    # no context, and masks that leave rows empty: zeros; a sequence without tokens; rows outside every sequence
    args, kw, want, tol = _attend(rng, [5, 4], [5, 40], 4, 2, 64, 16, False, True)
    kw["tree"][0] = 0
    kw["tree"][3] = 0
    out = torch.full((9, 4, 64), 7.0, dtype=torch.bfloat16, device=dev())
    got = _f64(w4.w4_tree_attention(*args, **kw, O=out))
    assert (got[0] == 0).all() and (got[3] == 0).all()
    keep = [1, 2, 4, 5, 6, 7, 8]
    assert np.max(np.abs(got - want)[keep] / tol[keep]) <= 1
    args[4] = _i32([0, 40])
    got = _f64(w4.w4_tree_attention(*args, **kw))
    assert (got[:5] == 0).all() and np.max(np.abs(got - want)[5:] / tol[5:]) <= 1
    args[5] = _i32([2, 5, 9])                # rows 0 and 1 belong to nobody
    out.fill_(7.0)
    w4.w4_tree_attention(*args, **kw, O=out)
    assert (out[:2] == 7).all()
    args[5] = _i32([0, 0, 0])
    out.fill_(7.0)
    w4.w4_tree_attention(*args, **kw, O=out)
    assert (out == 7).all()


def test_attention_pages_outside_the_cache_are_not_seen():
    require_gpu()
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(9)
    args, kw, want, _ = _attend(rng, [2], [200], 4, 2, 128, 16, False, True)
    table = args[3].cpu().numpy()
    full = w4.w4_tree_attention(*args, **kw)
    bad = table.copy()
    bad[0, 3], bad[0, 5] = -1, 10 ** 6
    args[3] = _i32(bad)
    got = _f64(w4.w4_tree_attention(*args, **kw))
    # the same as a cache without these 32 tokens: rebuild it, positions do not matter here
    good = np.delete(table, [3, 5], axis=1)
    args[3], args[4], args[7] = _i32(good), _i32([168]), 168
    rest = _f64(w4.w4_tree_attention(*args, **kw))
    assert np.isfinite(got).all() and np.max(np.abs(got - rest)) <= 2.0 ** -6 * np.max(np.abs(rest))
    assert np.max(np.abs(got - _f64(full))) > 0


def test_attention_strided_queries_and_other_streams():
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(10)
    args, kw, want, tol = _attend(rng, [9, 3], [300, 44], 8, 2, 128, 64, False, True)
    wide = torch.zeros((12, 8 * 128 + 40), dtype=torch.bfloat16, device=dev())
    wide[:, :1024] = args[0].reshape(12, -1)
    args[0] = wide[:, :1024].unflatten(1, (8, 128))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    O = w4.w4_tree_attention(*args, **kw, stream=side)
    side.synchronize()
    assert np.max(np.abs(_f64(O) - want) / tol) <= 1


# ------------------------------------------------------------------ sample

def _logits(rng, B, V, f32, stride=None):
    import torch
    x = rng.standard_normal((B, V)) * 2.5
    for r in range(B):
        x[r, rng.integers(0, V, 8)] += rng.uniform(3, 8, 8)
    t = torch.zeros((B, stride or V), dtype=torch.float32 if f32 else torch.bfloat16, device=dev())
    t[:, :V] = torch.from_numpy(x.astype(np.float32)).to(dev())
    return t[:, :V]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V,B,stride", [(1, 3, None), (7, 5, 9), (1000, 12, None), (5003, 9, 5011), (32768, 4, None),
                                        (131072, 3, None), (200003, 2, 200005)])
def test_sample(V, B, stride, f32):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(V + f32)
    x = _logits(rng, B, V, f32, stride)
    for filters in range(6):
        u = rng.random(B).astype(np.float32)
        u[0] = 0.0 if filters % 2 else 1 - 2.0 ** -24
        temp = rng.choice([0.5, 1.0, 1.7], B).astype(np.float32)
        k = rng.choice([0, 1, 5, 50, V], B).astype(np.int32) if filters in (1, 4, 5) else None
        p = rng.choice([0.0, 0.3, 0.9, 0.99, 1.0], B).astype(np.float32) if filters in (2, 4, 5) else None
        m = rng.choice([0.0, 0.05, 0.5, 1.0], B).astype(np.float32) if filters in (3, 5) else None
        to = lambda a: None if a is None else torch.from_numpy(a).to(dev())  # noqa: E731
        tokens, probs = w4.w4_sample(x, to(u), temperature=to(temp), top_k=to(k), top_p=to(p), min_p=to(m))
        for r in range(B):
            w = ref.kept_weights(_f64(x[r]), float(temp[r]), None if k is None else int(k[r]),
                                 None if p is None else float(p[r]), None if m is None else float(m[r]))
            tok = int(tokens[r])
            # the fp32 weights are within 2^-18 of these (the exponent's argument is at most 22 and rounded
            # twice, 2^-24 each), so the running sums, a filter's edge included, are
            slack = 2.0 ** -18 + V * 2.0 ** -32
            share = np.cumsum(w) / w.sum()
            assert 0 <= tok < V
            assert share[tok] >= u[r] - slack and (tok == 0 or share[tok - 1] <= u[r] + slack)
            edge = np.flatnonzero(np.abs(share - u[r]) < slack)
            if w[tok] == 0:                  # only where a filter's edge is within the slack
                assert len(edge) or p is not None or m is not None
            else:
                assert abs(float(probs[r]) - w[tok] / w.sum()) <= 2.0 ** -16 * w[tok] / w.sum() + 2.0 ** -30


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [1, 2, 63, 1000, 8193, 50001, 262144])
def test_sample_equal_logits_take_the_lowest_indices(V, f32):
    # equal weights are exact: token = floor(u n) of the n tokens kept, which are the first of equal ones
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    B = 16
    rng = np.random.default_rng(V)
    x = torch.full((B, V), -3.25, dtype=torch.float32 if f32 else torch.bfloat16, device=dev())
    u = rng.random(B).astype(np.float32)
    uu = torch.from_numpy(u).to(dev())
    units = np.floor(u.astype(np.float64) * 2 ** 24).astype(np.int64)
    tokens, probs = w4.w4_sample(x, uu)
    assert np.array_equal(tokens.cpu().numpy(), units * V >> 24)
    assert np.allclose(probs.cpu().numpy(), 1 / V, rtol=2.0 ** -22)
    k = np.arange(B, dtype=np.int32) * max(1, V // 12) % (V + 1)
    tokens, _ = w4.w4_sample(x, uu, top_k=torch.from_numpy(k).to(dev()))
    n = np.where(k > 0, k, V).astype(np.int64)
    assert np.array_equal(tokens.cpu().numpy(), units * n >> 24)
    p = (np.arange(B) / 16).astype(np.float32)
    tokens, _ = w4.w4_sample(x, uu, top_p=torch.from_numpy(p).to(dev()), min_p=torch.ones(B, device=dev()))
    n = np.maximum(1, -(-V * np.arange(B) // 16)).astype(np.int64)   # tokens until V p is reached
    assert np.array_equal(tokens.cpu().numpy(), units * n >> 24)
    # both filters: p of the k kept
    tokens, _ = w4.w4_sample(x, uu, top_k=torch.from_numpy(k).to(dev()), top_p=torch.from_numpy(p).to(dev()))
    kk = np.where(k > 0, k, V).astype(np.int64)
    n = np.maximum(1, -(-kk * np.arange(B) // 16))
    assert np.array_equal(tokens.cpu().numpy(), units * n >> 24)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [9000, 60001, 200000])
def test_sample_few_values_of_many_tokens(V, f32):
    # 24 different logits: a filter's edge falls inside thousands of equal ones, of which the first are kept
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    B = 8
    rng = np.random.default_rng(V)
    x = rng.choice(rng.uniform(-2, 2, 24), (B, V))
    x[1::2, rng.integers(0, V, 3)] = 1e-6    # among them values of unusual size
    x[2, 5] = 3.0
    x[3, V // 2] = -400.0
    x = torch.from_numpy(x.astype(np.float32)).to(torch.float32 if f32 else torch.bfloat16).to(dev())
    for p, k, m in ((0.9, 0, 0.0), (0.5, 0, 0.0), (0.99, 0, 0.1), (1.0, V // 3, 0.0), (0.7, V // 2, 0.0)):
        u = rng.random(B).astype(np.float32)
        full = lambda a, t: torch.full((B,), a, dtype=t, device=dev())  # noqa: E731
        tokens, probs = w4.w4_sample(x, _f32(u), top_p=full(p, torch.float32), top_k=full(k, torch.int32), min_p=full(m, torch.float32))
        for r in range(B):
            w = ref.kept_weights(_f64(x[r]), 1.0, k, p, m)
            tok, share = int(tokens[r]), np.cumsum(w) / w.sum()
            slack = 2.0 ** -18 + V * 2.0 ** -32 + 1 / np.count_nonzero(w)   # (a kept token more or less)
            assert share[tok] >= u[r] - slack and (tok == 0 or share[tok - 1] <= u[r] + slack)
            assert abs(float(probs[r]) - np.exp(_f64(x[r])[tok] - _f64(x[r]).max()) / w.sum()) <= 2.0 ** -12 * float(probs[r])


@pytest.mark.parametrize("f32", [False, True])
def test_sample_edges(f32):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    inf, nan = float("inf"), float("nan")
    dtype = torch.float32 if f32 else torch.bfloat16
    rows = [[-inf] * 6, [nan] * 6, [1, nan, 3, -inf, 3, 2], [-inf, -5, -inf, -inf, -inf, -inf], [1, inf, 2, inf, 0, 0],
            [-0.0, 0.0, -0.0, -1e30, 0.0, -inf], [-1e30, -2e30, -3e30, -1e30, -inf, -inf]]
    x = torch.tensor(rows, dtype=dtype, device=dev())
    B = len(rows)
    t = lambda *a: torch.tensor(a, dtype=torch.float32, device=dev())  # noqa: E731
    half = t(*[0.5] * B)
    # T = 0 and top_k = 1: the largest logit's lowest index
    for kw in ({"temperature": t(*[0.0] * B)}, {"top_k": _i32([1] * B)}, {"top_p": t(*[0.0] * B)}):
        tokens, probs = w4.w4_sample(x, half, **kw)
        assert tokens.tolist() == [-1, -1, 2, 1, 1, 0, 0], kw
        assert probs.tolist() == [0, 0, 1, 1, 1, 1, 1]
    # infinite logits share everything; equal zeros of both signs are ties
    tokens, _ = w4.w4_sample(x, half)
    assert tokens.tolist()[:2] == [-1, -1] and tokens.tolist()[3:] == [1, 3, 2, 3]
    # out of range numbers do not leave the row
    for bad in (1.0, 2.0, -1.0, nan, inf):
        tokens, _ = w4.w4_sample(x[2:], t(*[bad] * (B - 2)))
        assert all(0 <= v < 6 for v in tokens.tolist())
    # min_p above 1 keeps nothing
    tokens, probs = w4.w4_sample(x[5:6], half[:1], min_p=t(1.5))
    assert tokens.tolist() == [-1] and probs.tolist() == [0]
    assert w4.w4_sample(x[:0], half[:0])[0].shape == (0,)


def test_sample_draws_its_distribution():
    # u over a grid of 2^16 values gives each token its share to within one grid step
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(2)
    V, n = 700, 1 << 15
    x = rng.standard_normal(V).astype(np.float32)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    tokens, _ = w4.w4_sample(torch.from_numpy(x).to(dev()).expand(n, V), torch.from_numpy(u).to(dev()),
                             top_k=_i32([100] * n))
    w = ref.kept_weights(x, 1.0, 100, None, None)
    got = np.bincount(tokens.cpu().numpy(), minlength=V) / n
    assert np.max(np.abs(got - w / w.sum())) <= 1.01 / n


# -------------------------------------------------------------------- move

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layers,hk,d,page", [(None, 3, 64, 16), (3, 2, 128, 48), (2, 1, 256, 64)])
def test_move(layers, hk, d, page, e4m3):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(d + page)
    base, nodes = [0, 5, 40, 61, 7], 40
    pages, table = ref.page_table(rng, [b + nodes for b in base], page)
    n = layers or 1
    parts = [ref.random_cache(rng, pages, hk, d, page, e4m3, dev()) for _ in range(n)]
    k, v = (torch.stack([p[i] for p in parts]) for i in range(2))
    before = [ref.to_tokens(k[i], v[i]) for i in range(n)]
    path = np.zeros((len(base), 20), np.int32)
    count = [6, 20, 0, 1, 12]
    for b, c in enumerate(count):
        path[b, :c] = np.sort(rng.choice(nodes, c, replace=False))
    path[1] = np.arange(20)                  # stays where it is
    if layers is None:
        k, v = k[0], v[0]
    w4.w4_kv_move(k, v, _i32(table), _i32(base), _i32(path), _i32(count))
    for i in range(n):
        got = ref.to_tokens(k if layers is None else k[i], v if layers is None else v[i])
        for g, old in zip(got, before[i]):
            want = old.copy()
            for b, c in enumerate(count):
                slot = lambda t: int(table[b, t // page]) * page + t % page  # noqa: E731,B023
                for j in range(c):
                    want[slot(base[b] + j)] = old[slot(base[b] + int(path[b, j]))]
            assert np.array_equal(g, want, equal_nan=True)


@pytest.mark.parametrize("e4m3", [False, True])
def test_move_long_paths_and_places_outside(e4m3):
    """More tokens than are looked up at a time; a base below zero; pages outside the cache; a path past the table."""
    require_gpu()
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(4)
    hk, d, page, nodes = 3, 128, 32, 300
    base = [9, 0, -1, 70]
    pages, table = ref.page_table(rng, [max(b, 0) + nodes for b in base], page)
    table[3, 4], table[3, 9] = -1, pages
    k, v = ref.random_cache(rng, pages, hk, d, page, e4m3, dev())
    before = ref.to_tokens(k, v)
    count = [211, 150, 20, 100]
    path = np.zeros((4, 211), np.int32)
    for b, c in enumerate(count):
        path[b, :c] = np.sort(rng.choice(nodes, c, replace=False))
    path[1, 149] = 10 ** 9
    w4.w4_kv_move(k, v, _i32(table), _i32(base), _i32(path), _i32(count))
    for got, old in zip(ref.to_tokens(k, v), before):
        want = old.copy()
        for b, c in enumerate(count):
            def slot(t):
                p = int(table[b, t // page]) if 0 <= t // page < table.shape[1] else -1  # noqa: B023
                return p * page + t % page if 0 <= p < pages else None
            for j in range(c if base[b] >= 0 else 0):
                to, source = slot(base[b] + j), slot(base[b] + int(path[b, j]))
                if to is not None and source is not None:
                    want[to] = old[source]
        assert np.array_equal(got, want, equal_nan=True)


def test_results_of_another_stream_are_not_handed_out_early():
    """Outputs allocated for a call on another stream keep their memory until that stream is through, even if the
    caller drops them at once: what is allocated next on the current stream does not get it meanwhile."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    side = torch.cuda.Stream()
    x = torch.randn((8, 4099), device=dev())
    u = torch.rand(8, device=dev())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy = torch.randn((4096, 4096), device=dev())
        for _ in range(8):
            busy = busy @ busy * 1e-4        # (keeps the stream occupied for a while)
    tokens, probs = w4.w4_sample(x, u, stream=side)
    places = {tokens.data_ptr(), probs.data_ptr()}
    early = not side.query()
    del tokens, probs
    fresh = [torch.empty((8,), dtype=torch.int32, device=dev()) for _ in range(4)]
    if early:
        assert not places & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()


# ------------------------------------------------------------ graph capture

def test_calls_replay_from_a_graph():
    # a decode step captured once, replayed three times on new inputs, against the same calls run eagerly
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(4)
    B, hq, hk, d, page, V = 3, 8, 2, 128, 16, 4000
    lengths = [900, 33, 2500]
    pages, table = ref.page_table(rng, lengths, page)
    k_cache, v_cache = ref.random_cache(rng, pages, hk, d, page, False, dev())
    qkv = _bf16(rng.standard_normal((B, hq + 2 * hk, d)))
    at = np.array(lengths) - 1
    slots = _i32(table[np.arange(B), at // page] * page + at % page)
    rope = torch.from_numpy(ref.rope_table(2500, d)).to(dev())
    logits = torch.randn((B, V), device=dev())
    u = torch.rand(B, device=dev())
    t = [_i32(table), _i32(lengths), _i32([0, 1, 2, 3]), _i32(at), _i32([50] * B)]
    top_p = torch.full((B,), 0.9, device=dev())

    def step():
        Q = w4.w4_kv_append(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, k_cache, v_cache, rope=rope, positions=t[3])
        O = w4.w4_tree_attention(Q, k_cache, v_cache, t[0], t[1], t[2], 1, 2500)
        return (Q, O, *w4.w4_sample(logits, u, top_k=t[4], top_p=top_p))

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(3):
        qkv.copy_(torch.randn_like(qkv))
        logits.copy_(torch.randn_like(logits))
        u.copy_(torch.rand_like(u))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), rep
        torch.cuda.synchronize()
