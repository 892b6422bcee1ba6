"""The calls of a layer as a serving loop makes them: captured into graphs and replayed, on other streams, with
workspaces of its own, past 32-bit offsets, and one decoding step of all of them together."""
import numpy as np
import pytest

import decode_ref
import moe_ref as ref
from helpers import dev, require_gpu
from test_gpu_streams import _differ

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch
    return torch.Generator(device=dev()).manual_seed(seed)


def _bf(g, *shape):
    import torch
    return torch.randn(shape, generator=g, device=dev()).to(torch.bfloat16)


class _Absent:
    """In place of the binding's compiled way: takes no call."""

    def __getattr__(self, name):
        return lambda *args: None


# tokens, choices, experts, hidden, inner, group: dot products; rows of one pass with the lists in it; with lists of
# their own; two passes' rows; tiles with each group size, and with the down product's k split
MOE = [(1, 2, 8, 256, 384, 32), (2, 8, 16, 512, 256, 128), (12, 4, 4, 256, 1024, 64), (30, 8, 64, 256, 256, 128),
       (52, 2, 8, 128, 4352, 128), (200, 4, 6, 256, 256, 32), (200, 4, 6, 256, 512, 64), (90, 3, 3, 256, 4096, 128)]


def _moe_calls(w4, seed, T, k, E, H, I, G):
    """A layer's inputs and a call of route and experts."""
    g = _gen(seed)
    w = [ref.experts(g, E, n, kk, G, dev()) for n, kk in ((I, H), (I, H), (H, I))]
    x, router, res = _bf(g, T, H), _bf(g, E, H), _bf(g, T, H)

    def call(stream=None):
        ids, weights = w4.w4_route(x, router, k, stream=stream)
        y = w4.w4a16_moe(x, ids, weights, *w, G, residual=res, stream=stream)
        return [ids, weights, y]
    return [x, router, res, *(t[key] for t in w for key in ("wq", "sz"))], call


def _linear_calls(w4, seed, kind, M, N, K, G):
    import torch
    g = _gen(seed)
    w = ref.experts(g, 1, N, K, G, dev())
    wq, sz = w["wq"][0].contiguous(), w["sz"][0].contiguous()
    x, bias, res = _bf(g, M, K), torch.randn(N, generator=g, device=dev()), _bf(g, M, N)

    def call(stream=None):
        f = w4.w4a16_linear if kind == "a16" else w4.w4a8_linear
        r = f(x, wq, sz, G, bias=bias, act="silu", residual=res, stream=stream)
        return [r] if kind == "a16" else list(r)
    return [x, bias, res, wq, sz], call


def _adjust_calls(w4, seed, B, V, dtype):
    import torch
    g, rng = _gen(seed), np.random.default_rng(seed)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev())                  # noqa: E731
    f = lambda: torch.rand(B, generator=g, device=dev()) + 0.5                                    # noqa: E731
    logits = torch.randn((B, V), generator=g, device=dev()).to(dtype)
    lens = rng.integers(0, 400, B)
    starts = i32(np.concatenate([[0], np.cumsum(lens)]))
    history = i32(rng.integers(0, V, int(lens.sum())))
    prompt, rep, pres, freq = i32(lens // 2), f(), f(), f()
    bstart, bids = i32(np.arange(B + 1) * 3), i32(np.concatenate([rng.choice(V, 3, replace=False) for _ in range(B)]))
    bvals = torch.randn(3 * B, generator=g, device=dev())
    mask = torch.randint(-2**31, 2**31 - 1, (B, (V + 31) // 32), dtype=torch.int32, generator=g, device=dev())
    given = [logits, starts, history, prompt, rep, pres, freq, bstart, bids, bvals, mask]

    def call(stream=None):
        return [w4.w4_adjust_logits(logits, history=history, history_start=starts, prompt_len=prompt, repetition=rep,
                                    presence=pres, frequency=freq, bias_start=bstart, bias_ids=bids, bias_values=bvals,
                                    mask=mask, stream=stream)]
    return given, call


def _all_calls(w4):
    import torch
    for i, s in enumerate(MOE):
        yield f"moe {s}", *_moe_calls(w4, 40 + i, *s)
    for i, (kind, *s) in enumerate([("a16", 1, 576, 1536, 32), ("a16", 16, 520, 14336, 128), ("a16", 48, 1000, 4096, 64),
                                    ("a16", 300, 515, 2048, 128), ("a8", 1, 300, 1024, 128), ("a8", 40, 256, 8192, 128),
                                    ("a8", 300, 515, 2048, 64)]):
        yield f"linear {kind} {s}", *_linear_calls(w4, 60 + i, kind, *s)
    for i, s in enumerate([(1, 5001, torch.float32), (3, 131072, torch.float32), (70, 50001, torch.bfloat16)]):
        yield f"adjust {s}", *_adjust_calls(w4, 80 + i, *s)


def _same(a, b, what):
    import torch
    for i, (x, y) in enumerate(zip(a, b)):
        same = torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
        assert same, f"{what}: output {i}"


def _capture(torch, call):
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    return g, out


@pytest.mark.parametrize("which", range(18))
def test_graphs(which):
    """Captured twice, both graphs replayed in turn on new inputs, with eager calls between."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    what, inputs, call = list(_all_calls(w4))[which]
    print(f"[graph] {what}", flush=True)
    graphs = [_capture(torch, call) for _ in range(2)]
    gen = _gen(7)
    for rep in range(3):
        x = inputs[0]
        x.copy_(torch.randn(x.shape, generator=gen, device=dev()).to(x.dtype))
        for g, out in graphs:
            for o in out:
                o.zero_()
            g.replay()
        torch.cuda.synchronize()
        want = call()
        torch.cuda.synchronize()
        for g, out in graphs:
            _same(out, want, f"{what}, replay {rep}")


def test_graphs_that_share_a_workspace():
    """Two layers' graphs with one workspace, replayed one after the other."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    for i, (T, k, E, H, I, G) in enumerate(MOE):
        g = _gen(i)
        ws = torch.empty(w4.w4a16_moe_workspace_bytes(T, k, E, H, I, G), dtype=torch.uint8, device=dev())
        layers = []
        for _ in range(2):
            w = [ref.experts(g, E, n, kk, G, dev()) for n, kk in ((I, H), (I, H), (H, I))]
            ids = torch.randint(0, E, (T, k), generator=g, device=dev(), dtype=torch.int32)
            args = (_bf(g, T, H), ids, torch.rand((T, k), generator=g, device=dev()), *w, G)
            want = w4.w4a16_moe(*args)
            Y = torch.empty_like(want)
            graph, _ = _capture(torch, lambda: [w4.w4a16_moe(*args, Y=Y, workspace=ws)])
            layers.append((graph, Y, want, args))            # (a graph reads its inputs where they were)
        for rep in range(3):
            for graph, Y, *_ in layers:
                Y.zero_()
                graph.replay()
            ws.fill_(255)                                    # (behind the replays, on their stream)
            for _, Y, want, _ in layers:
                _same([Y], [want], f"{(T, k, E, H, I, G)} replay {rep}")


def test_streams(monkeypatch):
    require_gpu()
    import w4_dequant_gemm_amd as w4
    entries = {"moe": ("w4_route", "w4a16_moe"), "linear a16": ("w4a16_linear",), "linear a8": ("w4a8_linear",),
               "adjust": ("w4_adjust_logits",)}
    for what, given, call in _all_calls(w4):
        for entry in next(v for n, v in entries.items() if what.startswith(n)):
            if entry == "w4_route":
                call_ = lambda s, c=call: c(s)[:2]           # noqa: E731
            else:
                call_ = call
            monkeypatch.setattr(w4, "_call", _Absent())
            print(f"[streams] {what} {entry}", flush=True)
            given_ = list(given)
            if entry == "w4a16_moe":                         # (the routing's results are inputs of this one)
                ids, weights, _ = call(None)
                T, H, G, k = *given[0].shape, 8 * given[3].shape[2] // given[4].shape[2], ids.shape[1]
                gate, up, down = ({"wq": given[i], "sz": given[i + 1]} for i in (3, 5, 7))
                call_ = lambda s: [w4.w4a16_moe(given[0], ids, weights, gate, up, down, G, residual=given[2], stream=s)]  # noqa: E731
                given_ += [ids, weights]
            _differ(w4, monkeypatch, entry, call_, given_)


def test_memory_of_the_compiled_way_is_the_current_streams():
    """What a call on one stream dropped may still be in use there: a call under another current stream gets other
    memory, and its result is the same while the first stream is busy."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    side = torch.cuda.Stream()
    for what, _, call in _all_calls(w4):
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        busy = torch.randn((2048, 2048), device=dev())
        for _ in range(4):
            busy = busy @ busy * 1e-3
        dropped = {t.data_ptr() for t in call()}
        with torch.cuda.stream(side):
            got = call()
        torch.cuda.synchronize()
        assert not dropped & {t.data_ptr() for t in got}, what
        _same(got, want, what)


@pytest.mark.parametrize("shape", MOE)
def test_workspace_as_long_as_asked(shape):
    """Exactly the bytes asked for, full of NaN, are enough, and the bytes behind them stay; fewer are refused."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    T, k, E, H, I, G = shape
    g = _gen(3)
    w = [ref.experts(g, E, n, kk, G, dev()) for n, kk in ((I, H), (I, H), (H, I))]
    x, router = _bf(g, T, H), _bf(g, E, H)
    ids, weights = w4.w4_route(x, router, k)
    want = w4.w4a16_moe(x, ids, weights, *w, G)
    for entry, need in (("route", w4.w4_route_workspace_bytes(T, H, E)), ("moe", w4.w4a16_moe_workspace_bytes(T, k, E, H, I, G))):
        if not need:
            continue
        all_ = torch.full((need + 4096,), 255, dtype=torch.uint8, device=dev())
        ws = all_[:need]
        if entry == "route":
            got, expected = list(w4.w4_route(x, router, k, workspace=ws)), [ids, weights]
        else:
            got, expected = [w4.w4a16_moe(x, ids, weights, *w, G, workspace=ws)], [want]
        torch.cuda.synchronize()
        _same(got, expected, entry)
        assert bool((all_[need:] == 255).all())
        with pytest.raises(w4.W4Error):
            if entry == "route":
                w4.w4_route(x, router, k, workspace=ws[:need - 1])
            else:
                w4.w4a16_moe(x, ids, weights, *w, G, workspace=ws[:need - 1])


def test_calls_of_two_threads():
    """Each of two host threads on a stream of its own, at the same time: every result as by itself."""
    require_gpu()
    import threading

    import torch
    import w4_dequant_gemm_amd as w4
    calls = [(what, call) for what, _, call in _all_calls(w4)]
    want = [[t.clone() for t in call()] for _, call in calls]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), []

    def run(backwards):
        stream = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(stream):
            for _ in range(3):
                got = {i: calls[i][1]() for i in (reversed(range(len(calls))) if backwards else range(len(calls)))}
                stream.synchronize()
                for i, r in got.items():
                    wrong.extend(calls[i][0] for a, b in zip(r, want[i])
                                 if not torch.equal(a.view(torch.uint8), b.view(torch.uint8)))

    threads = [threading.Thread(target=run, args=(b,)) for b in (False, True)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_experts_behind_32_bits():
    """1024 experts of 4 MB of codes a matrix: the last ones lie past 2^32 bytes, and give what they give by
    themselves.  (All forms: their rules come out alike for 1024 and for 64 experts at these numbers of tokens.)"""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    E, H, I, G, few = 1024, 1024, 8192, 128, 64
    g = _gen(4)
    weight = lambda n, kk: {"wq": torch.randint(-2**31, 2**31 - 1, (E, n, kk // 8), dtype=torch.int32, generator=g, device=dev()),  # noqa: E731
                            "sz": torch.full((E, n, kk // G), 0x48001400, dtype=torch.int32, device=dev())}
    gate, up, down = weight(I, H), weight(I, H), weight(H, I)
    assert gate["wq"].nbytes >= 1 << 32
    last = [{key: t[key][-few:].contiguous() for key in t} for t in (gate, up, down)]
    for T, k in ((1, 2), (3, 2), (40, 8), (5000, 5)):
        print(f"[wide] {T} tokens", flush=True)
        x = _bf(g, T, H) / 32
        ids = torch.randint(0, few, (T, k), generator=g, device=dev(), dtype=torch.int32)
        wt = torch.rand((T, k), generator=g, device=dev())
        got, want = w4.w4a16_moe(x, ids + (E - few), wt, gate, up, down, G), w4.w4a16_moe(x, ids, wt, *last, G)
        torch.cuda.synchronize()
        # (the down product's k may be split differently: fp32 sums in another order, far below half a step of bf16)
        assert ((got.double() - want.double()).abs() <= 2 * ref.BF16 * want.double().abs() + 1e-3 * want.double().abs().mean()).all()
        assert torch.isfinite(want.float()).all() and want.float().abs().mean() > 0


def test_logits_behind_32_bits():
    """More logits than 2^31, and more bytes than 2^32: the last rows are as they are by themselves."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    B, V, rows = 8400, 262144, 3
    logits = torch.empty((B, V), dtype=torch.bfloat16, device=dev())
    logits.view(torch.int16).random_(0, 16000, generator=_gen(1))
    assert logits.numel() > 1 << 31
    history = torch.arange(0, V, 97, dtype=torch.int32, device=dev())
    starts = torch.full((B + 1,), history.numel(), dtype=torch.int32, device=dev())
    starts[:-rows] = 0                                       # (the last rows' histories, the last's being the whole)
    starts[-rows - 1:-1] = 0
    rep = torch.full((B,), 1.3, device=dev())
    mask = torch.randint(-2**31, 2**31 - 1, (B, V // 32), dtype=torch.int32, generator=_gen(2), device=dev())
    got = w4.w4_adjust_logits(logits, history=history, history_start=starts, repetition=rep, mask=mask)
    for first in (0, B - rows):
        part = slice(first, first + rows)
        want = w4.w4_adjust_logits(logits[part], history=history, history_start=starts[first:first + rows + 1].contiguous(),
                                   repetition=rep[part], mask=mask[part])
        assert torch.equal(got[part], want)
    assert not torch.equal(got[-1], torch.where(got[-1].isinf(), got[-1], logits[-1]))       # (its history did something)


@pytest.mark.parametrize("kind", ["a16", "a8"])
def test_results_behind_32_bits(kind):
    """M N beyond 2^31: residual, bias and result of the last rows, against the same rows by themselves."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    M, N, K, G, rows = 33000, 66000, 64, 32, 300
    g = _gen(2)
    w = ref.experts(g, 1, N, K, G, dev())
    wq, sz = w["wq"][0].contiguous(), w["sz"][0].contiguous()
    x, bias = _bf(g, M, K), torch.randn(N, generator=g, device=dev())
    res = torch.empty((M, N), dtype=torch.bfloat16, device=dev())
    res.view(torch.int16).random_(0, 16256, generator=g)     # 0 .. 1
    assert M * N > 1 << 31
    if kind == "a16":
        got, read = w4.w4a16_linear(x, wq, sz, G, bias=bias, residual=res), x[-rows:].double()
    else:
        got, xq, xs = w4.w4a8_linear(x, wq, sz, G, bias=bias, residual=res)
        read = xq[-rows:].view(torch.float8_e4m3fn).double() * xs[-rows:, None].double()
    want, bound = ref.product(read, torch.zeros_like(read), w, 0)
    want = want + bias.double() + res[-rows:].double()
    # (groups of 32, and tiles of many rows, multiply s (u - z) rounded to bf16: off by half a step, 2^-8 of each weight)
    bound = bound + ref.BF16 * (read.abs() @ w["W"][0].abs().T) + 4 * ref.U * (want.abs() + bias.abs().double() + 1)
    assert ((got[-rows:].double() - want).abs() <= bound + ref.BF16 * (want.abs() + bound)).all()


def test_decoding_step():
    """One token of each sequence through a layer and the head, every call of the library it takes, against the same in
    64 bits from the values that each call was given: product with bias, cache, attention, product with the stream
    added, routing, experts with the stream added, head, penalties and mask, and the sampled token."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng, g = np.random.default_rng(5), _gen(6)
    B, H, hq, hk, d, page, E, k, I, G, V = 3, 512, 8, 2, 64, 16, 8, 2, 384, 128, 1000
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev())                  # noqa: E731
    weight = lambda n, kk: ref.experts(g, 1, n, kk, G, dev())                                     # noqa: E731
    wqkv, wo, wh = weight((hq + 2 * hk) * d, H), weight(H, hq * d), weight(V, H)
    experts = [ref.experts(g, E, n, kk, G, dev()) for n, kk in ((I, H), (I, H), (H, I))]
    bqkv = torch.randn((hq + 2 * hk) * d, generator=g, device=dev())
    router, x = _bf(g, E, H), _bf(g, B, H)
    lens = [5, 40, 17]
    pages, table = decode_ref.page_table(rng, [n + 1 for n in lens], page)
    kc, vc = decode_ref.random_cache(rng, pages, hk, d, page, False, dev())
    table, at, kv_len, q_start = i32(table), [], i32([n + 1 for n in lens]), i32(range(B + 1))
    for b, n in enumerate(lens):
        at.append(int(table[b, n // page]) * page + n % page)
    slots = i32(at)
    history, hs = i32(rng.integers(0, V, sum(lens))), i32(np.concatenate([[0], np.cumsum(lens)]))
    rep = torch.full((B,), 1.2, device=dev())
    mask = torch.randint(-2**31, 2**31 - 1, (B, (V + 31) // 32), dtype=torch.int32, generator=g, device=dev())
    u = torch.rand(B, generator=g, device=dev())
    lin = lambda x_, w, **o: w4.w4a16_linear(x_, w["wq"][0], w["sz"][0], G, **o)                  # noqa: E731

    def step():
        qkv = lin(x, wqkv, bias=bqkv)
        q, kk, v = (t.reshape(B, -1, d) for t in qkv.split([hq * d, hk * d, hk * d], 1))
        w4.w4_kv_append(q, kk, v, slots, kc, vc)
        o = w4.w4_tree_attention(q, kc, vc, table, kv_len, q_start, 1, max(lens) + 1)
        x1 = lin(o.view(B, hq * d), wo, residual=x)
        ids, weights = w4.w4_route(x1, router, k)
        x2 = w4.w4a16_moe(x1, ids, weights, *experts, G, residual=x1)
        logits = lin(x2, wh)
        ready = w4.w4_adjust_logits(logits, history=history, history_start=hs, repetition=rep, mask=mask)
        tokens, probs = w4.w4_sample(ready, u)
        return qkv, o, x1, ids, weights, x2, logits, ready, tokens, probs

    out = step()
    torch.cuda.synchronize()
    qkv, o, x1, ids, weights, x2, logits, ready, tokens, probs = out

    def near(got, x_, w, plus):
        want, bound = ref.product(x_.double(), torch.zeros_like(x_).double(), w, 0)
        want = want + plus
        assert ((got.double() - want).abs() <= bound + 8 * ref.U * want.abs() + ref.BF16 * (want.abs() + bound)).all()
    near(qkv, x, wqkv, bqkv.double())
    # attention over the cache as it is now: the step's own key and value are in it
    kt, vt = decode_ref.to_tokens(kc, vc)
    places = table.cpu().numpy()
    for b, n in enumerate(lens):
        where = [places[b, i // page] * page + i % page for i in range(n + 1)]
        own = qkv[b].double().cpu().numpy()
        assert np.array_equal(kt[where[n]].reshape(-1), own[hq * d:(hq + hk) * d])
        assert np.array_equal(vt[where[n]].reshape(-1), own[(hq + hk) * d:])
        want, bound = decode_ref.attention(own[:hq * d].reshape(1, hq, d), kt[where], vt[where], n, d ** -0.5)
        assert (np.abs(o[b].double().cpu().numpy() - want[0]) <= bound[0]).all()
    near(x1, o.view(B, hq * d), wo, x.double())
    wid, w64, dl, sure = ref.route(x1, router, k)
    assert torch.equal(ids.long()[sure], wid[sure]) and sure.double().mean() >= 0.25
    want, bound = ref.moe(x1, ids, weights, *experts, "silu", x1)
    assert ((x2.double() - want).abs() <= bound).all()
    near(logits, x2, wh, 0)
    bits = (mask[:, torch.arange(V, device=dev()) // 32] >> (torch.arange(V, device=dev()) % 32).int()) & 1
    seen = torch.zeros((B, V), dtype=torch.bool, device=dev())
    for b in range(B):
        seen[b, history[hs[b]:hs[b + 1]].long()] = True
    l = logits.double()
    want = torch.where(seen, torch.where(l > 0, l / rep[:, None].double(), l * rep[:, None].double()), l)
    want = torch.where(bits == 1, want, torch.full_like(want, -float("inf")))
    assert torch.equal(ready.isinf(), want.isinf())
    ok = ~want.isinf()
    assert ((ready.double() - want).abs()[ok] <= ((ref.BF16 + 2 * ref.U) * want.abs())[ok]).all()
    p = torch.softmax(ready.double(), 1)
    rows = torch.arange(B, device=dev())
    assert (bits[rows, tokens.long()] == 1).all()
    # (V additions, and exponents of up to the span known to two roundings of it, above and below the fraction)
    span = ready.double()[ok].max() - ready.double()[ok].min()
    chosen = p[rows, tokens.long()]
    assert ((probs.double() - chosen).abs() <= 2 * ref.U * (V + 2 * span + 16) * chosen).all()

    # the same step captured and replayed
    g1, again = _capture(torch, lambda: list(step()))
    for rep_ in range(3):
        for t in again:
            t.zero_()
        g1.replay()
        torch.cuda.synchronize()
        _same(again, out, f"step, replay {rep_}")
        _same(step(), out, "eager step")
