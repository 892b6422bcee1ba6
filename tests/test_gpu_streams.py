"""Memory of calls on another stream than the current one.

What a call on the current stream allocated and dropped goes back to that stream's pool at once, while its kernels
may still run.  A call on another stream must not be given it: not for a workspace, which both would write at the
same time, and not for a result.  Addresses show it whatever the timing."""
import numpy as np
import pytest

import decode_ref as ref
from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu

PRODUCTS = ["quantize", "clip_search", "prepack", "rows", "w4a16", "w4a8", "e4m3", "gate_up16", "gate_up8", "nf4"]


def _pointers(w4, name, monkeypatch):
    """Device addresses that every call of the C entry point gets, collected in a list."""
    seen = []
    real = getattr(w4.lib(), name)

    def call(*args):
        seen.append({a for a in args[:-1] if isinstance(a, int) and a > 1 << 32})
        return real(*args)

    monkeypatch.setattr(w4.lib(), name, call)
    return seen


def _differ(w4, monkeypatch, entry, call, given):
    """`call(stream)` on the current stream and, while that may run, on another: memory that the binding allocated for
    the first is not used by the second, and both results are the same."""
    import torch
    side = torch.cuda.Stream()
    want = [x.clone() for x in call(None)]
    torch.cuda.synchronize()
    seen = _pointers(w4, entry, monkeypatch)
    busy = torch.randn((2048, 2048), device=dev())
    for _ in range(4):
        busy = busy @ busy * 1e-3            # (the current stream has work before the first call's)
    call(None)                               # results and workspace dropped at once
    got = call(side)
    torch.cuda.synchronize()
    monkeypatch.undo()
    given = {t.data_ptr() for t in given}
    first, second = (s - given for s in seen)
    assert first and second and not first & second, entry
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), entry


@pytest.mark.parametrize("name", PRODUCTS)
def test_products(name, monkeypatch):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    gen = torch.Generator(device=dev()).manual_seed(1)
    N, K, G, M = 512, 8192, 128, 100         # (products of these sizes split K: they need a workspace)
    W = torch.randn((N, K), generator=gen, device=dev()) * 0.02
    q = w4.w4_quantize_blockwise(W, G, "asym")
    p = w4.w4_prepack(q["packed"], q["scale"], q["zero"], G, "asym")
    X = torch.randn((M, K), generator=gen, device=dev()).to(torch.bfloat16)
    xq, xs = w4.w4_quantize_rows_e4m3(X)
    nf4 = w4.w4_nf4_quantize(W)
    assert w4.w4_gemm_workspace_bytes(M, K, N) > 0 and w4.w4a8_gemm_workspace_bytes(M, K, N) > 0
    entry, call = {
        "quantize": ("w4_quantize_blockwise", lambda s: list(w4.w4_quantize_blockwise(W, G, "asym", stream=s).values())),
        "clip_search": ("w4_mse_clip_search", lambda s: list(w4.w4_mse_clip_search(W, G, "asym", w4.FRACS_11, want_sse=True, stream=s).values())),
        "prepack": ("w4_prepack", lambda s: list(w4.w4_prepack(q["packed"], q["scale"], q["zero"], G, "asym", stream=s).values())),
        "rows": ("w4_quantize_rows_e4m3", lambda s: list(w4.w4_quantize_rows_e4m3(X, stream=s))),
        "w4a16": ("w4a16_gemm", lambda s: [w4.w4a16_gemm(X, p["wq"], p["sz"], G, stream=s)]),
        "w4a8": ("w4a8_gemm", lambda s: list(w4.w4a8_gemm(X, p["wq"], p["sz"], G, stream=s))),
        "e4m3": ("w4a8_gemm_e4m3", lambda s: [w4.w4a8_gemm_e4m3(xq, xs, p["wq"], p["sz"], G, stream=s)]),
        "gate_up16": ("w4a16_gate_up", lambda s: [w4.w4a16_gate_up(X, p, p, G, stream=s)]),
        "gate_up8": ("w4a8_gate_up", lambda s: list(w4.w4a8_gate_up(X, p, p, G, emit_e4m3=True, stream=s))),
        "nf4": ("w4_nf4_gemv", lambda s: [w4.w4_nf4_gemv(X[0], nf4, stream=s)]),
    }[name]
    _differ(w4, monkeypatch, entry, call, [W, X, xq, xs, *q.values(), *p.values(), *nf4.values()])


def test_decoding_calls(monkeypatch):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    rng = np.random.default_rng(3)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev())  # noqa: E731
    length, hq, hk, d, page = 20000, 8, 2, 128, 64
    pages, table = ref.page_table(rng, [length], page)
    k_cache, v_cache = ref.random_cache(rng, pages, hk, d, page, False, dev())
    q = torch.randn((3, hq, d), device=dev()).to(torch.bfloat16)
    k = torch.randn((3, hk, d), device=dev()).to(torch.bfloat16)
    t = [i32(table), i32([length]), i32([0, 3]), i32([5, 70, 9])]
    assert w4.w4_tree_attention_workspace_bytes(3, 1, hq, hk, d, False, 3, length) > 0
    own = [(x.clone(), y.clone()) for x, y in [(k_cache, v_cache)] * 2]   # (appended to at the same time)
    given = [q, k, k_cache, v_cache, *t, *own[0], *own[1]]
    _differ(w4, monkeypatch, "w4_tree_attention",
            lambda s: [w4.w4_tree_attention(q, k_cache, v_cache, t[0], t[1], t[2], 3, length, stream=s)], given)
    _differ(w4, monkeypatch, "w4_kv_append", lambda s: [w4.w4_kv_append(q, k, k, t[3], *own[s is None], stream=s)], given)
    x, u = torch.randn((9, 5000), device=dev()), torch.rand(9, device=dev())
    _differ(w4, monkeypatch, "w4_sample", lambda s: w4.w4_sample(x, u, stream=s), [x, u])
