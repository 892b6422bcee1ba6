"""The decoding calls without a GPU: their C ABI refuses bad arguments on the
host before any launch, and the binding refuses wrong shapes and types."""
import ctypes
import os

import pytest
import torch

FAKE = ctypes.c_void_p(0x1000)          # never dereferenced: the calls below fail their checks or do nothing
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    import w4_dequant_gemm_amd as w4
    if not os.path.exists(w4.library_path):
        from w4_dequant_gemm_amd import build
        build.build()
    return w4.lib()


def _cache(**kw):
    import w4_dequant_gemm_amd as w4
    f = dict(k=0x1000, v=0x1000, k_scale=None, v_scale=None, pages=10, layers=1, kv_heads=2, head_dim=128, page_size=32,
             dtype=0)
    f.update(kw)
    return w4._KvCache(**f)


BAD_CACHES = [(dict(dtype=2), 1), (dict(head_dim=96), 2), (dict(head_dim=512), 2), (dict(page_size=24), 2),
              (dict(page_size=0), 2), (dict(page_size=2048), 2), (dict(kv_heads=0), 1), (dict(layers=0), 1),
              (dict(pages=0), 1), (dict(pages=1 << 27), 1), (dict(k=None), 1), (dict(v=0x1008), 1)]


def _append(lib, cache=None, **kw):
    a = dict(q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, T=3, hq=4, slots=FAKE, rope=FAKE, rows=9, rot=128, inter=0,
             pos=FAKE, qn=None, kn=None, eps=1e-6, Q=FAKE)
    a.update(kw)
    return lib.w4_kv_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["hq"],
                            ctypes.byref(cache) if cache is not None else None, a["slots"], a["rope"], a["rows"], a["rot"],
                            a["inter"], a["pos"], a["qn"], a["kn"], a["eps"], a["Q"], None)


def test_append_refusals(lib):
    import w4_dequant_gemm_amd as w4
    for f, status in BAD_CACHES:
        assert _append(lib, _cache(**f)) == status, f
    assert _append(lib, None) == 1
    assert _append(lib, _cache(layers=2)) == 1
    assert _append(lib, _cache(dtype=1)) == 1 and "k_scale" in w4.w4_last_error()
    assert _append(lib, _cache(k_scale=0x1000, v_scale=0x1000)) == 1
    for f, status in ((dict(q=None), 1), (dict(Q=None), 1), (dict(hq=0), 1), (dict(T=-1), 1), (dict(T=1 << 30), 1),
                      (dict(qs=511), 1), (dict(qs=504), 1), (dict(ks=248), 1), (dict(vs=260), 1), (dict(k=None), 1),
                      (dict(v=ODD), 1), (dict(Q=ODD), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(rope=None), 1),
                      (dict(rope=ODD), 1), (dict(rows=0), 1), (dict(rot=0), 1), (dict(rot=144), 1), (dict(rot=24), 2),
                      (dict(qn=ODD), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1)):
        assert _append(lib, _cache(), **f) == status, f
    assert _append(lib, _cache(), T=0, q=None, Q=None, k=None, v=None) == 0


def _attend(lib, cache=None, **kw):
    a = dict(q=FAKE, qs=512, T=6, hq=4, table=FAKE, pages=5, kv=FAKE, start=FAKE, B=2, max_q=3, max_kv=150, tree=FAKE,
             words=1, pos=None, window=0, scale=0.1, O=FAKE, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return lib.w4_tree_attention(a["q"], a["qs"], a["T"], a["hq"], ctypes.byref(cache) if cache is not None else None,
                                 a["table"], a["pages"], a["kv"], a["start"], a["B"], a["max_q"], a["max_kv"], a["tree"],
                                 a["words"], a["pos"], a["window"], a["scale"], a["O"], a["ws"], a["ws_bytes"], None)


def test_attention_refusals(lib):
    import w4_dequant_gemm_amd as w4
    for f, status in BAD_CACHES:
        assert _attend(lib, _cache(**f)) == status, f
    assert _attend(lib, None) == 1 and _attend(lib, _cache(layers=2)) == 1 and _attend(lib, _cache(dtype=1)) == 1
    for f, status in ((dict(T=-1), 1), (dict(B=-1), 1), (dict(hq=3), 1), (dict(hq=0), 1), (dict(max_q=7), 1),
                      (dict(max_q=-1), 1), (dict(max_kv=-1), 1), (dict(max_kv=161), 1), (dict(max_kv=1 << 30), 1),
                      (dict(window=-1), 1), (dict(window=5), 1), (dict(q=None), 1), (dict(q=ODD), 1), (dict(qs=500), 1),
                      (dict(O=None), 1), (dict(O=ODD), 1), (dict(table=None), 1), (dict(pages=0), 1), (dict(kv=None), 1),
                      (dict(start=None), 1), (dict(words=0), 1), (dict(T=200, max_q=65), 1), (dict(scale=float("inf")), 1),
                      (dict(ws=ODD), 1), (dict(B=70000), 2)):
        assert _attend(lib, _cache(), **f) == status, f
    for f in (dict(T=0), dict(B=0), dict(max_q=0)):
        assert _attend(lib, _cache(), **f) == 0, f
    # split tokens need their workspace
    need = lib.w4_tree_attention_workspace_bytes(6, 2, 4, 2, 128, 0, 3, 100000, 0)
    assert need > 0
    long = dict(pages=4000, max_kv=100000)
    assert _attend(lib, _cache(), **long, ws=None) == 1 and "workspace" in w4.w4_last_error()
    assert _attend(lib, _cache(), **long, ws_bytes=need - 4) == 1
    for bad in ((0, 2, 4, 2, 128, 0, 3, 100, 0), (6, 2, 4, 3, 128, 0, 3, 100, 0), (6, 2, 4, 2, 100, 0, 3, 100, 0),
                (6, 2, 4, 2, 128, 5, 3, 100, 0), (6, 2, 4, 2, 128, 0, 7, 100, 0), (6, 2, 4, 2, 128, 0, 3, -1, 0)):
        assert lib.w4_tree_attention_workspace_bytes(*bad) == 0, bad


def test_sample_refusals(lib):
    def call(**kw):
        a = dict(x=FAKE, dtype=0, B=2, V=100, stride=100, u=FAKE, tokens=FAKE)
        a.update(kw)
        return lib.w4_sample(a["x"], a["dtype"], a["B"], a["V"], a["stride"], a["u"], None, None, None, None, a["tokens"],
                             None, None)

    for f, status in ((dict(dtype=2), 1), (dict(B=-1), 1), (dict(B=1 << 20), 1), (dict(V=0), 1), (dict(V=1 << 21, stride=1 << 21), 2),
                      (dict(stride=99), 1), (dict(x=None), 1), (dict(x=ctypes.c_void_p(0x1001)), 1), (dict(x=ctypes.c_void_p(0x1002), dtype=1), 1), (dict(u=None), 1), (dict(tokens=None), 1)):
        assert call(**f) == status, f
    assert call(B=0, x=None) == 0


def test_move_refusals(lib):
    def call(cache, **kw):
        a = dict(table=FAKE, pages=5, base=FAKE, path=FAKE, n=4, count=FAKE, B=2)
        a.update(kw)
        return lib.w4_kv_move(ctypes.byref(cache) if cache is not None else None, a["table"], a["pages"], a["base"],
                              a["path"], a["n"], a["count"], a["B"], None)

    for f, status in BAD_CACHES:
        assert call(_cache(**f)) == status, f
    assert call(None) == 1
    for f in (dict(table=None), dict(pages=0), dict(base=None), dict(path=None), dict(count=None), dict(n=-1), dict(B=-1),
              dict(B=1 << 17)):
        assert call(_cache(layers=3), **f) == 1, f
    assert call(_cache(), B=0) == 0 and call(_cache(), n=0, path=None) == 0


def test_binding_refusals():
    """Wrong shapes and types raise ValueError before the library is called (host tensors: nothing could run)."""
    import w4_dequant_gemm_amd as w4
    bf = torch.bfloat16
    k, v = w4.w4_kv_cache(4, 2, 64, 32, device="cpu")
    assert k.shape == (4, 2, 2, 8, 16, 8) and v.shape == (4, 2, 2, 2, 64, 8)
    k8, v8 = w4.w4_kv_cache(4, 2, 64, 32, e4m3=True, layers=3, device="cpu")
    assert k8.shape == (3, 4, 2, 2, 4, 16, 16) and v8.shape == (3, 4, 2, 2, 1, 64, 16) and k8.dtype == torch.uint8
    x = torch.zeros((3, 2, 64), dtype=bf)
    i = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros((1, 4), dtype=torch.int32)
    for bad in ((k[0], v), (k, v[:3]), (k.float(), v.float()), (k8[0], v), (k8, v8), (k, v8[0])):
        with pytest.raises(ValueError):
            w4.w4_kv_append(None, x, x, i, *bad)
        with pytest.raises(ValueError):
            w4.w4_tree_attention(x, *bad, table, i[:1], i[:2], 3, 50)
    with pytest.raises(ValueError, match="device tensor"):
        w4.w4_kv_append(None, x, x, i, k, v)
    with pytest.raises(ValueError, match="logits"):
        w4.w4_sample(torch.zeros(2, 8), torch.zeros(2))
    with pytest.raises(ValueError):
        w4.w4_kv_move(k, v, table, i[:1], table, i[:1])


def test_binding_refuses_other_types_of_one_byte():
    """An 8-bit cache holds OCP E4M3 codes: other types of that size would be read as them."""
    import w4_dequant_gemm_amd as w4
    k, v = w4.w4_kv_cache(4, 2, 64, 32, e4m3=True, device="cpu")
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros((1, 4), dtype=torch.int32)
    for dtype in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.int8, torch.bool):
        bad = k.view(dtype), v.view(dtype)
        with pytest.raises(ValueError, match="E4M3 codes"):
            w4.w4_kv_append(None, x, x, i, *bad, k_scale=i, v_scale=i)
        with pytest.raises(ValueError, match="E4M3 codes"):
            w4.w4_tree_attention(x, *bad, table, i[:1], i[:2], 3, 50, k_scale=i, v_scale=i)
        with pytest.raises(ValueError, match="E4M3 codes"):
            w4.w4_kv_move(*bad, table, i[:1], table, i[:1])
    for dtype in (torch.uint8, torch.float8_e4m3fn):     # these come as far as the pointers
        with pytest.raises(ValueError, match="device tensor"):
            w4.w4_kv_move(k.view(dtype), v.view(dtype), table, i[:1], table, i[:1])


def test_largest_integers_are_refused(lib):
    """Sizes whose sums with other sizes would pass 64 bits."""
    most = (1 << 63) - 1
    for T in (most, most - 15, most - 16, 1 << 62, 1 << 32):
        assert _append(lib, _cache(), T=T) == 1, T
        assert _attend(lib, _cache(), T=T, max_q=3) in (1, 2), T
    for window in (most, most - 66, most - 67, (1 << 29) + 1):
        assert lib.w4_tree_attention_workspace_bytes(6, 2, 4, 2, 128, 0, 3, 100000, window) == 0, window
        assert _attend(lib, _cache(), window=window, pos=FAKE) == 1, window
    for f in (dict(B=most), dict(max_q=most), dict(max_kv=most), dict(pages=most)):
        assert _attend(lib, _cache(), **f) in (1, 2), f
    assert _append(lib, _cache(pages=most)) == 1


def test_cache_sizes_are_not_rounded():
    # a page of 24 tokens is not one of 16
    import w4_dequant_gemm_amd as w4
    for d, page, e4m3 in ((64, 24, False), (64, 0, False), (64, 8, True), (100, 16, False), (72, 16, True), (0, 16, False)):
        with pytest.raises(ValueError, match="multiple"):
            w4.w4_kv_cache(4, 2, d, page, e4m3=e4m3, device="cpu")
