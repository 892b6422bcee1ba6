"""The products with an epilogue, the mixture-of-experts calls and w4_adjust_logits without a GPU: bad arguments are
refused on the host before any launch."""
import ctypes
import os

import pytest
import torch

FAKE = ctypes.c_void_p(0x1000)          # never dereferenced: the calls below fail their checks or do nothing
ODD = ctypes.c_void_p(0x1008)
SKEW = ctypes.c_void_p(0x1001)
MOST = (1 << 63) - 1


@pytest.fixture(scope="module")
def lib():
    import w4_dequant_gemm_amd as w4
    if not os.path.exists(w4.library_path):
        from w4_dequant_gemm_amd import build
        build.build()
    return w4.lib()


def test_linear_refusals(lib):
    import w4_dequant_gemm_amd as w4

    def a16(**kw):
        a = dict(X=FAKE, M=2, K=96, wq=FAKE, sz=FAKE, N=8, G=32, bias=FAKE, act=1, res=FAKE, Y=FAKE, ws=None, n=0)
        a.update(kw)
        return lib.w4a16_linear(a["X"], a["M"], a["K"], a["wq"], a["sz"], a["N"], a["G"], a["bias"], a["act"], a["res"],
                                a["Y"], a["ws"], a["n"], None)

    def a8(**kw):
        a = dict(X=FAKE, M=2, K=96, wq=FAKE, sz=FAKE, N=8, G=32, bias=FAKE, act=1, res=FAKE, Y=FAKE, xq=FAKE, xs=FAKE,
                 ws=None, n=0)
        a.update(kw)
        return lib.w4a8_linear(a["X"], a["M"], a["K"], a["wq"], a["sz"], a["N"], a["G"], a["bias"], a["act"], a["res"],
                               a["Y"], a["xq"], a["xs"], a["ws"], a["n"], None)

    for call in (a16, a8):
        for f, status in ((dict(act=-1), 1), (dict(act=5), 1), (dict(bias=SKEW), 1), (dict(res=ODD), 1), (dict(X=None), 1),
                          (dict(Y=ODD), 1), (dict(M=-1), 1), (dict(K=100), 1), (dict(G=48), 2), (dict(N=-1), 1),
                          (dict(wq=None), 1), (dict(sz=ODD), 1), (dict(ws=ODD), 1)):
            assert call(**f) == status, f
        assert call(M=0, X=None) == 0 and call(N=0, X=None) == 0
        big = dict(M=256, K=15360, N=3840, G=128)
        assert call(**big) == 1 and "workspace" in w4.w4_last_error()
        need = lib.w4_gemm_workspace_bytes(256, 15360, 3840) if call is a16 else lib.w4a8_gemm_workspace_bytes(256, 15360, 3840)
        assert need > 0
    assert a8(xq=None) == 1 and a8(xs=None) == 1

    def e4m3(**kw):
        a = dict(xq=FAKE, xs=FAKE, M=2, K=96, N=8, G=32, bias=FAKE, act=1, res=FAKE, Y=FAKE, ws=None, n=0)
        a.update(kw)
        return lib.w4a8_linear_e4m3(a["xq"], a["xs"], a["M"], a["K"], FAKE, FAKE, a["N"], a["G"], a["bias"], a["act"], a["res"],
                                    a["Y"], a["ws"], a["n"], None)

    for f in (dict(act=5), dict(act=-1), dict(bias=SKEW), dict(res=ODD), dict(xq=None), dict(xs=None), dict(Y=None), dict(M=-1)):
        assert e4m3(**f) == 1, f
    assert e4m3(M=0, xq=None) == 0


def test_route_refusals(lib):
    def call(**kw):
        a = dict(X=FAKE, T=3, H=64, R=FAKE, E=20, k=2, score=0, bias=None, re=1, scale=1.0, ids=FAKE, w=FAKE, ws=FAKE, n=240)
        a.update(kw)
        return lib.w4_route(a["X"], a["T"], a["H"], a["R"], a["E"], a["k"], a["score"], a["bias"], a["re"], a["scale"],
                            a["ids"], a["w"], a["ws"], a["n"], None)

    for f, status in ((dict(T=-1), 1), (dict(T=MOST), 1), (dict(H=0), 1), (dict(H=60), 1), (dict(H=MOST - 7), 1), (dict(E=0), 1),
                      (dict(E=2000), 2), (dict(E=MOST), 2), (dict(k=0), 1), (dict(k=21), 1), (dict(E=64, k=33), 2), (dict(score=2), 1),
                      (dict(scale=float("nan")), 1), (dict(X=None), 1), (dict(X=ODD), 1), (dict(R=None), 1), (dict(R=ODD), 1),
                      (dict(ids=None), 1), (dict(w=None), 1), (dict(ws=None), 1), (dict(ws=ODD), 1), (dict(n=239), 1)):
        assert call(**f) == status, f
    assert call(T=0, X=None, ws=None) == 0
    assert lib.w4_route_workspace_bytes(3, 64, 20) == 240
    assert lib.w4_route_workspace_bytes(3, 64, 8) == 0                 # one kernel
    assert lib.w4_route_workspace_bytes(3, 4096, 8) == 8 * 96          # eight ranges of 512 k
    for bad in ((0, 64, 8), (-1, 64, 8), (3, 64, 0), (3, 64, MOST), (MOST, 64, 8), (3, 0, 8), (3, 60, 8), (3, MOST - 7, 8)):
        assert lib.w4_route_workspace_bytes(*bad) == 0, bad


def test_moe_refusals(lib):
    import w4_dequant_gemm_amd as w4
    need = lib.w4a16_moe_workspace_bytes(3, 2, 8, 128, 64, 64)
    assert need > 0

    def call(**kw):
        a = dict(X=FAKE, T=3, H=128, ids=FAKE, w=FAKE, k=2, p=[FAKE] * 6, E=8, I=64, G=64, act=1, res=None,
                 Y=ctypes.c_void_p(0x2000), ws=FAKE, n=need)
        a.update(kw)
        return lib.w4a16_moe(a["X"], a["T"], a["H"], a["ids"], a["w"], a["k"], *a["p"], a["E"], a["I"], a["G"], a["act"],
                             a["res"], a["Y"], a["ws"], a["n"], None)

    for f, status in ((dict(T=-1), 1), (dict(T=MOST), 1), (dict(H=0), 1), (dict(H=96), 1), (dict(H=MOST), 1), (dict(I=0), 1),
                      (dict(I=32), 1), (dict(I=1 << 40), 1), (dict(G=128), 1), (dict(G=48), 2), (dict(G=0), 2), (dict(E=0), 1),
                      (dict(E=1025), 2), (dict(k=0), 1), (dict(k=33), 2), (dict(act=0), 1), (dict(act=3), 1),
                      (dict(X=None), 1), (dict(X=ODD), 1), (dict(ids=None), 1), (dict(w=None), 1), (dict(res=ODD), 1),
                      (dict(Y=None), 1), (dict(Y=ODD), 1), (dict(Y=FAKE), 1), (dict(ws=None), 1), (dict(ws=ODD), 1),
                      (dict(n=need - 1), 1)):
        assert call(**f) == status, f
    for i in range(6):
        for bad in (None, ODD):
            assert call(p=[FAKE] * i + [bad] + [FAKE] * (5 - i)) == 1
    assert call(n=need - 1) == 1 and "w4a16_moe_workspace_bytes" in w4.w4_last_error()
    assert call(T=0, X=None, ws=None) == 0
    for bad in ((0, 2, 8, 128, 64, 64), (3, 0, 8, 128, 64, 64), (3, 2, 0, 128, 64, 64), (3, 2, 8, 96, 64, 64),
                (3, 2, 8, 128, 64, 48), (MOST, 2, 8, 128, 64, 64), (3, 2, MOST, 128, 64, 64), (3, 2, 8, MOST, 64, 64)):
        assert lib.w4a16_moe_workspace_bytes(*bad) == 0, bad


def test_adjust_refusals(lib):
    def call(**kw):
        a = dict(x=FAKE, dtype=0, B=2, V=100, xs=100, h=FAKE, hn=9, hs=FAKE, pl=None, rep=None, pres=None, freq=None, bs=FAKE,
                 bi=FAKE, bv=FAKE, bn=4, mask=FAKE, ms=4, out=ctypes.c_void_p(0x3000), os=100)
        a.update(kw)
        return lib.w4_adjust_logits(a["x"], a["dtype"], a["B"], a["V"], a["xs"], a["h"], a["hn"], a["hs"], a["pl"], a["rep"],
                                    a["pres"], a["freq"], a["bs"], a["bi"], a["bv"], a["bn"], a["mask"], a["ms"], a["out"],
                                    a["os"], None)

    for f, status in ((dict(dtype=2), 1), (dict(B=-1), 1), (dict(B=1 << 16), 1), (dict(V=0), 1), (dict(V=MOST, xs=MOST, os=MOST), 2),
                      (dict(V=(1 << 20) + 1, xs=1 << 21, os=1 << 21), 2), (dict(xs=99), 1), (dict(xs=MOST), 1), (dict(os=99), 1),
                      (dict(os=0), 1), (dict(os=MOST), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(x=SKEW), 1),
                      (dict(x=ctypes.c_void_p(0x1002), dtype=1), 1), (dict(out=ctypes.c_void_p(0x1002), dtype=1), 1),
                      (dict(hs=None), 1), (dict(h=None), 1), (dict(hn=-1), 1), (dict(hn=1 << 31), 1), (dict(bn=1 << 31), 1),
                      (dict(bn=-1), 1), (dict(bs=None), 1), (dict(bi=None), 1), (dict(bv=None), 1), (dict(ms=3), 1),
                      (dict(ms=-1), 1), (dict(ms=MOST), 1), (dict(out=FAKE, os=101), 1), (dict(out=FAKE, xs=0), 1)):
        assert call(**f) == status, f
    assert call(B=0, x=None, out=None) == 0


def test_binding_refusals():
    """Wrong shapes and types raise ValueError before the library is called (host tensors: nothing could run)."""
    import w4_dequant_gemm_amd as w4
    bf = torch.bfloat16
    N, K, G, M = 64, 256, 128, 3
    X = torch.zeros((M, K), dtype=bf)
    wq, sz = torch.zeros((N, K // 8), dtype=torch.int32), torch.zeros((N, K // G), dtype=torch.int32)
    for f in (w4.w4a16_linear, w4.w4a8_linear):
        with pytest.raises(ValueError, match="act must"):
            f(X, wq, sz, G, act="tanh")
        with pytest.raises(ValueError, match="residual has shape"):
            f(X, wq, sz, G, residual=torch.zeros((M, N + 1), dtype=bf))
        with pytest.raises(ValueError, match="bias has"):
            f(X, wq, sz, G, bias=torch.zeros(N + 1))
        with pytest.raises(ValueError, match="wq holds"):
            f(X[:, :128].contiguous(), wq, sz, G)
        with pytest.raises(ValueError, match="device tensor"):
            f(X, wq, sz, G)
    r = torch.zeros((8, K), dtype=bf)
    for bad in (dict(X=X[0]), dict(router=r[:, :8]), dict(score="relu"), dict(bias=torch.zeros(7)), dict(router=r.float())):
        a = dict(X=X, router=r, top_k=2)
        a.update(bad)
        with pytest.raises(ValueError):
            w4.w4_route(**a)
    with pytest.raises(ValueError, match="device tensor"):
        w4.w4_route(X, r, 2)
    stack = lambda n, k: {"wq": torch.zeros((8, n, k // 8), dtype=torch.int32), "sz": torch.zeros((8, n, k // G), dtype=torch.int32)}  # noqa: E731
    ids, ws = torch.zeros((M, 2), dtype=torch.int32), torch.zeros((M, 2))
    good = dict(X=X, ids=ids, weights=ws, gate=stack(N * 2, K), up=stack(N * 2, K), down=stack(K, N * 2), G=G)
    for bad, text in ((dict(ids=ids[:2]), "top_k"), (dict(weights=ws[:, :1]), "top_k"), (dict(G=96), "multiples"),
                      (dict(up=stack(N * 4, K)), "up holds"), (dict(down=stack(N * 2, K * 2)), "down holds"),
                      (dict(residual=X[:2]), "residual has shape"), (dict(Y=X[:, :8]), "Y has shape"),
                      (dict(gate={k: v[0] for k, v in stack(N * 2, K).items()}), "gate wq must"), ({}, "device tensor")):
        with pytest.raises(ValueError, match=text):
            w4.w4a16_moe(**{**good, **bad})
    with pytest.raises(ValueError, match="logits"):
        w4.w4_adjust_logits(torch.zeros(2, 8))


def test_results_on_their_inputs_are_refused(lib):
    """A product's result in place of its activations, and logits that partly lie on their own results: refused.  (In
    place of the logits, between their rows, and on the residual is allowed: tested where it runs.)"""
    import w4_dequant_gemm_amd as w4
    place = ctypes.c_void_p(0x2000)
    for call in (lambda: lib.w4a16_linear(place, 2, 96, FAKE, FAKE, 96, 32, None, 0, place, place, None, 0, None),
                 lambda: lib.w4a8_linear(place, 2, 96, FAKE, FAKE, 96, 32, None, 0, None, place, FAKE, FAKE, None, 0, None),
                 lambda: lib.w4a8_linear_e4m3(place, FAKE, 2, 96, FAKE, FAKE, 96, 32, None, 0, None, place, None, 0, None)):
        assert call() == 1 and "Y must not be X" in w4.w4_last_error()

    def adjust(B, V, xs, os, shift, dtype=0):
        size = 4 if dtype else 2
        return lib.w4_adjust_logits(ctypes.c_void_p(0x100000), dtype, B, V, xs, None, 0, None, None, None, None, None, None, None,
                                    None, 0, None, 0, ctypes.c_void_p(0x100000 + size * shift), os, None)

    for dtype in (0, 1):
        for a in ((1, 100, 100, 100, 1), (1, 100, 500, 100, 99), (1, 100, 100, 100, -99), (4, 100, 250, 250, 99),
                  (4, 100, 250, 250, 151), (4, 100, 250, 250, 250), (4, 100, 250, 250, -250), (4, 100, 250, 250, 750),
                  (4, 100, 250, 250, 849), (4, 100, 250, 250, -849), (3, 100, 100, 100, 200), (3, 100, 100, 100, -101)):
            assert adjust(*a, dtype=dtype) == 1 and "overlaps" in w4.w4_last_error(), a


def test_logits_of_one_row_or_other_strides_on_their_results_are_refused(lib):
    """One row of logits for all, or rows of logits and results not equally far apart: refused where any row of the
    results shares an element with one of the logits, against a list of the elements."""
    import random

    import w4_dequant_gemm_amd as w4
    base = 0x100000

    def refused(B, V, xs, os, shift, dtype):
        # (a length of no array is refused behind the overlap, so nothing runs on these addresses)
        size = 4 if dtype else 2
        assert lib.w4_adjust_logits(ctypes.c_void_p(base), dtype, B, V, xs, None, 0, None, None, None, None, None, None, None,
                                    None, 1, None, 0, ctypes.c_void_p(base + size * shift), os, None) == 1
        assert "overlaps" in w4.w4_last_error() or "bias_len" in w4.w4_last_error()
        return "overlaps" in w4.w4_last_error()

    def meets(B, V, xs, os, shift):
        given = {i * xs + v for i in range(B) for v in range(V)}
        return any(shift + j * os + v in given for j in range(B) for v in range(V))

    # the second of the results' rows is the logits' one row; rows 100 apart against rows 130 apart
    for a in ((3, 100, 0, 100, -100), (3, 100, 0, 100, 99), (3, 100, 0, 250, -599), (3, 100, 130, 100, -150), (3, 100, 130, 100, 100),
              (2, 100, 100, 400, -301), (2, 100, 400, 100, 301)):
        assert meets(*a), a
        for dtype in (0, 1):
            assert refused(*a, dtype), a
    rng = random.Random(3)
    both = [0, 0]
    for _ in range(400):
        B, V = rng.randint(1, 6), rng.randint(1, 9)
        xs, os = rng.choice([0, V + rng.randint(0, 30)]), V + rng.randint(0, 30)
        shift = rng.randint(-200, 200)
        if shift == 0:
            continue
        met = meets(B, V, xs, os, shift)
        both[met] += 1
        assert refused(B, V, xs, os, shift, 1) == met, (B, V, xs, os, shift)
    assert min(both) > 40


def test_products_whose_results_overlap_their_inputs_are_refused(lib):
    """Y on a part of X or of the residual, and codes or scales on a part of X, Y, the residual or each other."""
    import w4_dequant_gemm_amd as w4
    M, K, N, G = 4, 96, 64, 32
    at = lambda a: ctypes.c_void_p(a)                                       # noqa: E731
    # places far apart: X 4 x 96 x 2 bytes = 768, Y and the residual 512, codes 384, scales 16
    far = dict(X=0x10000, res=0x20000, Y=0x30000, xq=0x40000, xs=0x50000)

    def a16(X, res, Y, xq, xs):
        return lib.w4a16_linear(at(X), M, K, FAKE, FAKE, N, G, None, 1, at(res), at(Y), None, 0, None)

    def a8(X, res, Y, xq, xs):
        return lib.w4a8_linear(at(X), M, K, FAKE, FAKE, N, G, None, 1, at(res), at(Y), at(xq), at(xs), None, 0, None)

    def e4m3(X, res, Y, xq, xs):
        return lib.w4a8_linear_e4m3(at(X), at(xs), M, K, FAKE, FAKE, N, G, None, 1, at(res), at(Y), None, 0, None)

    def refused(call, text, **places):
        assert call(**{**far, **places}) == 1 and text in w4.w4_last_error(), (places, w4.w4_last_error())

    for call, x_bytes in ((a16, 768), (a8, 768), (e4m3, 384)):
        for shift in (16, x_bytes - 16, -16, 16 - 512):
            refused(call, "Y overlaps X", Y=far["X"] + shift)
        for shift in (16, 512 - 16, -16, 16 - 512):
            refused(call, "Y overlaps the residual", Y=far["res"] + shift)
        refused(call, "Y must not be X", Y=far["X"], res=far["X"])
    for name, text, n in (("X", "X", 768), ("Y", "Y", 512), ("res", "the residual", 512)):
        for shift in (16, n - 16, 16 - 384):
            refused(a8, f"xq overlaps {text}", xq=far[name] + shift)
        refused(a8, f"xq must not be {text}", xq=far[name])
        for shift in (4, n - 4, -12):
            refused(a8, f"xscale overlaps {text}", xs=far[name] + shift)
    refused(a8, "xscale overlaps xq", xs=far["xq"] + 380)
    refused(a8, "xscale overlaps xq", xs=far["xq"] - 12)
    # the bias, which all rows read, and the scales of ready codes
    for shift in (0, 16, -16):
        assert lib.w4a16_linear(at(far["X"]), M, K, FAKE, FAKE, N, G, at(far["Y"] - shift), 1, None, at(far["Y"]), None, 0, None) == 1
        refused(e4m3, "xscale", xs=far["Y"] + max(shift, 0))


def test_experts_whose_results_overlap_their_inputs_are_refused(lib):
    """Y or the workspace on a part of what the call reads."""
    import w4_dequant_gemm_amd as w4
    T, k, E, H, I, G = 3, 2, 8, 128, 64, 64
    need = lib.w4a16_moe_workspace_bytes(T, k, E, H, I, G)
    at = lambda a: ctypes.c_void_p(a)                                       # noqa: E731
    far = dict(X=0x10000, ids=0x20000, w=0x30000, res=0x40000, Y=0x50000, ws=0x100000)

    def refused(text, **places):
        a = {**far, **places}
        status = lib.w4a16_moe(at(a["X"]), T, H, at(a["ids"]), at(a["w"]), k, *[FAKE] * 6, E, I, G, 1, at(a["res"]), at(a["Y"]),
                               at(a["ws"]), need, None)
        assert status == 1 and text in w4.w4_last_error(), (places, w4.w4_last_error())

    rows = T * H * 2
    for name, text, n in (("X", "X", rows), ("res", "the residual", rows), ("ids", "ids", 24), ("w", "weights", 24)):
        for shift in (16, 16 - rows):
            refused(f"Y overlaps {text}", Y=far[name] + shift)
            refused(f"the workspace overlaps {text}", ws=far[name] + 16 - need // 16 * 16)
        if name != "res":
            refused(f"Y must not be {text}", Y=far[name], res=far[name] if name == "X" else far["res"])
        refused(f"the workspace must not be {text}", ws=far[name])
    refused("the workspace must not be Y", ws=far["Y"])
    refused("the workspace overlaps Y", ws=far["Y"] + rows - 16)


def test_routing_whose_results_overlap_its_inputs_is_refused(lib):
    import w4_dequant_gemm_amd as w4
    T, H, E, k = 3, 64, 20, 2
    need = lib.w4_route_workspace_bytes(T, H, E)
    assert need == 240
    at = lambda a: ctypes.c_void_p(a)                                       # noqa: E731
    far = dict(X=0x10000, R=0x20000, bias=0x30000, ids=0x40000, w=0x50000, ws=0x60000)

    def refused(text, **places):
        a = {**far, **places}
        status = lib.w4_route(at(a["X"]), T, H, at(a["R"]), E, k, 0, at(a["bias"]), 1, 1.0, at(a["ids"]), at(a["w"]), at(a["ws"]),
                              need, None)
        assert status == 1 and text in w4.w4_last_error(), (places, w4.w4_last_error())

    for name, text, n in (("X", "X", T * H * 2), ("R", "router", E * H * 2), ("bias", "bias", 80)):
        for shift in (4, n - 4, -20):
            refused(f"ids overlaps {text}", ids=far[name] + shift)
            refused(f"weights overlaps {text}", w=far[name] + shift)
        for shift in (16, n - 16, 16 - need):
            refused(f"the workspace overlaps {text}", ws=far[name] + shift)
    refused("ids must not be weights", w=far["ids"])
    refused("ids overlaps weights", w=far["ids"] + 20)
    refused("the workspace overlaps ids", ws=far["ids"] + 16)
    refused("the workspace overlaps weights", ws=far["w"] - 224)
