"""The compiled way that the binding takes for its usual calls gives what the other way gives, and takes none of the
calls that the other way refuses."""
import pytest

from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu


class _Counted:
    """The compiled functions, with how many calls each took and how many it left."""

    def __init__(self, module):
        self._module, self.took, self.left = module, {}, {}

    def __getattr__(self, name):
        f = getattr(self._module, name)

        def call(*args):
            r = f(*args)
            which = self.left if r is None else self.took
            which[name] = which.get(name, 0) + 1
            return r
        return call


class _Absent:
    def __getattr__(self, name):
        return lambda *args: None


def _weights(w4, gen, N, K, G):
    import torch
    q = w4.w4_quantize_blockwise(torch.randn((N, K), generator=gen, device=dev()) * 0.05, G, "asym")
    return w4.w4_prepack(q["packed"], q["scale"], q["zero"], G, "asym")


def _inputs():
    import torch
    import w4_dequant_gemm_amd as w4
    gen = torch.Generator(device=dev()).manual_seed(5)
    T, E, k, H, I, G, V, B = 3, 5, 2, 128, 256, 32, 1000, 4
    bf = lambda *s: torch.randn(s, generator=gen, device=dev()).to(torch.bfloat16)      # noqa: E731
    stack = lambda N, K: {key: torch.stack([p[key] for p in ps]) for ps in                # noqa: E731
                          [[_weights(w4, gen, N, K, G) for _ in range(E)]] for key in ("wq", "sz")}
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev())                   # noqa: E731
    f = lambda n: torch.rand((n,), generator=gen, device=dev())                          # noqa: E731
    return dict(x=bf(T, H), w=_weights(w4, gen, I, H, G), lbias=f(I), lres=bf(T, I), G=G, router=bf(E, H), pick=f(E), k=k,
                ids=ints(0, 4, 2, 2, 7, 1).view(T, k), wt=f(T * k).view(T, k), gate=stack(I, H), up=stack(I, H),
                down=stack(H, I), res=bf(T, H), logits=bf(B, V), history=ints(1, 1, 999, 3, 4, 4, 5, 4),
                hs=ints(0, 3, 3, 7, 8), pl=ints(1, 0, 2, 1), rep=1 + f(B), pres=f(B), freq=f(B), bs=ints(0, 1, 1, 2, 3),
                bi=ints(5, 6, 7), bv=f(3), mask=torch.randint(-2**31, 2**31 - 1, (B, 32), dtype=torch.int32, generator=gen,
                                                              device=dev()))


def _calls(w4, d):
    """Name, the compiled function, a call that it takes."""
    adjust = dict(history=d["history"], history_start=d["hs"], prompt_len=d["pl"], repetition=d["rep"], presence=d["pres"],
                  frequency=d["freq"], bias_start=d["bs"], bias_ids=d["bi"], bias_values=d["bv"], mask=d["mask"])
    lin = lambda f, **o: (lambda: f(d["x"], d["w"]["wq"], d["w"]["sz"], d["G"], **o))     # noqa: E731
    moe = lambda **o: (lambda: w4.w4a16_moe(d["x"], d["ids"], d["wt"], d["gate"], d["up"], d["down"], d["G"], **o))  # noqa: E731
    return {
        "linear": ("linear", lin(w4.w4a16_linear)),
        "linear all": ("linear", lin(w4.w4a16_linear, bias=d["lbias"], act="silu", residual=d["lres"])),
        "linear a8": ("linear", lin(w4.w4a8_linear, bias=d["lbias"], act="relu")),
        "linear a8 all": ("linear", lin(w4.w4a8_linear, bias=d["lbias"], act="gelu", residual=d["lres"])),
        "route": ("route", lambda: w4.w4_route(d["x"], d["router"], d["k"])),
        "route all": ("route", lambda: w4.w4_route(d["x"], d["router"], d["k"], score="sigmoid", bias=d["pick"],
                                                   renormalize=False, scale=2.5)),
        "moe": ("moe", moe()),
        "moe residual": ("moe", moe(act="gelu_tanh", residual=d["res"])),
        "adjust": ("adjust", lambda: w4.w4_adjust_logits(d["logits"])),
        "adjust all": ("adjust", lambda: w4.w4_adjust_logits(d["logits"], **adjust)),
        "adjust fp32": ("adjust", lambda: w4.w4_adjust_logits(d["logits"].float(), **adjust)),
        "adjust one mask": ("adjust", lambda: w4.w4_adjust_logits(d["logits"], mask=d["mask"][:1])),
        "adjust no history": ("adjust", lambda: w4.w4_adjust_logits(d["logits"], history=d["history"][:0],
                                                                    history_start=d["hs"] * 0, repetition=d["rep"])),
    }


def _flat(r):
    import torch
    return [r] if torch.is_tensor(r) else list(r)


@pytest.mark.parametrize("name", ["linear", "linear all", "linear a8", "linear a8 all", "route", "route all", "moe",
                                  "moe residual", "adjust", "adjust all", "adjust fp32", "adjust one mask",
                                  "adjust no history"])
def test_both_ways_agree(name, monkeypatch):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    method, call = _calls(w4, _inputs())[name]
    counted = _Counted(w4._short())
    monkeypatch.setattr(w4, "_call", counted)
    got = _flat(call())
    assert counted.took == {method: 1} and not counted.left
    monkeypatch.setattr(w4, "_call", _Absent())
    want = _flat(call())
    torch.cuda.synchronize()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.shape == b.shape and a.dtype == b.dtype and a.device == b.device and a.is_contiguous()
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# one input replaced: by one elsewhere, of another type, not contiguous, of another size
_BROKEN = {"cpu": lambda t: t.cpu(), "type": lambda t: t.double() if t.is_floating_point() else t.long(),
           "stride": lambda t: __import__("torch").stack([t, t], dim=-1)[..., 0], "size": lambda t: t[..., :-1].contiguous()}


@pytest.mark.parametrize("how", list(_BROKEN))
@pytest.mark.parametrize("name,keys", [("linear all", ["x", "lbias", "lres"]), ("linear a8 all", ["x", "lbias", "lres"]),
                                       ("route all", ["x", "router", "pick"]), ("moe residual", ["x", "ids", "wt", "res"]),
                                       ("adjust all", ["hs", "pl", "rep", "pres", "freq", "bs", "bv", "mask"])])
def test_what_is_refused_stays_refused(name, keys, how):
    require_gpu()
    import w4_dequant_gemm_amd as w4
    for key in keys:
        d = _inputs()
        d[key] = _BROKEN[how](d[key])
        with pytest.raises((ValueError, w4.W4Error)):
            _calls(w4, d)[name][1]()


@pytest.mark.parametrize("how", list(_BROKEN))
@pytest.mark.parametrize("part", ["wq", "sz"])
def test_weights_are_refused(part, how):
    require_gpu()
    import w4_dequant_gemm_amd as w4
    for key, name in (("w", "linear"), ("w", "linear a8"), ("gate", "moe"), ("up", "moe"), ("down", "moe")):
        d = _inputs()
        d[key] = dict(d[key], **{part: _BROKEN[how](d[key][part])})
        with pytest.raises((ValueError, w4.W4Error)):
            _calls(w4, d)[name][1]()


def test_arguments_are_refused():
    require_gpu()
    import w4_dequant_gemm_amd as w4
    d = _inputs()
    w = d["w"]
    refused = (ValueError, TypeError, w4.W4Error, __import__("ctypes").ArgumentError)
    for call in (lambda: w4.w4a16_linear(d["x"], w["wq"], w["sz"], 48), lambda: w4.w4a16_linear(d["x"], w["wq"], w["sz"], 0),
                 lambda: w4.w4a16_linear(d["x"], w["wq"], w["sz"], 32, act="tanh"),
                 lambda: w4.w4_route(d["x"], d["router"], 0), lambda: w4.w4_route(d["x"], d["router"], 6),
                 lambda: w4.w4_route(d["x"], d["router"], 2, score="none"), lambda: w4.w4_route(d["x"], d["router"], 2.5),
                 lambda: w4.w4a16_moe(d["x"], d["ids"], d["wt"], d["gate"], d["up"], d["down"], 64),
                 lambda: w4.w4a16_moe(d["x"], d["ids"], d["wt"], d["gate"], d["up"], d["down"], -32),
                 lambda: w4.w4_adjust_logits(d["logits"], history=d["history"]),
                 lambda: w4.w4_adjust_logits(d["logits"], bias_ids=d["bi"], bias_start=d["bs"])):
        with pytest.raises(refused):
            call()


def test_results_are_from_the_current_stream():
    """On a side stream the compiled way works there, and its results are that stream's memory."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    d = _inputs()
    calls = _calls(w4, d)
    side = torch.cuda.Stream()
    for name in ("linear all", "linear a8 all", "route all", "moe residual", "adjust all"):
        want = [t.clone() for t in _flat(calls[name][1]())]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = _flat(calls[name][1]())
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
