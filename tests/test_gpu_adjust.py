"""w4_adjust_logits on the GPU against the definition in plain fp32 (whose every operation the kernel does alike) and,
as a second reading, in 64 bits."""
import numpy as np
import pytest

from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu


def _reference(logits, dtype64, history, start, prompt, rep, pres, freq, bstart, bids, bvals, mask):
    """Row by row in numpy; dtype64: in 64 bits without the last rounding, else fp32 in the documented order."""
    f = np.float64 if dtype64 else np.float32
    out = logits.astype(f).copy()
    B, V = out.shape
    for b in range(B):
        x = out[b]
        if history is not None:
            lo, hi = max(0, int(start[b])), min(len(history), int(start[b + 1]))
            toks = history[lo:hi].astype(np.int64)
            where = np.arange(lo, hi)
            ok = (toks >= 0) & (toks < V)
            all_ = np.bincount(toks[ok], minlength=V)
            p = 0 if prompt is None else int(prompt[b])
            later = np.bincount(toks[ok & (where >= lo + p)], minlength=V)
            r = f(1 if rep is None else rep[b])
            with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
                x = np.where(all_ > 0, np.where(x > 0, x / r, x * r), x)
                x = np.where(later > 0, x - f(0 if freq is None else freq[b]) * later.astype(f) - f(0 if pres is None else pres[b]), x)
        if bids is not None:
            lo, hi = max(0, int(bstart[b])), min(len(bids), int(bstart[b + 1]))
            last = {}
            for i in range(lo, hi):
                if 0 <= bids[i] < V:
                    last[int(bids[i])] = f(bvals[i])
            for v, y in last.items():
                x[v] = x[v] + y
        if mask is not None:
            m = mask[b if mask.shape[0] > 1 else 0]
            bits = (m.view(np.uint32)[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
            x = np.where(bits == 1, x, f(-np.inf))
        out[b] = x
    return out


def _case(seed, B, V, hist, biases):
    rng = np.random.default_rng(seed)
    lens = [int(rng.integers(0, hist + 1)) for _ in range(B)]
    d = {"logits": (4 * rng.standard_normal((B, V))).astype(np.float32),
         "history": (V * rng.random(sum(lens)) ** 3).astype(np.int32),
         "start": np.concatenate([[0], np.cumsum(lens)]).astype(np.int32),
         "prompt": np.array([rng.integers(0, n + 1) for n in lens], np.int32),
         "rep": rng.choice([1.0, 1.15, 0.8], B).astype(np.float32), "pres": rng.choice([0, 0.5, -0.25], B).astype(np.float32),
         "freq": rng.choice([0, 0.3, -0.1], B).astype(np.float32)}
    n = [int(rng.integers(0, biases + 1)) for _ in range(B)]
    d["bstart"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    d["bids"] = rng.integers(0, V, sum(n)).astype(np.int32)      # (some twice)
    d["bvals"] = (5 * rng.standard_normal(sum(n))).astype(np.float32)
    d["mask"] = (rng.integers(0, 1 << 32, (B, -(-V // 32)), dtype=np.uint64)).astype(np.uint32).view(np.int32)
    return d


def _t(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev())


def _run(d, x, **kw):
    import w4_dequant_gemm_amd as w4
    return w4.w4_adjust_logits(x, history=_t(d["history"]), history_start=_t(d["start"]), prompt_len=_t(d["prompt"]),
                               repetition=_t(d["rep"]), presence=_t(d["pres"]), frequency=_t(d["freq"]),
                               bias_start=_t(d["bstart"]), bias_ids=_t(d["bids"]), bias_values=_t(d["bvals"]),
                               mask=_t(d["mask"]), **kw)


def _want(d, logits, dtype64=False):
    return _reference(logits, dtype64, d["history"], d["start"], d["prompt"], d["rep"], d["pres"], d["freq"], d["bstart"],
                      d["bids"], d["bvals"], d["mask"])


@pytest.mark.parametrize("B,V,hist,biases", [(1, 1, 3, 2), (1, 31, 10, 3), (2, 33, 100, 40), (3, 1000, 0, 0), (5, 4096, 300, 9),
                                             (4, 4097, 2000, 50), (1, 50001, 700, 20), (2, 131072, 60000, 300),
                                             (37, 777, 64, 5), (1, 1 << 20, 5000, 1000), (300, 130, 20, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adjust(B, V, hist, biases, dtype):
    require_gpu()
    import torch
    d = _case(B + V, B, V, hist, biases)
    x = _t(d["logits"]).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    before = x.clone()
    got = _run(d, x)
    assert got.dtype == x.dtype and torch.equal(x, before)
    logits = x.float().cpu().numpy()
    want = torch.from_numpy(_want(d, logits)).to(x.dtype)
    # every operation is one rounding in fp32, in the documented order: the same bits
    assert torch.equal(got.cpu().view(torch.int32 if dtype == "f32" else torch.int16),
                       want.view(torch.int32 if dtype == "f32" else torch.int16))
    exact = _want(d, logits, True)
    fine = np.isfinite(exact)
    off = np.abs(got.double().cpu().numpy()[fine] - exact[fine])
    # five roundings to fp32, each of at most the largest number on the way, and one to the logits' type
    most = np.abs(logits).max() * 1.25 + 0.3 * hist + 0.5 + 40
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    assert (off <= 5 * 2.0 ** -24 * most + half * (np.abs(exact[fine]) + 1e-5 * most)).all()


@pytest.mark.parametrize("left_out", ["history", "prompt", "rep", "pres", "freq", "bids", "mask", "all"])
def test_adjust_without(left_out):
    """Each part may be missing."""
    require_gpu()
    import torch
    d = _case(6, 3, 5000, 400, 30)
    for name in list(d)[1:]:
        if left_out in (name, "all") or (left_out == "history" and name == "start") or (left_out == "bids" and name in ("bstart", "bvals")):
            d[name] = None
    got = _run(d, _t(d["logits"])).cpu()
    assert torch.equal(got, torch.from_numpy(_want(d, d["logits"])))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adjust_strides_place_and_one_for_all(dtype):
    """Strided rows at odd offsets, results in place and between other numbers, one row and one mask for all."""
    require_gpu()
    import torch
    B, V = 4, 9001
    d = _case(2, B, V, 500, 20)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    wide = torch.randn((B, V + 13), device=dev()).to(t)
    x = wide[:, 3:3 + V]
    want = torch.from_numpy(_want(d, x.float().cpu().numpy())).to(t)
    frame = torch.full((B, V + 7), 7.0, device=dev(), dtype=t)
    out = frame[:, 5:5 + V]
    assert _run(d, x, out=out) is out
    assert torch.equal(out.cpu(), want)
    assert (frame[:, :5] == 7).all() and (frame[:, 5 + V:] == 7).all()
    edges = wide[:, :3].clone(), wide[:, 3 + V:].clone()
    assert _run(d, x, out=x) is x and torch.equal(x.cpu(), want)
    assert torch.equal(wide[:, :3], edges[0]) and torch.equal(wide[:, 3 + V:], edges[1])
    one = torch.randn((1, V), device=dev()).to(t)
    d["mask"] = d["mask"][:1]
    got = _run(d, one.expand(B, V))
    assert torch.equal(got.cpu(), torch.from_numpy(_want(d, one.expand(B, V).float().cpu().numpy())).to(t))


def test_adjust_values_without_number():
    """Infinities and NaN among the logits, rows with nothing allowed, tokens and entries outside the vocabulary, and
    starts outside the arrays."""
    require_gpu()
    import torch
    B, V = 4, 300
    d = _case(9, B, V, 80, 10)
    d["logits"][0, :4] = [np.inf, -np.inf, np.nan, 0.0]
    d["history"][:4] = [0, 1, 2, 3]
    d["history"][4:8] = [-1, V, 1 << 30, -(1 << 31)]
    d["start"][1] = max(d["start"][1], 8)
    d["start"][-1] += 1000
    d["bids"] = np.concatenate([d["bids"], [V, -5, 0, 0]]).astype(np.int32)
    d["bvals"] = np.concatenate([d["bvals"], [1, 1, 2, 3]]).astype(np.float32)
    d["bstart"][-1] = len(d["bids"]) + 50
    d["mask"][0] = -1
    d["mask"][1] = 0
    got = _run(d, _t(d["logits"])).cpu().numpy()
    want = _want(d, d["logits"])
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got[0, 2])
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])
    assert (got[1] == -np.inf).all()


def test_adjust_then_sample():
    """A row bound to one token draws it; a row without any draws none."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    V = 5000
    x = torch.randn((3, V), device=dev())
    mask = torch.zeros((3, -(-V // 32)), dtype=torch.int32, device=dev())
    mask[0, 100] = 1 << 7
    mask[2] = -1
    y = w4.w4_adjust_logits(x, mask=mask)
    tokens, probs = w4.w4_sample(y, torch.rand(3, device=dev()), temperature=torch.tensor([1.0, 1.0, 0.0], device=dev()))
    assert tokens.tolist() == [3207, -1, int(x[2].argmax())] and probs[0] == 1.0


def test_adjust_between_the_rows_of_its_logits():
    """Results in the same array, beside the logits of each row or behind all of them."""
    require_gpu()
    import torch
    B, V = 4, 1001
    d = _case(12, B, V, 100, 8)
    wide = torch.randn((B, 2 * V), device=dev())
    want = torch.from_numpy(_want(d, wide[:, :V].cpu().numpy()))
    assert torch.equal(_run(d, wide[:, :V], out=wide[:, V:]).cpu(), want)
    flat = torch.randn((2 * B, V), device=dev())
    for first in (0, B):
        x, out = flat[first:first + B], flat[B - first:2 * B - first]
        want = torch.from_numpy(_want(d, x.cpu().numpy()))
        assert torch.equal(_run(d, x, out=out).cpu(), want)
