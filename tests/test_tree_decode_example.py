"""The decoding example end to end: the texts that it writes with and without drafted trees against the same model
in float32 on the dequantized weights."""
import importlib.util
import os

import numpy as np
import pytest

import oracle
from helpers import dev, require_gpu


PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decode.py")


def _example():
    spec = importlib.util.spec_from_file_location("tree_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _weight(lin):
    import torch
    c = {k: v.cpu() for k, v in lin.codes.items()}
    bits = lambda t: t.view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    return torch.from_numpy(oracle.dequant(c["packed"].numpy(), bits(c["scale"]), bits(c["zero"]), lin.G, "asym")).float().to(dev())


def _logits(model, text):
    """[tokens, vocab] of one text, in float32."""
    import torch
    n, d, hq, hk = len(text), model.head_dim, model.heads, model.kv_heads
    norm = lambda x: x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    cos, sin = (model.rope[:n, None, i * d // 2:(i + 1) * d // 2] for i in range(2))

    def turned(x):
        a, b = norm(x).chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    x = model.embed[torch.tensor(text, device=dev())].float()
    for layer in model.layers:
        qkv = (norm(x) @ _weight(layer["qkv"]).T).unflatten(1, (hq + 2 * hk, d))
        q, k, v = turned(qkv[:, :hq]), turned(qkv[:, hq:hq + hk]), qkv[:, hq + hk:]
        k, v = (t.repeat_interleave(hq // hk, 1).transpose(0, 1).contiguous() for t in (k, v))
        s = (q.transpose(0, 1) @ k.transpose(1, 2).contiguous()) * d ** -0.5
        s = s.masked_fill(torch.ones((n, n), dtype=torch.bool, device=dev()).triu(1), -float("inf"))
        x = x + (s.softmax(-1) @ v).transpose(0, 1).flatten(1) @ _weight(layer["o"]).T
        h = norm(x)
        x = x + (torch.nn.functional.silu(h @ _weight(layer["gate"]).T) * (h @ _weight(layer["up"]).T)) @ _weight(layer["down"]).T
    return norm(x) @ _weight(model.out).T


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_tree_decoding_writes_the_text_of_the_model(e4m3):
    require_gpu()
    import torch
    ex = _example()
    model = ex.Model(layers=3)
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, 2048, n).tolist() for n in (40, 1, 23)]
    count = 90
    plain, plain_steps, _ = ex.decode(model, prompts, count, nodes=1, e4m3=e4m3)
    trees, steps, _ = ex.decode(model, prompts, count, nodes=12, e4m3=e4m3)
    assert plain_steps == count - 1 and steps < count // 2
    # Every token has the model's largest logit up to the arithmetic: about 12 bf16 roundings a layer (2^-9 of the
    # value each, independent) leave x with a relative error of about 6 2^-9 = 0.012, a logit (|row| about 1.3) with a
    # deviation of 0.016, a difference of two at six deviations 0.13.  An E4M3 cache adds 2.5 % of a key or value
    # each, at most 4 % of the attention's part a layer: 0.04 in all, or 0.44.
    slack = 0.5 if e4m3 else 0.15
    for texts in (plain, trees):
        for text, prompt in zip(texts, prompts):
            assert len(text) == len(prompt) + count and text[:len(prompt)] == prompt
            x = _logits(model, text[:-1])[len(prompt) - 1:]
            drawn = torch.tensor(text[len(prompt):], device=dev())[:, None]
            assert float((x.amax(1) - x.gather(1, drawn)[:, 0]).max()) <= slack


def test_draft_follows_earlier_occurrences():
    ex = _example()
    tokens, parents, depths = ex.draft([1, 2, 3, 1, 2, 4, 1], 16, 3)
    # the latest first: 2 4 1, then 2 3 1 under the same 2
    assert tokens == [1, 2, 4, 1, 3, 1] and parents == [-1, 0, 1, 2, 1, 4] and depths == [0, 1, 2, 3, 2, 3]
    assert ex.draft([5, 6], 16, 3) == ([6], [-1], [0])
    assert len(ex.draft([1, 2, 3, 1, 2, 4, 1], 3, 3)[0]) == 3
