"""What the binding of a layer's calls refuses before it calls the library, without a GPU: tensors on another GPU than
the call's, in the form of objects that say they are there."""
import math
import os

import pytest
import torch


class On:
    """A contiguous tensor on a GPU, as far as the binding looks at one."""

    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device = torch.device("cuda", index)

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()

    def numel(self):
        return math.prod(self.shape)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return math.prod(self.shape[i + 1:])

    @property
    def nbytes(self):
        return self.numel() * self.element_size()

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def at(self, index):
        return On(self.shape, self.dtype, index)


BF, I32, F32, U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


@pytest.fixture
def w4(monkeypatch):
    """The binding with GPU 0 current and a library that may be asked for sizes only."""
    import w4_dequant_gemm_amd as w4
    if not os.path.exists(w4.library_path):
        from w4_dequant_gemm_amd import build
        build.build()
    real = w4.lib()

    class Sizes:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return getattr(real, name)

            def called(*args):
                raise AssertionError(f"{name} was called")
            return called

    class NoWay:
        def __getattr__(self, name):
            return lambda *args: None

    monkeypatch.setattr(w4, "lib", lambda: Sizes())
    monkeypatch.setattr(w4, "_call", NoWay())
    monkeypatch.setattr(w4, "_current_device", lambda: 0)
    monkeypatch.setattr(w4, "_raw_stream", lambda i: 0)
    return w4


def _linear(w4, M=200, K=4096, N=96, G=128):
    x, wq, sz = On((M, K), BF), On((N, K // 8), I32), On((N, K // G), I32)
    made = dict(Y=On((M, N), BF), workspace=On((1 << 24,), U8), bias=On((N,), F32), residual=On((M, N), BF))
    codes = dict(xq=On((M, K), U8), xscale=On((M,), F32))
    return [(w4.w4a16_linear, (x, wq, sz, G), made), (w4.w4a8_linear, (x, wq, sz, G), {**made, **codes}),
            (w4.w4a8_linear_e4m3, (codes["xq"], codes["xscale"], wq, sz, G), made)]


def _experts(w4, T=3, k=2, E=20, H=128, I=64, G=64):
    stack = lambda n, kk: {"wq": On((E, n, kk // 8), I32), "sz": On((E, n, kk // G), I32)}     # noqa: E731
    ids, weights = On((T, k), I32), On((T, k), F32)
    return [(w4.w4_route, (On((T, H), BF), On((E, H), BF), k), dict(ids=ids, weights=weights, workspace=On((4096,), U8), bias=On((E,), F32))),
            (w4.w4a16_moe, (On((T, H), BF), ids, weights, stack(I, H), stack(I, H), stack(H, I), G),
             dict(Y=On((T, H), BF), workspace=On((1 << 20,), U8), residual=On((T, H), BF)))]


def _logits(w4, B=3, V=1000):
    i, f = (lambda n: On((n,), I32)), (lambda n: On((n,), F32))
    return [(w4.w4_adjust_logits, (On((B, V), F32),),
             dict(history=i(9), history_start=i(B + 1), prompt_len=i(B), repetition=f(B), presence=f(B), frequency=f(B),
                  bias_start=i(B + 1), bias_ids=i(4), bias_values=f(4), mask=On((B, 32), I32), out=On((B, V), F32)))]


@pytest.mark.parametrize("which", range(6))
def test_tensors_on_another_gpu_are_refused(w4, which):
    f, args, kw = (_linear(w4) + _experts(w4) + _logits(w4))[which]
    with pytest.raises(AssertionError, match="was called"):      # all on GPU 0: it comes to the call
        f(*args, **kw)
    for i, t in enumerate(args):
        if isinstance(t, On):
            with pytest.raises(ValueError, match="cuda:"):
                f(*args[:i], t.at(1), *args[i + 1:], **kw)
        elif isinstance(t, dict):
            for key in t:
                with pytest.raises(ValueError, match="cuda:"):
                    f(*args[:i], {**t, key: t[key].at(1)}, *args[i + 1:], **kw)
    for name, t in kw.items():
        with pytest.raises(ValueError, match="cuda:"):
            f(*args, **{**kw, name: t.at(1)})


@pytest.mark.parametrize("which", range(6))
def test_streams_of_another_gpu_are_refused(w4, which):
    from types import SimpleNamespace
    f, args, kw = (_linear(w4) + _experts(w4) + _logits(w4))[which]
    if which == 1:
        kw.update(xq=On((200, 4096), U8), xscale=On((200,), F32))
    with pytest.raises(AssertionError, match="was called"):
        f(*args, **kw, stream=SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 0)))
    with pytest.raises(ValueError, match="the stream is one of cuda:1"):
        f(*args, **kw, stream=SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1)))


@pytest.mark.parametrize("act", ["relu", None, "tanh", 7])
def test_experts_have_two_activations(w4, act):
    f, args, kw = _experts(w4)[1]
    with pytest.raises(ValueError, match="act must be 'silu' or 'gelu_tanh'"):
        f(*args, act, **kw)
