"""w4_route where the chosen scores themselves leave the range of 32 bits: their shares, which do not, against the
definition in 64 bits."""
import pytest

from helpers import dev, require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _layer(logits, H=64):
    """Tokens and a router whose logits are exactly the rows given (bf16 numbers): one value a token, times one."""
    import torch
    logits = torch.as_tensor(logits, dtype=torch.float64, device=dev())
    assert torch.equal(logits.to(torch.bfloat16).double(), logits)
    T, E = logits.shape
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=dev())
    r = torch.zeros((E, H), dtype=torch.bfloat16, device=dev())
    for t in range(T):
        x[t, t] = 1.0
        r[:, t] = logits[t].to(torch.bfloat16)
    return x, r, logits


def _shares(logits, ids, score):
    """s_j / sum s of the choices, from the logits in 64 bits by logarithms."""
    import torch
    log = torch.nn.functional.logsigmoid(logits) if score == "sigmoid" else torch.log_softmax(logits, 1)
    log = log.gather(1, ids.long())
    return torch.softmax(log, 1)


# sizes of one launch, of two, and of each number of experts a lane holds
@pytest.mark.parametrize("E,k", [(5, 5), (16, 3), (40, 8), (100, 6), (200, 32), (700, 7)])
@pytest.mark.parametrize("bias", [False, True])
def test_sigmoid_scores_of_far_negative_logits(E, k, bias):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    g = torch.Generator(device=dev()).manual_seed(E)
    # from logits whose scores are whole numbers of 32 bits to ones that are none: no row mixes both sides of a wide gap
    base = torch.tensor([-10.0, -40, -41, -42, -44, -60, -80, -87, -88, -89, -95, -104, -110, -150, -1000, -30000], device=dev())
    far = (-4 * torch.rand((16, E), generator=g, device=dev()) + base[:, None]).to(torch.bfloat16).double()
    x, r, logits = _layer(far)
    b = torch.rand(E, generator=g, device=dev()) if bias else None
    for scale in (1.0, 2.5):
        ids, weights = w4.w4_route(x, r, k, score="sigmoid", bias=b, scale=scale)
        # the scores vanish beside a bias: it alone chooses
        want = (torch.sigmoid(logits) + b.double() if bias else logits).sort(dim=1, descending=True, stable=True).indices[:, :k]
        if not bias:
            assert torch.equal(ids.long(), want)
        share = _shares(logits, ids, "sigmoid") * scale
        # exponents of at most 42 from logits that are exact; sums of 32, a division, a factor
        assert ((weights.double() - share).abs() <= (2 * 42 + 2 * k + 16) * U * share + scale * 2.0 ** -58).all()
        assert ((weights.double().sum(1) - scale).abs() <= (k + 8) * U * scale).all()


@pytest.mark.parametrize("E,k", [(6, 2), (30, 4), (130, 5)])
def test_softmax_scores_that_a_bias_chose_far_below_the_largest(E, k):
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    g = torch.Generator(device=dev()).manual_seed(E)
    below = torch.tensor([0.0, -30, -45, -86, -90, -104, -120, -300, -2000], device=dev())
    logits = (-3 * torch.rand((9, E), generator=g, device=dev()) + below[:, None]).to(torch.bfloat16).double()
    logits[:, 0] = 8.0
    b = torch.rand(E, generator=g, device=dev())
    b[0] = -4.0                                              # the largest logit is never chosen
    x, r, logits = _layer(logits)
    ids, weights = w4.w4_route(x, r, k, bias=b)
    assert (ids > 0).all()
    share = _shares(logits, ids, "softmax")
    # (a softmax score of l is off by the rounding of l - top, at most 128 here until the shares are made without it)
    assert ((weights.double() - share).abs() <= (2 * 128 + 2 * E + 16) * U * share + 2.0 ** -58).all()


def test_choices_without_a_number_beside_far_ones():
    """A choice of -inf or NaN has nothing, the others share; none but such: no weight, as before."""
    require_gpu()
    import torch
    import w4_dequant_gemm_amd as w4
    inf = float("inf")
    x, r, _ = _layer([[-200.0, -201, -256, -300]])
    r[1, 0], r[3, 0] = -inf, float("nan")
    ids, weights = w4.w4_route(x, r, 4, score="sigmoid")
    assert ids.tolist() == [[0, 2, 1, 3]] and weights.tolist() == [[1.0, pytest.approx(4.780892883885469e-25, rel=1e-6), 0.0, 0.0]]
    r[:, 0] = -inf
    ids, weights = w4.w4_route(x, r, 3, score="sigmoid")
    assert ids.tolist() == [[0, 1, 2]] and not weights.any()
