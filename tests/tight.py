"""How far results may be from the 64-bit ones on the whole: the root mean square of the error, set against that of the
result.  A worst case over long sums allows any one output far more than its errors ever add up to; these limits count
errors that do not conspire, and what a kernel leaves out or computes otherwise stands out against them.

The roundings.  A number rounded to bf16 is off by at most half a step, evenly spread over the step of 2^-7 of its power of
two: 2^-7 / sqrt(12) = 0.00226 of the power of two in the root mean square, and of the number itself at most that.  With
the result so rounded, nothing smaller than 0.00226 could be seen; so a call is made again with its first result as a
negative residual, and what is left, some 0.002 of the result, is rounded to 0.002 of itself.

Sums of products with 128 + u pass through s (256 + 2 |z|) |x| a term.  Each of the roundings in a chain is off by at most
U = 2^-24 of a partial sum, whose root mean square is that of its terms times the square root of their number."""
import torch

U = 2.0 ** -24
STEP = 2.0 ** -7 / 12 ** 0.5          # root mean square of a rounding to bf16, of the number's power of two
TWICE = 2.0 ** -8 * 2.0 ** -8         # the most that is left of h = hi + lo


def rms(x):
    return x.double().pow(2).mean().sqrt().item()


# T, choices, experts, hidden, inner, group: every form of the experts' call, long and short sums, ends inside steps
MOE = [
    (1, 2, 4, 64, 32, 32), (1, 8, 8, 256, 128, 128), (3, 1, 2, 128, 128, 64), (5, 4, 16, 576, 1536, 32), (7, 2, 4, 192, 320, 64),
    (16, 2, 4, 256, 384, 128), (17, 3, 5, 288, 96, 32), (33, 8, 40, 512, 256, 128), (70, 2, 3, 320, 192, 64),
    (2, 32, 32, 128, 128, 128), (64, 1, 64, 256, 128, 64), (2, 8, 64, 512, 320, 64), (1, 2, 4, 256, 14336, 128), (2, 4, 9, 8192, 96, 32),
    (52, 2, 8, 64, 4352, 32), (52, 2, 8, 64, 4352, 64), (52, 2, 8, 128, 4352, 128), (14, 4, 4, 64, 8320, 32), (60, 2, 9, 256, 384, 128),
    (100, 2, 4, 128, 128, 128), (200, 6, 16, 384, 640, 128), (90, 3, 3, 256, 4096, 128), (65, 1, 1, 4096, 256, 128),
    (100, 2, 4, 64, 192, 64), (130, 1, 2, 576, 1536, 64), (200, 3, 5, 96, 160, 32), (90, 2, 2, 576, 1536, 32), (100, 2, 4, 128, 14336, 64),
]


def tiled(T, k, E, H, I, G):
    """Whether the experts' call takes the tiles, which keep h as one bf16 number."""
    wide = max(H, I)
    return T * k > 64 and T * k >= 16 * E and -(-wide // 128) * (128 // G) * 64 <= 16384 and 2 * T * k * wide < 2 ** 31


def moe_limit(shape, once=None):
    """Root mean square of the error over that of the result, the result's own rounding taken off.  h is off by STEP or
    TWICE of itself, term by term; the first product's sums and the second's by U times what passes through (40 times the
    sum, which is that of u - z), and the roundings of chains of at most some 400: 40 * 20 U; what is left is rounded.
    `once`: whether h may be rounded once (by default what the shape's form does)."""
    h = STEP if (tiled(*shape) if once is None else once) else TWICE
    return h + 3 * 40 * 20 * U + STEP * STEP


def moe_error(first, left, want):
    """From a call's result, what a second call leaves with the first's negative as its residual, and the 64-bit result."""
    return rms(left.double() - (want - first.double())) / rms(want)


def linear_limit(exact, K, x, size, slope, plain, want):
    """Root mean square of act(sum + bias) + residual's error, the result's own rounding taken off: the sums' roundings
    (and, with weights rounded to bf16, STEP of each product) through the activation's slope, and what is left."""
    sums = U * (K / 32 + 160) ** 0.5 * (x.double().pow(2) @ size.double().pow(2).T).mean().sqrt().item()
    return slope * (sums + (0.0 if exact else STEP * plain)) + 12 * U * rms(want) + STEP * STEP * rms(want) + 1e-7


def bf16(x):
    return x.float().to(torch.bfloat16).double()
