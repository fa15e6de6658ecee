"""Rotary positions in 64 bits, from the definition, for the tests: pairs turned by exact angles."""
import functools
from decimal import Decimal, getcontext

import torch

getcontext().prec = 90
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
ONE = 1 << 128  # a turn


@functools.lru_cache(maxsize=None)
def _turn(f: float) -> int:
    return int((Decimal(f) / TWO_PI * ONE).to_integral_value())


def angles(rope, positions) -> torch.Tensor:
    """Radians in [0, 2 pi) of every (position, pair): whole turns are dropped in integers, so that
    far positions lose nothing."""
    rows = [[float(Decimal(p * _turn(f) % ONE) / ONE * TWO_PI) for f in rope.inv_freq]
            for p in positions.flatten().tolist()]
    return torch.tensor(rows, dtype=torch.float64).view(*positions.shape, -1)


def pairs(rope):
    rd = rope.rotary_dim
    return ((slice(0, rd, 2), slice(1, rd, 2)) if rope.interleaved
            else (slice(0, rd // 2), slice(rd // 2, rd)))


def turned(rope, x, positions, transposed=False):
    """(y, bound): x [..., heads, 128] turned, in 64 bits on the CPU, and how far fp32 arithmetic may
    be off before the last rounding.

    The bound, relative to m (|x_a| + |x_b|): the angle is cut at 2^-32 of a turn (1.5e-9) and its
    rest within an eighth of a turn rounded to 24 bits (2^-25 * pi / 2 = 4.7e-8, as the cosine's and
    sine's derivatives are at most 1); a cosine or sine within 1e-7, its product with m, m's own
    rounding, the product with x and the sum: four roundings of 2^-24, 2.4e-7.  Together below 2^-20
    (9.5e-7)."""
    x = x.double().cpu()
    t = angles(rope, positions.cpu())[..., None, :]
    cos, sin = torch.cos(t) * rope.magnitude, torch.sin(t) * rope.magnitude
    if transposed:
        sin = -sin
    a, b = pairs(rope)
    y, bound = x.clone(), torch.zeros_like(x)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    near = (x[..., a].abs() + x[..., b].abs()) * (abs(rope.magnitude) * 2.0 ** -20)
    bound[..., a] = near
    bound[..., b] = near
    return y, bound


TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def check(got, y, bound):
    """|got - y| within the arithmetic's bound and half a step of got's type (half the smallest
    subnormal near zero)."""
    far = (got.double().cpu() - y).abs()
    eps = torch.finfo(got.dtype).eps
    room = bound + (y.abs() + bound) * (eps / 2) + TINY[got.dtype]
    assert bool((far <= room).all()), float((far / room).max())
