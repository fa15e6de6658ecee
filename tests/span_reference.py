"""Plain 64-bit forms of windowed attention and of the narrow (8-bit) cache, and the
tolerances of the kernels against them.

Tolerances.  With w_t the softmax weights, A = sum_t w_t |v_t| and U = sum_i |q_i k_i| / sqrt(128)
(largest over the visible tokens):
* a score is an fp32 sum of 128 exact products, scaled twice: off by at most
  e = 132 * 2^-24 * U; a weight is then off by 2 e + 2^-20 relative (its own score, the sum
  of all, exp2 and the sums over tokens);
* the decode kernel's weights enter the second product with 22 bits (inside the 2^-20), the
  prompt kernel's as one fp16 number: half a step, 2^-11, more;
* the result is rounded to fp16 once: 2^-11 |out|, or 2^-25 below fp16's normal range, and
  from 65520 on (half a step past 65504, the largest fp16 number) to an infinity.
The log-sum-exp is off by e + 2^-20 + 2^-22 |lse|.
"""
from __future__ import annotations

import math

import torch

D = 128


def attend(q, k, v, allowed):
    """q [R, 128], k / v [T, 128], allowed [R, T] -> out, lse, and per row A [R, 128] and the
    largest U among the visible tokens; hidden tokens' values are not looked at."""
    q, k, v = q.double(), k.double(), v.double()
    s = q @ torch.where(torch.isfinite(k), k, torch.zeros_like(k)).T / math.sqrt(D)
    s = s.masked_fill(~allowed, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    w = torch.where(allowed, w, torch.zeros_like(w))
    v0 = torch.where(allowed.any(0)[:, None], v, torch.zeros_like(v))
    u = (q.abs() @ torch.where(torch.isfinite(k), k, torch.zeros_like(k)).abs().T) / math.sqrt(D)
    u = torch.where(allowed, u, torch.zeros_like(u)).amax(-1) if k.shape[0] else q.new_zeros(len(q))
    return w @ v0, lse, w @ v0.abs(), u


def assert_close(out, lse, ref, prompt=False, what=""):
    r_out, r_lse, A, U = ref
    e = (132 * 2.0 ** -24 * U)[:, None]
    rel = 2 * e + 2.0 ** -20 + (2.0 ** -11 if prompt else 0.0)
    tol = rel * A + 2.0 ** -11 * (r_out.abs() + rel * A) + 2.0 ** -25
    err = (out.double() - r_out).abs()
    past = (r_out.abs() + tol >= 65520) & (out.double() == torch.copysign(torch.full_like(r_out, math.inf), r_out))
    bad = ~((err <= tol) | past)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values beyond tolerance, worst "
                           f"{float((err / tol).max()):.3g} of it")
    none = torch.isinf(r_lse)
    assert torch.equal(torch.isneginf(lse.double()), none), f"{what}: rows without a token"
    assert not out[none].any(), f"{what}: rows without a token are 0"
    z = (lse.double() - r_lse).abs()[~none]
    lim = (e[:, 0] + 2.0 ** -20 + 2.0 ** -22 * r_lse.abs())[~none]
    assert bool((z <= lim).all()), f"{what}: lse off by {float((z / lim).max()):.3g} of its tolerance"


def window_mask(L, n, sink, window, device):
    """[n, L]: which tokens the last n query positions see."""
    at = torch.arange(L - n, L, device=device)[:, None]
    j = torch.arange(L, device=device)[None]
    return (j <= at) & ((j < sink) | (at - j < window))


def pow2_scale(top):
    """The smallest power of two s with top <= 448 s; 1 for 0 (top: fp64 tensor)."""
    s = torch.exp2(torch.ceil(torch.log2(top / 448)))
    return torch.where(top > 0, s, torch.ones_like(s))


def e4m3_grid():
    return torch.tensor([(m / 8) * 2.0 ** -6 for m in range(8)] +
                        [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64)


def e4m3(y):
    """The nearest e4m3 number of every value (fp64), ties to even, saturating."""
    grid = e4m3_grid().to(y.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = y.abs().contiguous()
    lo = torch.searchsorted(mid, a)
    tie = (lo < mid.numel()) & (mid[lo.clamp(max=mid.numel() - 1)] == a)
    return torch.copysign(grid[torch.where(tie & (lo % 2 == 1), lo + 1, lo)], y)


class NarrowReference:
    """A narrow cache kept as lists of fp16 tokens per sequence: what every page must hold."""

    def __init__(self, batch, hkv, page):
        self.P, self.hkv = page, hkv
        self.k = [torch.zeros((hkv, 0, D), dtype=torch.float16) for _ in range(batch)]
        self.v = [x.clone() for x in self.k]

    def write(self, k, v):
        """k, v [B, n, hkv, 128] fp16 (CPU)."""
        for b in range(len(self.k)):
            self.k[b] = torch.cat([self.k[b], k[b].transpose(0, 1)], 1)
            self.v[b] = torch.cat([self.v[b], v[b].transpose(0, 1)], 1)

    def length(self, b):
        return self.k[b].shape[1]

    def pages(self, b, name):
        """(codes' values [N, hkv, P, 128] fp64, scales [N, hkv]) of the complete pages, and
        the rows of the open one."""
        x = getattr(self, name)[b].double()
        full = x.shape[1] // self.P
        pages = x[:, :full * self.P].reshape(self.hkv, full, self.P, D).transpose(0, 1)
        fin = torch.where(torch.isfinite(pages), pages, torch.zeros_like(pages))
        s = pow2_scale(fin.abs().amax((-1, -2))) if full else x.new_zeros((0, self.hkv))
        y = (pages / s[:, :, None, None]).clamp(-448, 448)
        return e4m3(y), s, getattr(self, name)[b][:, full * self.P:]

    def values(self, b, name):
        """[hkv, L, 128] fp64: what attention reads."""
        code, s, rest = self.pages(b, name)
        return torch.cat([(code * s[:, :, None, None]).transpose(0, 1).reshape(self.hkv, -1, D),
                          rest.double()], 1)
