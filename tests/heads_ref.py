"""The head operators (rotary positions, the head norm, its backward) in 64
bits from their formulas, on the host, and how far the kernels may be off.

Bounds.  A stored value is rounded once: half a step, 2^-8 of the value for
bf16 and 2^-24 for fp32.  Before that:
  - cos and sin: the angle is off by at most half an ulp of half a turn
    (2 pi 2^-26) plus the rounding of its product with 2 pi; the
    special-function unit (bf16) by 2^-20.9, the accurate functions (fp32) by
    two ulp.  Together at most 2^-20, which multiplies |a| + |b| of the pair.
  - r: a sum of at most 512 squares, 16 values in a lane and 5 shuffles, 21
    additions deep: below 2^-19 of r, and the same for mean(g w x r) of the
    sum of its magnitudes; the products around them add a few 2^-24.
So a rotated pair is within 2^-18 (|a| + |b|) of the exact one, the norm
included, and dx within 2^-17 r (|g| w + |x r| mean(|g w x r|)), |g| <= A
(|dy_a| + |dy_b|).  dw adds n terms, at worst one after the other: n 2^-24
plus the terms' own 2^-18, of the sum of their magnitudes.
"""
import math

import torch


def frequencies(rot, base=10000.0, scaling=None, freqs=None):
    s = scaling or {}
    kind = s.get("kind")
    if kind == "ntk":
        base = base * s["factor"] ** (rot / (rot - 2.0))
    out = []
    for i in range(rot // 2):
        f = float(freqs[i]) if freqs is not None else math.pow(base, -2.0 * i / rot)
        if kind == "linear":
            f = f / s["factor"]
        if kind == "by_parts":
            low, high = s.get("low", 1.0), s.get("high", 32.0)
            turns = s["original_length"] * f / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = f * keep + f / s["factor"] * (1.0 - keep)
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def turns_mod_1(positions, freq):
    """Fraction of a turn of each (position, pair): the integer and fractional
    parts of the step are reduced apart, in Python integers, so that far
    positions lose nothing."""
    steps = [int(round((f / (2.0 * math.pi)) % 1.0 * 2.0 ** 64)) for f in freq.tolist()]
    flat = [[((p * s) % 2 ** 64) / 2.0 ** 64 for s in steps] for p in positions.reshape(-1).tolist()]
    return torch.tensor(flat, dtype=torch.float64).reshape(tuple(positions.shape) + (len(steps),))


class Angles:
    """cos and sin (batch, tokens, 1, rot / 2) of positions (batch, tokens)."""

    def __init__(self, positions, rot, layout, amplitude=1.0, **freq):
        t = turns_mod_1(positions, frequencies(rot, **freq)) * (2.0 * math.pi)
        self.c, self.s = torch.cos(t).unsqueeze(-2), torch.sin(t).unsqueeze(-2)
        self.rot, self.layout, self.amplitude = rot, layout, amplitude

    def pairs(self, x):
        r = self.rot
        return (x[..., :r // 2], x[..., r // 2:r]) if self.layout == "half" else (x[..., 0:r:2], x[..., 1:r:2])

    def put(self, a, b, rest):
        first = torch.cat([a, b], -1) if self.layout == "half" else torch.stack([a, b], -1).flatten(-2)
        return torch.cat([first, rest], -1)

    def rotate(self, x, inverse=False):
        a, b = self.pairs(x)
        s = -self.s if inverse else self.s
        A = self.amplitude
        return self.put(A * (a * self.c - b * s), A * (b * self.c + a * s), x[..., self.rot:])

    def spread(self, x):
        """A (|a| + |b|) at both places of each pair, |x| elsewhere: what a
        rotated pair's error is measured against."""
        a, b = self.pairs(x.abs())
        m = abs(self.amplitude) * (a + b)
        return self.put(m, m, x[..., self.rot:].abs())


def norm(x, w, eps):
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r if w is None else x * r * w


def backward(dy, x, w, eps, ang):
    """(dx, dw, magnitude dx is measured against, sum of dw's magnitudes)."""
    g, gm = ang.rotate(dy, inverse=True), ang.spread(dy)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    mag = r * (gm * w.abs() + n.abs() * (gm * w.abs() * n.abs()).mean(-1, keepdim=True))
    flat = lambda t: t.reshape(-1, x.shape[-1]).sum(0)  # noqa: E731
    return dx, flat(g * n), mag, flat(gm * n.abs())


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, want, mag, dtype, rel):
    """|got - want| <= half a step of the value + rel * magnitude (values below
    the type's normal range round by its smallest step)."""
    err = (got.double().cpu() - want).abs()
    bound = want.abs() * half_step(dtype) * (1 + 2.0 ** -7) + rel * mag + torch.finfo(dtype).tiny
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, "worst error is %.3f of its bound" % worst
    return worst
