"""Dropout, layer norm and its backward in 64 bits from their formulas, on the
host, and how far the kernels may be off.

Bounds.  u = 2^-24 is half a step of fp32; a stored value is rounded once more,
half a step of its type (2^-8 of it for bf16, 2^-24 for fp32).  Before that:
  - a kept element: the scale's rounding and the product's, 2u of it, and the
    residual's addition, u of the sum (a fused multiply-add: less).
  - a sum over a row: a thread's values one after the other, 5 shuffles, up to 16
    warps: an addition chain of `depth` values errs by depth u of the sum of
    magnitudes.  depth = 8 ceil(N / 4096) + 96 holds for every kernel: 32 values
    to a thread below 16384 columns, N / 512 above.
  - mean: that, over N, and the errors of h;  variance: differences from a mean
    that is off by dm add dm^2, those of h 2 |h - mean| dh, the sum depth + 4 u.
    Warps take theirs from their own means, each off by dm at most; of the
    differences of these from the row's mean, 2 dm |m_w - mean| stays, at most
    2 dm times the row's standard deviation.
  - backward: n = (x - mean) rstd 2u; the means of a and a n as sums, with 4 u for
    the products in them; their combination 4 u of each term.
  - dw and db: at worst one row after the other, (M + 64) u of the magnitudes, and
    4u of each term.
"""
import numpy as np
import torch

U = 2.0 ** -24
LOW = 0xFFFFFFFF


def philox(counter, key):
    """Philox 4x32-10: four arrays of counter words (or numbers) and a key of two."""
    c = [np.asarray(w, dtype=np.uint64) for w in counter]
    k = [np.uint64(w) for w in key]
    for _ in range(10):
        x, y = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(y >> np.uint64(32)) ^ c[1] ^ k[0], y & np.uint64(LOW), (x >> np.uint64(32)) ^ c[3] ^ k[1], x & np.uint64(LOW)]
        k = [(k[0] + np.uint64(0x9E3779B9)) & np.uint64(LOW), (k[1] + np.uint64(0xBB67AE85)) & np.uint64(LOW)]
    return c


def kept(rows, cols, threshold, seed, step, site, row0=0):
    """True (rows, cols) where an element stays."""
    g, r = np.meshgrid(np.arange((cols + 7) // 8, dtype=np.uint64), np.arange(row0, row0 + rows, dtype=np.uint64))
    words = philox((g, r, np.uint64(site), np.uint64(step & LOW)), (seed & LOW, seed >> 32))
    halves = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], -1)
    return torch.from_numpy(halves.reshape(rows, -1)[:, :cols] >= threshold)


class Mask:
    """A call's mask; None as rng: everything stays."""

    def __init__(self, rng, rows, cols, site=0, row0=0):
        if rng is None or rng.threshold == 0:
            self.keep, self.scale = torch.ones(rows, cols, dtype=torch.bool), 1.0
            return
        self.keep = kept(rows, cols, rng.threshold, rng.seed, int(rng.step), site, row0)
        self.scale = 65536.0 / (65536 - rng.threshold) if rng.threshold < 65536 else 0.0

    def __call__(self, x):
        return torch.where(self.keep, x * self.scale, torch.zeros_like(x))


def wide(t):
    return None if t is None else t.detach().cpu().double().reshape(-1, t.shape[-1])


def rounding(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, bound, dtype, what):
    """got within bound + half a step of its type of want; where want is not finite, got is the same."""
    got = got.detach().cpu().double().reshape(want.shape)
    fine = torch.isfinite(want)
    assert bool(((got == want) | (torch.isnan(got) & torch.isnan(want)) | fine).all()), what + ": not the same infinities"
    smallest = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149  # a subnormal's step
    off = (got - want).abs() - (bound + rounding(dtype) * (want.abs() + bound) + smallest)
    off = torch.where(fine, off, torch.zeros_like(off))
    assert bool((off <= 0).all()), "%s: %d of %d off, worst by %g at %s" % (
        what, int((off > 0).sum()), off.numel(), float(off.max()), np.unravel_index(int(off.argmax()), off.shape))


def depth(n):
    return 8 * ((n + 4095) // 4096) + 96


def summed(x, residual, mask):
    """h and what it may be off by before it is stored."""
    d = mask(wide(x))
    if residual is None:
        return d, (2 * U * d.abs() if mask.scale != 1.0 else torch.zeros_like(d))
    h = d + wide(residual)
    return h, 2 * U * d.abs() + U * h.abs()


def norm(h, dh, w, b, eps):
    """{name: (value, bound)} of y, mean and rstd."""
    n = h.shape[1]
    k = depth(n)
    mean = h.mean(1, keepdim=True)
    d_mean = k * U * h.abs().mean(1, keepdim=True) + dh.mean(1, keepdim=True)
    c = h - mean
    var = (c * c).mean(1, keepdim=True)
    d_c = dh + d_mean + U * c.abs()
    d_var = (k + 4) * U * var + 2 * (c.abs() * (dh + U * c.abs())).mean(1, keepdim=True) \
        + d_mean ** 2 + (d_c ** 2).mean(1, keepdim=True) + 2 * torch.sqrt(var) * d_mean
    r = 1.0 / torch.sqrt(var + eps)
    d_r = r * (0.5 * d_var * r * r * 1.1 + 4 * U)
    w = torch.ones(n, dtype=torch.float64) if w is None else w.cpu().double()
    b = torch.zeros(n, dtype=torch.float64) if b is None else b.cpu().double()
    z = c * r * w
    d_y = (d_c * r + c.abs() * d_r) * w.abs() * 1.01 + 4 * U * z.abs() + U * (z + b).abs()
    return {"y": (z + b, d_y), "mean": (mean[:, 0], d_mean[:, 0]), "rstd": (r[:, 0], d_r[:, 0])}


def norm_backward(dy, x, mean, rstd, w, add, mask):
    """{name: (value, bound)} of d_residual (g), dx, dw and db."""
    dy, x = wide(dy), wide(x)
    rows, cols = x.shape
    k = depth(cols)
    mean, rstd = mean.cpu().double().reshape(-1, 1), rstd.cpu().double().reshape(-1, 1)
    w = torch.ones(cols, dtype=torch.float64) if w is None else w.cpu().double()
    n = (x - mean) * rstd
    a = dy * w
    m1, m2 = a.mean(1, keepdim=True), (a * n).mean(1, keepdim=True)
    d1, d2 = (k + 2) * U * a.abs().mean(1, keepdim=True), (k + 6) * U * (a * n).abs().mean(1, keepdim=True)
    g = rstd * (a - m1 - n * m2)
    d_g = rstd * (d1 + n.abs() * d2 + 4 * U * (a.abs() + m1.abs() + (n * m2).abs()))
    if add is not None:
        g = g + wide(add)
        d_g = d_g + U * g.abs()
    dx = mask(g)
    out = {"d_residual": (g, d_g), "dx": (dx, mask(d_g) + 2 * U * dx.abs())}
    for name, term in (("dw", dy * n), ("db", dy)):
        out[name] = (term.sum(0), (rows + 68) * U * term.abs().sum(0))
    return out
