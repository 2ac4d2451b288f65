"""Plain 64-bit forms of the many-tensor AdamW operators, with the bounds
their 32-bit evaluation keeps, for the tests. Nothing here is taken from the
library.

Bounds. U = 2^-24 is half a step of binary32 relative to the value. Each
operation of the kernel's sequence adds U times its own result, a scalar
rounded to binary32 adds U times the term it multiplies, and an error of an
input goes through the derivative; products of two such errors (2^-48) are
covered by the factor SAFE."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
SAFE = 1.01
PIECE, BLOCK = 2048, 32


def scalars(lr, betas, eps, t):
    b1, b2 = betas
    return dict(lr=lr, b1=b1, b2=b2, eps=eps, bc1=1.0 - b1 ** t, bc2=1.0 - b2 ** t)


def mean_gradient(reps, sumsq=None, max_norm=None):
    """(g, error bound) of the mean over reps (float64 arrays), clipped."""
    n = len(reps)
    total, mass, err = np.zeros_like(reps[0]), np.zeros_like(reps[0]), np.zeros_like(reps[0])
    for q, r in enumerate(reps):
        total = total + r
        mass = mass + np.abs(r)
        if q:
            err = err + U * mass              # each partial sum is at most the mass so far
    g, err = total / n, err / n + U * np.abs(total / n) * (n > 1)
    if sumsq is not None:
        c = max_norm / (np.sqrt(sumsq) + 1e-6)
        if c < 1.0:
            g, err = g * c, err * c + 2 * U * np.abs(g * c)
    return g, err


def _update(p, u, du, lr, factor, decay):
    """p * (1 - lr*factor*decay) - u. keep: lr_k has two roundings, its
    product with the decay (itself rounded) two more, the difference one."""
    ld = lr * factor * decay
    keep = 1.0 - ld
    new = p * keep - u
    dp = np.abs(p) * (U * (4 * abs(ld) + abs(keep)) + U * abs(keep)) + du + U * np.abs(new)
    return new, SAFE * dp


def moments(g, dg, m, v, sc):
    """Fresh m and v with bounds. m*b1: b1 and the product; (1-b1)*g in the
    fma: 1-b1; the fma's own rounding."""
    b1, b2 = sc["b1"], sc["b2"]
    c1, c2 = 1.0 - b1, 1.0 - b2
    mn = b1 * m + c1 * g
    dm = c1 * dg + U * (2 * b1 * np.abs(m) + c1 * np.abs(g) + np.abs(mn))
    vn = b2 * v + c2 * g * g
    dv = 2 * c2 * np.abs(g) * dg + U * (2 * b2 * v + 2 * c2 * g * g + vn)
    return mn, SAFE * dm, vn, SAFE * dv


def _ratio(a, b):
    return np.divide(a, b, out=np.zeros_like(a), where=b > 0)


def step32(p, m, v, g, dg, sc, factor, decay):
    """(p, m, v) and their bounds. The step u has m/bc1 (bc1, quotient), the
    product with lr_k (two roundings of lr_k, product), v/bc2 (bc2,
    quotient; half through the root), root, eps, sum, quotient: 10 U."""
    mn, dm, vn, dv = moments(g, dg, m, v, sc)
    den = np.sqrt(vn / sc["bc2"]) + sc["eps"]
    lr = sc["lr"] * factor
    u = _ratio(lr * mn / sc["bc1"], den)
    du = _ratio(abs(lr) * dm / sc["bc1"], den) + np.abs(u) * (0.5 * _ratio(dv, vn) + 10 * U)
    pn, dp = _update(p, u, SAFE * du, sc["lr"], factor, decay)
    return (pn, mn, vn), (dp, dm, dv)


def step8(p, m, r, g, dg, sc, factor, decay):
    """(p, m, r) before coding, and their bounds. r*r rounds once. The root is
    a Newton step from the hardware's: at most one ulp, 2 U, off. The step
    (lr_k/bc1) * (m / (r/sqrt(bc2) + eps)): lr_k (2), bc1, its reciprocal from
    the hardware (one ulp, 2) and their product; r's root (2), 1/sqrt(bc2) as
    bc2 through the root (1/2) and the hardware's reciprocal root (one ulp,
    2), its product with r and the sum in one fma, the hardware's reciprocal
    of it (2), the product: 14.5 U. The last product is inside the fma that
    _update counts."""
    mn, dm, vn, dv = moments(g, dg, m, r * r, sc)
    dv = dv + U * sc["b2"] * r * r
    rn = np.sqrt(vn)
    dr = SAFE * (0.5 * rn * _ratio(dv, vn) + 2 * U * rn)
    den = rn / np.sqrt(sc["bc2"]) + sc["eps"]
    lr = sc["lr"] * factor
    u = _ratio(lr * mn / sc["bc1"], den)
    du = _ratio(abs(lr) * dm / sc["bc1"], den) + np.abs(u) * (0.5 * _ratio(dv, vn) + 14.5 * U)
    pn, dp = _update(p, u, SAFE * du, sc["lr"], factor, decay)
    return (pn, mn, rn), (dp, dm, dr)


# ------------------------------------------------------------------ 8 bits

def noise(seed, t, count, start=0):
    """(of m, of r): 16 bits per element [start, start + count) of the state."""
    def mix(x):
        x = (x * np.uint64(0x9E3B5A35)) & np.uint64(0xFFFFFFFF)
        x = x ^ (x >> np.uint64(15))
        x = (x * np.uint64(0x5D2C9E1B)) & np.uint64(0xFFFFFFFF)
        return x ^ (x >> np.uint64(16))

    key = mix(mix(np.uint64(seed)) ^ np.uint64(t & 0xFFFFFFFF))
    i = np.arange(start, start + count, dtype=np.uint64)
    q = i >> np.uint64(2)
    x = mix(((q & np.uint64(0xFFFFFFFF)) + (q >> np.uint64(32)) * np.uint64(0x7F4A7C15) + key)
            & np.uint64(0xFFFFFFFF))
    by = np.array([1, 0xB5297A4D, 0x68E31DA5, 0x1B56C4E9], np.uint64)[(i & np.uint64(3)).astype(int)]
    w = (x * by) & np.uint64(0xFFFFFFFF)
    return (w >> np.uint64(16)).astype(np.float64), (w & np.uint64(0xFFFF)).astype(np.float64)


def scale_exponent(top):
    """e of the scale 2^e: the least that keeps `top` within 448 * 2^e, and
    at least -126."""
    half, octave = np.frexp(top)                 # half in [1/2, 1)
    e = octave - 9 + (half > 0.875)
    return np.where(top > 0, np.maximum(e, -126), -126)


def code_value(x, noise16, e, root):
    """What x is stored as, on the scale 2^e."""
    half, octave = np.frexp(np.abs(x))
    y = np.ldexp(np.floor(half * 16.0 + noise16 / 65536.0), octave - 4)
    y = np.ldexp(y, -e)
    y = np.where(y < 2.0 ** -6, np.round(y * 512.0) / 512.0, y)
    if root:
        y = np.where(x > 0, np.maximum(y, 2.0 ** -9), y)
    return np.copysign(np.ldexp(y, e), x)


def check_codes(got, e, x, dx, noise16, root, what):
    """got (values) and e (scale exponents per block) against x known to dx:
    the code is monotone in x, so it lies between those of x - dx and x + dx."""
    got, x, dx, noise16 = (a.reshape(-1, BLOCK) for a in (got, x, dx, noise16))
    top = np.abs(x)
    lo = scale_exponent(np.max(np.maximum(top - dx, 0), axis=1))
    hi = scale_exponent(np.max(top + dx, axis=1))
    assert np.all((e >= lo) & (e <= hi)), f"{what}: scale"
    e = e[:, None]
    a = code_value(np.maximum(x - dx, 0) if root else x - dx, noise16, e, root)
    b = code_value(x + dx, noise16, e, root)
    bad = ~((got >= a) & (got <= b))
    assert not bad.any(), (f"{what}: {int(bad.sum())} codes off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} not in [{a[bad][0]}, {b[bad][0]}] of {x[bad][0]}")
