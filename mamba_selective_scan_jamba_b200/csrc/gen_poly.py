"""Derives the polynomial constants of the scan kernel's FMA-pipe functions and of the
normal distribution's tail, and writes csrc/poly_consts.cuh.

* exp2(f) on f in [-1/2, 1/2]: degree-6 minimax polynomial in the relative
  error (Remez exchange algorithm).  Used with the exact base-2 range
  reduction x = j + f, j = round(x), 2^x = 2^j * p(f).
* log1p(w) on w in [0, 1]: w * P(w), P of degree 8, minimax in the relative
  error of log1p.

* 1/x: Newton-Raphson r <- r (2 - x r) from the bit-pattern initial guess
  r0 = as_float(K - bits(x)); K is chosen here to minimise the largest
  relative error of r0 over one binade (the error pattern repeats per binade).

* Phi(-a) exp(a^2 / 2) for a in [0, 14], the normal tail without its exponential:
  t * P(t), t = 1 / (1 + NC a), P of degree 7, minimax in the relative error (1.7e-7).
  The function is the integral of exp(-a s - s^2 / 2) over s >= 0, divided by
  sqrt(2 pi).

The polynomials are fitted in float64 and stored as float32; the float32
evaluation error bounds are checked by tests/test_poly_consts.py.
"""
import os

import numpy as np


def remez(f, deg, a, b, iters=40, grid=400001):
    """Minimax polynomial (coefficients low -> high) of f on [a, b] in relative error."""
    n = deg + 2
    x = (a + b) / 2 + (b - a) / 2 * np.cos(np.pi * np.arange(n)[::-1] / (n - 1))
    t = np.linspace(a, b, grid)
    c = None
    for _ in range(iters):
        A = np.zeros((n, n))
        for i in range(n):
            A[i, :deg + 1] = x[i] ** np.arange(deg + 1)
            A[i, deg + 1] = -((-1) ** i) * f(x[i])
        c = np.linalg.solve(A, f(x))[:deg + 1]
        err = (np.polyval(c[::-1], t) - f(t)) / f(t)
        zc = np.where(np.diff(np.sign(err)) != 0)[0]
        bounds = np.concatenate([[0], zc + 1, [len(t)]])
        ext = [t[np.argmax(np.abs(err[bounds[i]:bounds[i + 1]])) + bounds[i]]
               for i in range(len(bounds) - 1)]
        if len(ext) == n:
            x = np.array(ext)
    return c


def exp2_coeffs():
    return remez(np.exp2, 6, -0.5, 0.5).astype(np.float32)


def log1p_over_w(w):
    w = np.asarray(w, dtype=np.float64)
    safe = np.where(w == 0, 1.0, w)
    return np.where(w == 0, 1.0, np.log1p(safe) / safe)


def log1p_coeffs():
    return remez(log1p_over_w, 8, 0.0, 1.0).astype(np.float32)


def rcp_magic() -> int:
    x = np.linspace(1.0, 2.0, 100001, dtype=np.float32)[:-1]
    bx = x.view(np.int32).astype(np.int64)
    xd = x.astype(np.float64)

    def err(k):
        r0 = (k - bx).astype(np.int32).view(np.float32).astype(np.float64)
        return np.abs(r0 * xd - 1).max()

    best = min(range(0x7EF00000, 0x7F000001, 0x100), key=err)
    return min(range(best - 0x100, best + 0x101), key=err)


TAIL_C = 0.3


def tail_over_t(t):
    t = np.asarray(t, dtype=np.float64)
    a = ((1.0 / t - 1.0) / TAIL_C).reshape(-1, 1)
    x, w = np.polynomial.legendre.leggauss(96)
    s, w = 4.5 * (x + 1.0), 4.5 * w          # (behind 9 the integrand is below 1e-17)
    r = np.exp(-a * s - 0.5 * s * s) @ w / np.sqrt(2.0 * np.pi)
    return r.reshape(t.shape) / t


def tail_coeffs():
    return remez(tail_over_t, 7, 1.0 / (1.0 + 14.0 * TAIL_C), 1.0, grid=4001).astype(np.float32)


def render() -> str:
    e, l, n = exp2_coeffs(), log1p_coeffs(), tail_coeffs()
    fmt = lambda v: "%.9ef" % float(v)
    out = ["// Generated by gen_poly.py: minimax polynomials (Remez exchange) in float32.",
           "#pragma once", "", "namespace jmix {", "namespace poly {", "",
           "// 2^f ~ E0 + f*(E1 + f*(E2 + ...)) for f in [-1/2, 1/2]"]
    out += ["constexpr float E%d = %s;" % (i, fmt(v)) for i, v in enumerate(e)]
    out += ["", "// log1p(w) ~ w*(L0 + w*(L1 + ...)) for w in [0, 1]"]
    out += ["constexpr float L%d = %s;" % (i, fmt(v)) for i, v in enumerate(l)]
    out += ["", "// Phi(-a) exp(a^2 / 2) ~ t*(N0 + t*(N1 + ...)), t = 1 / (1 + NC a), for a in [0, 14]",
            "constexpr float NC = %s;" % fmt(TAIL_C)]
    out += ["constexpr float N%d = %s;" % (i, fmt(v)) for i, v in enumerate(n)]
    out += ["", "// 1/x initial guess: as_float(RCP_MAGIC - bits(x)), then Newton-Raphson",
            "constexpr int RCP_MAGIC = 0x%x;" % rcp_magic()]
    out += ["", "}  // namespace poly", "}  // namespace jmix", ""]
    return "\n".join(out)


if __name__ == "__main__":
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "poly_consts.cuh")
    with open(path, "w") as f:
        f.write(render())
    print(path)
