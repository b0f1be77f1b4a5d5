"""Coefficients of the polynomials that capped scores use for tanh, on |x| <= 1
and, with fewer terms, on |x| <= 0.4.

tanh(x) / x is a function of z = x^2, analytic but for poles, the nearest at
z = -pi^2 / 4.  It is interpolated at the N Chebyshev nodes of [0, X^2] (a standard
Chebyshev interpolation; with p = pi^2 / 4 / X^2 the error falls by (sqrt(1 + p) +
sqrt(p))^2 per coefficient, a factor of 11.8 for X = 1) and rewritten in powers
of z.

Run: python quantized_kv_cache_quantize_gb300/csrc/tanh_fit.py  (prints the
constants of kvq_scores.cuh's tanh_small, the highest power first there, and low_cap).
"""
from __future__ import annotations

import numpy as np

N_TERMS, LOW_TERMS, LOW_X = 7, 4, 0.4


def tanh_over_x(z: np.ndarray) -> np.ndarray:
    """tanh(sqrt z) / sqrt z, with its series near 0."""
    z = np.asarray(z, dtype=np.float64)
    x = np.sqrt(np.maximum(z, 1e-4))
    return np.where(z < 1e-4, 1.0 - z / 3.0 + 2.0 * z * z / 15.0, np.tanh(x) / x)


def fit_coefficients(n: int = N_TERMS, x_max: float = 1.0) -> np.ndarray:
    """c_0 .. c_(n-1) (float64) of tanh(x) ~ x sum c_k x^(2k) on |x| <= x_max."""
    from numpy.polynomial import chebyshev as C
    from numpy.polynomial import polynomial as P
    k = np.arange(n)
    t = np.cos(np.pi * (k + 0.5) / n)
    in_t = C.cheb2poly(C.chebfit(t, tanh_over_x((t + 1.0) * x_max ** 2 / 2.0), n - 1))
    in_z = np.zeros(1)
    for i, ci in enumerate(in_t):                  # t = 2 z - 1
        in_z = P.polyadd(in_z, ci * P.polypow([-1.0, 2.0 / x_max ** 2], i))
    return np.asarray(in_z[:n], dtype=np.float64)


if __name__ == "__main__":
    for fit in (fit_coefficients(), fit_coefficients(LOW_TERMS, LOW_X)):
        print(", ".join(f"{float(np.float32(c)):.9e}f" for c in fit))
