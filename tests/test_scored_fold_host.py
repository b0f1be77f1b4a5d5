"""Capped scores by their polynomials, step by step in fp32 as the kernels take
them, over every raw score and cap that the calls allow (no GPU)."""
import os
import re

import numpy as np
import pytest

from quantized_kv_cache_quantize_gb300.csrc import tanh_fit

SOURCE = open(os.path.join(os.path.dirname(tanh_fit.__file__), "kvq_scores.cuh")).read()
LOG2E = np.float32(1.4426950408889634)


def constants(function: str) -> list[np.float32]:
    """The decimal constants of a function of the source, in order."""
    body = SOURCE[SOURCE.index(function):]
    return [np.float32(v) for v in re.findall(r"-?\d\.\d+e[-+]\d+(?=f)", body[:body.index("\n}")])]


def test_the_constants_stand_in_their_places():
    small = tanh_fit.fit_coefficients().astype(np.float32)
    low = tanh_fit.fit_coefficients(tanh_fit.LOW_TERMS, tanh_fit.LOW_X).astype(np.float32)
    assert constants("uint64_t tanh_small(") == list(small[::-1])
    assert constants("LowCap low_cap(") == list(low)


def fma(a, b, c):
    """Rounded once: fp32 products are exact in 64 bits, their sums nearly."""
    return (a.astype(np.float64) * b + c).astype(np.float32)


@pytest.mark.parametrize("raw", [1.0, 300.0, 7e4, 6e5, 2e6, 1.47e7])
@pytest.mark.parametrize("cap", [2.0 ** -20, 2.0 ** -9, 1.0, 5.0, 50.0, 256.0, 3e4, 2.0 ** 20])
def test_low_scores(raw, cap):
    """Off by 2^-21 of the score, what the calls promise.  The fit with fp32
    coefficients is off by 2^-23.0; the cap's place in the leading coefficient, x, the
    last sum of the polynomial and the result are rounded by 2^-24 each at most, all
    other steps stand beside terms a tenth of the leading one or less: 2^-24 together."""
    c = [np.float32(k) for k in tanh_fit.fit_coefficients(tanh_fit.LOW_TERMS, tanh_fit.LOW_X).astype(np.float32)]
    cap2 = np.float32(np.float32(cap) * LOG2E)
    c = [np.float32(k * cap2) for k in c]
    x_max = np.linspace(1e-3, 0.4, 400)
    ck = (x_max / raw).astype(np.float32)
    for s in (np.float32(raw), np.float32(-raw / 3), np.float32(raw / 1000)):
        x = (s * ck).astype(np.float32)
        z = (x * x).astype(np.float32)
        p = fma(c[3], z, np.full_like(z, c[2]))
        p = fma(p, z, c[1])
        p = fma(p, z, c[0])
        got = fma(p, x, np.float32(0.0)).astype(np.float64)
        want = float(cap2) * np.tanh(ck.astype(np.float64) * float(s))
        assert np.abs(got / want - 1).max() <= 2.0 ** -21
