"""The scan's log(1 + u) polynomial, from the coefficients in its source."""
import os
import re

import numpy as np

import gated_delta_rule_158_b200 as kda

SRC = os.path.join(os.path.dirname(kda.__file__), "csrc", "kda_scan.cuh")


def coefficients():
    """Highest power first."""
    body = open(SRC).read().split("f2 log1p_unit(f2 u) {")[1].split("return")[0]
    c = [float(np.float32(a)) for a in re.findall(r"pack2\((-?[0-9.e-]+)f,", body)]
    assert len(c) == 9
    return c


def horner(c, u, after=lambda v: v):
    p = np.full_like(u, c[0])
    for k in c[1:]:
        p = after(p * u + k)  # an fp32 multiply-add: fp64 product and sum, rounded once
    return p


def test_log1p_polynomial_error():
    """The stated bounds: 3.4e-8 of the exact polynomial, 1.5e-7 as evaluated in
    fp32, where a mean error of small steps (which adds up over a state's memory)
    is far below a rounding."""
    c = coefficients()
    u = np.concatenate([np.logspace(-12, 0, 200001), np.linspace(1e-4, 1, 200001)])
    ref = np.log1p(u) / u
    assert np.abs(horner(c, u) / ref - 1).max() <= 3.4e-8
    u = u.astype(np.float32).astype(np.float64)
    f32 = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    err = f32(horner(c, u, f32) * u) / np.log1p(u) - 1
    assert np.abs(err).max() <= 1.5e-7
    assert abs(err.mean()) <= 2e-9
    assert abs(err[u < 1e-4].mean()) <= 1e-9
