"""The polynomials of the normal distribution's tail as the source holds them, against erfcx in float64 (CPU only):
Q(t) = exp(t^2 / 2) erfc(t / sqrt 2) / 2 within what the source states."""

import math
import os
import re

import numpy as np
import pytest
import torch

from fp8_block_scaled_03_amd import build

U = 2.0 ** -24


def f32(v):
    return np.asarray(v).astype(np.float32).astype(np.float64)


def source(function):
    """(a, coefficients from the highest) of u = 1 / (1 + a t) and its polynomial, as fp32 holds them."""
    text = open(os.path.join(build.CSRC, "activation.hpp")).read()
    body = text[text.index(function):]
    body = body[:body.index("\n}\n")]
    number = r"(-?[\d.]+(?:e-?\d+)?)f"
    a = re.search(r"rcpf\(__builtin_fmaf\(t, " + number, body).group(1)
    c = re.findall(r"float q = " + number, body) + re.findall(r"q = __builtin_fmaf\(q, u, " + number, body)
    return float(f32(float(a))), [float(f32(float(v))) for v in c]


def tail_ratio(t):
    return 0.5 * torch.special.erfcx(torch.from_numpy(t) / math.sqrt(2)).numpy()


def grid(high):
    return f32(np.concatenate([np.linspace(0, high, 300001), np.geomspace(1e-30, high, 20001)]))


def evaluated(t, a, c, rounded=lambda v: v, reciprocal=lambda v: v):
    """As the source does it; a fused multiply-add rounds once (the float64 sum's own rounding is far below)."""
    u = reciprocal(rounded(1.0 / rounded(t * a + 1.0)))
    q = np.full_like(t, c[0])
    for v in c[1:]:
        q = rounded(q * u + v)
    return rounded(q * u)


def off(t, got):
    want = tail_ratio(t)
    return (np.abs(got - want) / want).max()


def test_the_gradients_polynomial():
    a, c = source("float normal_tail_ratio(")
    assert len(c) == 9
    t = grid(14.5)
    assert off(t, evaluated(t, a, c)) <= 0.76 * U
    for ulp in (0.0, np.inf, -np.inf):  # the reciprocal's last bit either way
        def reciprocal(v):
            return v if ulp == 0.0 else np.nextafter(v.astype(np.float32), np.float32(ulp)).astype(np.float64)
        assert off(t, evaluated(t, a, c, f32, reciprocal)) <= 9.5 * U


def test_the_results_polynomial():
    a, c = source("float gelu(")
    assert len(c) == 6
    t = grid(13.3)
    assert off(t, evaluated(t, a, c)) <= 4e-6
    assert off(t, evaluated(t, a, c, f32)) <= 4.5e-6


@pytest.mark.parametrize("k", range(9))
def test_another_coefficient_is_seen(k):
    a, c = source("float normal_tail_ratio(")
    c[k] = float(np.nextafter(np.float32(c[k]), np.float32(10)) * (1 + 2.0 ** -19))
    t = grid(14.5)
    assert off(t, evaluated(t, a, c)) > 0.76 * U
