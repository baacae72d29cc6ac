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


def exactly(v):
    return v


def source(function, variable, argument):
    """(a, coefficients from the highest) of a function's polynomial, as fp32 holds them."""
    text = open(os.path.join(build.CSRC, "activation.hpp")).read()
    body = text[text.index(function):]
    body = body[:body.index("\n}\n")]
    number = r"(-?[\d.]+(?:e-?\d+)?)f"
    a = (re.search(r"constexpr float A = " + number, body) or
         re.search(r"rcpf\(__builtin_fmaf\(t, " + number, body)).group(1)
    c = re.findall(rf"float {variable} = " + number, body)
    c += re.findall(rf"{variable} = __builtin_fmaf\({variable}, {argument}, " + number, body)
    return float(f32(float(a))), [float(f32(float(v))) for v in c]


def tail_ratio(t):
    return 0.5 * torch.special.erfcx(torch.from_numpy(t) / math.sqrt(2)).numpy()


def grid(high):
    return f32(np.concatenate([np.linspace(0, high, 300001), np.geomspace(1e-30, high, 20001)]))


def horner(c, x, rounded):
    q = np.full_like(x, c[0])
    for v in c[1:]:  # a fused multiply-add rounds once (the float64 sum's own rounding is far below)
        q = rounded(q * x + v)
    return q


def reciprocal(v, rounded, ulp=0):
    r = rounded(1.0 / v)
    return r if ulp == 0 else np.nextafter(r.astype(np.float32), np.float32(ulp * np.inf)).astype(np.float64)


def gradients(t, a, c, rounded=exactly, ulp=0):
    """1/2 - v r(v), v = a t / (1 + a t)."""
    v = rounded(rounded(t * a) * reciprocal(rounded(t * a + 1.0), rounded, ulp))
    return rounded(0.5 - v * horner(c, v, rounded))


def gradients_error(t, got):
    """In 2^-24, by what may be off: as t phi(t) does it grows from t = 3 on."""
    return np.abs(got - tail_ratio(t)) / np.maximum(1.0, 0.3 * t) / U


def test_the_gradients_polynomial():
    a, c = source("float normal_tail_ratio(", "r", "v")
    assert len(c) == 8
    t = grid(14.5)
    assert gradients_error(t, gradients(t, a, c)).max() <= 0.15
    for ulp in (0, 1, -1):  # the reciprocal's last bit either way
        assert gradients_error(t, gradients(t, a, c, f32, ulp)).max() <= 1.5


def test_the_slope_on_ordinary_values():
    """exp(-t^2 / 2) (Q - t phi0), from 1 where z > 0, on normal bf16 z: 0.42 x 2^-24 rms off, a plain fp32 form with
    erfc and exp 0.45."""
    a, c = source("float normal_tail_ratio(", "r", "v")
    g = torch.Generator().manual_seed(0)
    z = (torch.randn(400000, generator=g, dtype=torch.float64) * 1.5).to(torch.bfloat16).double()
    want = (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)).numpy()
    plain = z.float()
    plain = (0.5 * torch.special.erfc(plain * -math.sqrt(0.5))
             + plain * torch.exp(-0.5 * plain * plain) * math.sqrt(0.5 / math.pi)).double().numpy()
    z = z.numpy()
    t = np.abs(z)
    for ulp in (0, 1, -1):
        q = gradients(t, a, c, f32, ulp)
        s = f32(f32(np.exp(-t * t / 2)) * f32(t * float(np.float32(-0.3989422917366028)) + q))
        got = np.where(z < 0, s, f32(1.0 - s))
        off = math.sqrt(((got - want) ** 2).mean())
        assert off <= 0.5 * U and off <= 1.1 * math.sqrt(((plain - want) ** 2).mean())


def results(t, a, c, rounded=exactly):
    """u q(u), u = 1 / (1 + a t)."""
    u = reciprocal(rounded(t * a + 1.0), rounded)
    return rounded(horner(c, u, rounded) * u)


def test_the_results_polynomial():
    a, c = source("float gelu(", "q", "u")
    assert len(c) == 6
    t = grid(13.3)
    want = tail_ratio(t)
    assert (np.abs(results(t, a, c) - want) / want).max() <= 4e-6
    assert (np.abs(results(t, a, c, f32) - want) / want).max() <= 4.5e-6


@pytest.mark.parametrize("k", range(8))
def test_another_coefficient_is_seen(k):
    a, c = source("float normal_tail_ratio(", "r", "v")
    c[k] *= 1 + 2.0 ** -18
    t = grid(14.5)
    assert gradients_error(t, gradients(t, a, c)).max() > 0.15
