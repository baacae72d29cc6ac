"""The digits of layer norm's mean, and of deviations that are far below the row's own: values are multiples of 2^-6
below 4, so that sums of up to 32 are exact in fp32 and the 64-bit sum over the lanes is exact.  U = 2^-24.

The mean is then mu rounded once, U |mu|, and 2^-45 for what 64 bits lose.  A deviation is (h - m) - delta with two
roundings of 32 bits and no error of the mean's beside delta's own U^2 |mu|; rstd is off by half of (46 + 3) U (sums
46 additions deep, two roundings of a squared deviation, its product's) and 3 U for the sum, root and quotient, and
y by a rounding for each product:
    |y - ref| <= rstd (31 U |h - mu| + 2 U^2 |mu|),  without weight and bias, and the scale of 128 of them has one more."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


def rows_of(rows, d, shift):
    """Multiples of 2^-6 below 4 in magnitude; of the first 128 columns all of a row are the one next to its mean."""
    g = torch.Generator().manual_seed(d)
    h = ((torch.randn(rows, d, generator=g) * 0.8 + shift).clamp(-3.98, 3.98) * 64).round() / 64
    if d >= 256:
        mean = h[:, 128:].double().mean(1, keepdim=True)
        h[:, :128] = ((mean * 64).round() / 64).float()
    assert torch.equal(h.to(torch.bfloat16).float(), h)
    return h.to(torch.bfloat16)


@pytest.mark.parametrize("d", [16, 48, 256, 272, 512, 528, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 16384])
@pytest.mark.parametrize("shift", [0.0, 0.25, 1.3, -2.0])
def test_mean_and_small_deviations(d, shift):
    rows = 64
    h = rows_of(rows, d, shift)
    x = h.to(DEV)
    say(f"layernorm digits {rows}x{d} {shift}")
    ones = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    q, s, mean, rstd = fp8bs.layernorm_quantize_tg128(x, ones, None, EPS, want_stats=True)
    h = h.double().numpy()
    mu = h.mean(1)
    rs = 1.0 / np.sqrt(((h - mu[:, None]) ** 2).mean(1) + EPS)
    assert (np.abs(mean.cpu().double().numpy() - mu) <= U * np.abs(mu) + 2.0 ** -45).all()
    assert (np.abs(rstd.cpu().double().numpy() - rs) <= 29 * U * rs).all()
    s = s.cpu().double().numpy()
    for b in range(s.shape[1]):
        y = np.abs((h[:, 128 * b:128 * b + 128] - mu[:, None]) * rs[:, None]).max(1)
        off = 31 * U * y + rs * 2 * U * U * np.abs(mu)
        assert (np.abs(s[:, b] - y / 448) <= off / 448 + U * y / 448 + 2.0 ** -149).all(), b


@pytest.mark.parametrize("d", [16, 48, 272, 512, 1040, 2064, 4096, 8208, 16368])
@pytest.mark.parametrize("value", [3.0, -0.1, 1e-20, 1000.0, 1e30, 2.0 ** -130])
def test_equal_values_are_their_mean(d, value):
    x = torch.full((3, d), value, dtype=torch.bfloat16, device=DEV)
    gamma, beta = torch.ones(d, dtype=torch.bfloat16, device=DEV), torch.full((d,), 0.5, dtype=torch.bfloat16,
                                                                              device=DEV)
    say(f"equal values {d} {value}")
    for b, want in ((None, 0.0), (beta, 0.5)):
        q, s, y, mean, rstd = fp8bs.layernorm_quantize_tg128(x, gamma, b, EPS, want_y=True, want_stats=True)
        assert torch.equal(mean, x[:, 0].float()) and (y == want).all()
        assert ((q & 0x7F == 0).all() and (s == 0).all()) if b is None else (s == np.float32(0.5) / 448).all()
