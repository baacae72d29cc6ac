"""silu(gate) * up and its gradient where the gates of a group lie far from zero: the fp32 scales show the fp32
values behind them, which bf16 results and codes round away.

With u = 2^-24 an fp32 operation is off by at most u of its value.  exp(-|g|): the two roundings of the reduced
exponent (at most 1/2 + u, so 2^-25 each, times ln 2) 0.7 u and the hardware's exp2 2 u; 1 + e, its reciprocal and
their product u each: sigma within 5.7 u.  g sigma and the division by 448 make it 7.7 u, a factor `up` that is not one
8.7 u.  The slope sigma (1 + g (1 - sigma)) for g <= -11 has sigma's 5.7 u, 3 u of its second term, which is at most
1.1 of the sum, and u of the sum: 10 u; with the division 11 u, with dy * up (exact in fp32) not one 12 u.  Half a u
covers the second order."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def gates(lo, hi):
    """Every bf16 value of [lo, hi], both positive."""
    v = torch.arange(0x0080, 0x7F80, dtype=torch.int16).view(torch.bfloat16)
    return v[(v >= lo) & (v <= hi)]


def one_per_row(values, d):
    """[R, 2d]: gate r in column r % d of row r, up 1 there, zeros elsewhere; and dy alike."""
    R = len(values)
    row, col = torch.arange(R), torch.arange(R) % d
    gu, dy = torch.zeros(R, 2 * d, dtype=torch.bfloat16), torch.zeros(R, d, dtype=torch.bfloat16)
    gu[row, col], gu[row, d + col], dy[row, col] = values, 1.0, 1.0
    return gu, dy


def filled(seed, values, rows, d):
    """[rows, 2d] with gates drawn from `values`, normal ups and dys."""
    gen = torch.Generator().manual_seed(seed)
    at = torch.randint(0, len(values), (rows, d), generator=gen)
    up, dy = (torch.randn(rows, d, generator=gen).bfloat16() for _ in range(2))
    return torch.cat([values[at], up], 1), dy


def scales_are(s, exact, tol):
    """s = max |exact| / 448 of each group of 128 columns, within `tol` of it."""
    s = s.cpu().double().numpy()
    want = np.stack([np.abs(exact[:, c:c + 128]).max(1) for c in range(0, exact.shape[1], 128)], 1) / 448
    rel = np.abs(s - want) / np.where(want > 0, want, 1)
    assert rel.max() <= tol * U, (float(rel.max() / U), np.unravel_index(rel.argmax(), rel.shape))


@pytest.mark.parametrize("d", [128, 144])
@pytest.mark.parametrize("sign", [-1, 1])
def test_every_gate_alone_in_its_row(d, sign):
    say(f"swiglu, one gate a row, sign {sign}, d {d}")
    v = gates(2.0 ** -7, 80.0) * sign
    gu, dy = one_per_row(v, d)
    _, s = fp8bs.swiglu_quantize_tg128(gu.to(DEV))
    scales_are(s, oracle.swiglu(gu.double().numpy()), 8.2)
    gu, dy = one_per_row(v[v.abs() >= 11], d)
    if d == 128:   # the two halves have groups of their own
        _, _, s = fp8bs.swiglu_backward_quantize_tg128(gu.to(DEV), dy.to(DEV))
        exact = oracle.swiglu_grad(gu.double().numpy(), dy.double().numpy())
        scales_are(s[:, :1], exact[:, :d], 11.5)
        scales_are(s[:, 1:], exact[:, d:], 8.2)


@pytest.mark.parametrize("rows,d", [(1, 128), (70, 400), (33, 1024)])
def test_groups_of_far_negative_gates(rows, d):
    say(f"swiglu, gates of [-80, -11], {rows}x{d}")
    gu, dy = filled(rows + d, -gates(11.0, 80.0), rows, d)
    _, s = fp8bs.swiglu_quantize_tg128(gu.to(DEV))
    scales_are(s, oracle.swiglu(gu.double().numpy()), 9.2)
    _, _, s = fp8bs.swiglu_backward_quantize_tg128(gu.to(DEV), dy.to(DEV))
    scales_are(s, oracle.swiglu_grad(gu.double().numpy(), dy.double().numpy()), 12.5)
