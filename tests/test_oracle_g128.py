"""Pins of the 128-value oracle: against the 32-value oracle, brute force and differences."""

from fractions import Fraction

import numpy as np
import pytest

import oracle
from fp8_block_scaled_03_amd import workloads as W


def f32(bits):
    return oracle.bf16_bits_to_f32(bits)


def test_groups_of_32_columns_are_the_32_value_oracle():
    """A matrix of 32 columns is one partial group: the 1x32 token group."""
    x = W.normal_bf16(31, 0, 40, 32, 1.0, 0.05)
    q, s = oracle.quantize_g128(f32(x), 1)
    qo, so = oracle.quantize_token_groups(x)
    assert np.array_equal(q, qo) and np.array_equal(s, so)
    q, s = oracle.quantize_g128(f32(x)[:32], 128)
    qo, so = oracle.quantize_blocks(x[:32])
    assert np.array_equal(q, qo) and np.array_equal(s, so)


def test_blocks_transpose():
    x = f32(W.normal_bf16(32, 0, 200, 144, 1.0, 0.05))
    q, s = oracle.quantize_g128(x, 128)
    qt, st = oracle.quantize_g128(np.ascontiguousarray(x.T), 128)
    assert np.array_equal(q.T, qt) and np.array_equal(s.T, st)


def test_half_step_bounds_every_code():
    x = f32(W.normal_bf16(33, 0, 30, 272, 1.0, 0.05))
    q, s = oracle.quantize_g128(x, 1)
    full = np.repeat(s.astype(np.float64), 128, 1)[:, :272]
    off = np.abs(oracle.dequantize_g128(q, s, 1) - x) / full
    # the fp32 quotient is rounded before the code is
    assert (off <= oracle.e4m3_half_step(x / full * (1 + 2.0 ** -20)) + 448 * 2.0 ** -23).all()


def test_gemm_reference_is_exact_brute_force():
    rng = np.random.default_rng(5)
    M, N, K = 3, 130, 272
    qa = rng.integers(0, 256, (M, K)).astype(np.uint8) & 0xF7
    qb = rng.integers(0, 256, (N, K)).astype(np.uint8) & 0xF7
    sa = rng.uniform(0.01, 2, (M, 3)).astype(np.float32)
    sb = rng.uniform(0.01, 2, (2, 3)).astype(np.float32)
    ref, bound = oracle.gemm_g128_bound(qa, sa, qb, sb)
    a, b = oracle.decode_e4m3(qa), oracle.decode_e4m3(qb)
    for i, j in [(0, 0), (2, 129), (1, 127), (0, 128)]:
        want = sum(Fraction(float(sa[i, k // 128])) * Fraction(float(sb[j // 128, k // 128]))
                   * Fraction(float(a[i, k])) * Fraction(float(b[j, k])) for k in range(K))
        assert abs(ref[i, j] - float(want)) <= 1e-12 * (np.abs(a[i]) @ np.abs(b[j])) * 4
    assert (bound > 0).all()


def test_bound_covers_the_emulated_instruction():
    """One K-block with unit scales against the exact-rational emulation of the instruction."""
    rng = np.random.default_rng(6)
    qa = rng.integers(0, 256, (2, 128)).astype(np.uint8) & 0xF7
    qb = rng.integers(0, 256, (32, 128)).astype(np.uint8) & 0xF7
    one = np.ones((2, 1), np.float32)
    ref, bound = oracle.gemm_g128_bound(qa, one, qb, np.ones((1, 1), np.float32))
    zero = np.full((1, 4), 127, np.uint8)
    for later in ("exact", "grid", "drop"):
        out = oracle.emulate_gemm_e8m0_nt(qa, zero, qb, zero, later=later)
        assert all(abs(float(out[i, j]) - ref[i, j]) <= bound[i, j] for i in range(2) for j in range(32))


@pytest.mark.parametrize("scale", [0.1, 1.0, 5.0])
def test_swiglu_gradient_against_differences(scale):
    rng = np.random.default_rng(7)
    gu = rng.normal(size=(4, 24)) * scale
    dy = rng.normal(size=(4, 12))
    grad = oracle.swiglu_grad(gu, dy)
    h = 1e-6
    for i, j in [(0, 0), (1, 5), (3, 11), (2, 12), (0, 23)]:
        up, down = gu.copy(), gu.copy()
        up[i, j] += h
        down[i, j] -= h
        d = ((oracle.swiglu(up) - oracle.swiglu(down)) * dy).sum() / (2 * h)
        assert abs(d - grad[i, j]) <= 1e-7 * max(1.0, abs(d))
