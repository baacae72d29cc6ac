"""The 128-value forms (test oracle only): E4M3 quantizers with one scale per row
and 128 columns or per 128x128 block, the GEMM on them with its error bound,
silu(gate) * up and its gradient.  Plain numpy, fp64 (fp32 where the definition
says fp32).

The quantizer's rule is the one of the 32x32 blocks (DeepGEMM write-up, sections
2.1 and 5.2, on the group sizes of the determinism article's table, part 三,
section 2): s = fp32(amax / 448), code = E4M3(fp32(x / s)), round half to even,
clamped, sign kept; s == 0 gives 0x00.  A last block shorter than 128 is scaled
by itself.
"""

from __future__ import annotations

import numpy as np

from .e4m3 import decode_e4m3, encode_e4m3
from .e8m0 import code_exponents, step_bound

G128 = 128
E4M3_MAX = np.float32(448.0)


def _codes(x, s):
    """fp32 x of one group and its fp32 scale -> codes."""
    if s == 0:
        return np.zeros(x.shape, np.uint8)
    t = (x / np.float32(s)).astype(np.float32)
    return encode_e4m3(t)


def quantize_g128(x, band):
    """fp32 x [R, C] -> (codes uint8 [R, C], scales fp32 [ceil(R/band), ceil(C/128)]),
    groups of `band` rows (1 or 128) by 128 columns."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    q = np.zeros((R, C), np.uint8)
    s = np.zeros((-(-R // band), -(-C // G128)), np.float32)
    for rb in range(s.shape[0]):
        for cb in range(s.shape[1]):
            at = np.s_[rb * band:(rb + 1) * band, cb * G128:(cb + 1) * G128]
            s[rb, cb] = np.abs(x[at]).max() / E4M3_MAX
            q[at] = _codes(x[at], s[rb, cb])
    return q, s


def dequantize_g128(q, s, band):
    """The fp64 values of codes [R, C] with scales per `band` rows and 128 columns."""
    R, C = q.shape
    full = np.repeat(np.repeat(np.asarray(s, np.float64), band, 0)[:R], G128, 1)[:, :C]
    return decode_e4m3(q) * full


def gemm_g128_bound(qa, sa, qbt, sbt):
    """(ref, bound) of C = sum_kb sa[i,kb] sbt[j/128,kb] P for K-major weights.

    Per K-block: P is one 128-deep instruction with a zero accumulator (the
    summation model of the E8M0 GEMM, unit scales): its summation loss and half
    an fp32 ulp of P; the scale product is rounded once (2**-24), and so is the
    fused multiply-add (2**-24 of the running sum).  At the end half a bf16 step
    of the result.  K may be any length (missing codes are zeros)."""
    qa, qbt = np.asarray(qa, np.uint8), np.asarray(qbt, np.uint8)
    M, K = qa.shape
    N = qbt.shape[0]
    a, b = decode_e4m3(qa), decode_e4m3(qbt)
    xa, xb = code_exponents(qa), code_exponents(qbt)
    sa, sbt = np.asarray(sa, np.float64), np.asarray(sbt, np.float64)
    ref = np.zeros((M, N))
    B = np.zeros((M, N))
    u = 2.0 ** -24
    for kb, k0 in enumerate(range(0, K, G128)):
        ks = slice(k0, min(K, k0 + G128))
        pad = G128 - (ks.stop - ks.start)
        wide = [(0, 0), (0, 0), (0, pad)]
        absp = np.pad(np.abs(a[:, None, ks]) * np.abs(b[None, :, ks]), wide)
        S = np.pad(xa[:, None, ks] + xb[None, :, ks], wide, constant_values=-12)
        loss = step_bound(absp, S, np.zeros((M, N)))
        P = a[:, ks] @ b[:, ks].T
        s = np.abs(sa[:, kb])[:, None] * np.repeat(np.abs(sbt[:, kb]), G128)[:N][None, :]
        off = loss + u * (np.abs(P) + loss) + 2.0 ** -150
        ref = ref + sa[:, kb][:, None] * np.repeat(sbt[:, kb], G128)[:N][None, :] * P
        B = B + s * (1 + u) * off + u * s * np.abs(P) + 2.0 ** -150 * np.abs(P)
        B = B + u * (np.abs(ref) + B) + 2.0 ** -150
    return ref, (B + 2.0 ** -8 * (np.abs(ref) + B) + 2.0 ** -134) * (1.0 + 2.0 ** -30)


def swiglu(gu):
    """fp64 y [R, d] of gu [R, 2d] = [gate | up]."""
    gu = np.asarray(gu, np.float64)
    d = gu.shape[1] // 2
    g, u = gu[:, :d], gu[:, d:]
    return g / (1.0 + np.exp(-g)) * u


def swiglu_grad(gu, dy):
    """fp64 [dg | du] for dy [R, d]."""
    gu, dy = np.asarray(gu, np.float64), np.asarray(dy, np.float64)
    d = gu.shape[1] // 2
    g, u = gu[:, :d], gu[:, d:]
    s = 1.0 / (1.0 + np.exp(-g))
    return np.concatenate([dy * u * s * (1.0 + g * (1.0 - s)), dy * g * s], axis=1)


def e4m3_half_step(v):
    """Half the distance between E4M3 codes around |v| (at most, below 448)."""
    v = np.abs(np.asarray(v, np.float64))
    e = np.maximum(np.floor(np.log2(np.where(v > 0, v, 1.0))), -6)
    return np.where(v > 0, np.ldexp(1.0, e.astype(np.int64) - 4), 2.0 ** -10)
