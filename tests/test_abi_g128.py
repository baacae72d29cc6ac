"""The entry points of include/fp8bs_g128.h are exported and refuse bad
arguments on the host before any launch (CPU only: no GPU call is made)."""

import os
import re

import pytest
import torch

import fp8_block_scaled_03_amd as fp8bs
from fp8_block_scaled_03_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, ESHAPE, EALIGN = 0, 1, 2, 3
A16 = 0x10000          # fake, 16-byte aligned "device" addresses: never dereferenced
A4 = 0x10004
BIG = 1 << 30


def test_library_exports_every_declared_symbol():
    lib = binding.load_library()
    text = open(os.path.join(ROOT, "include", "fp8bs_g128.h")).read()
    names = set(re.findall(r"^fp8bs_status (fp8bs_[a-z0-9_]+)\(", text, re.M))
    assert names == {"fp8bs_quantize_tg128", "fp8bs_quantize_b128", "fp8bs_gemm_tg128_nt",
                     "fp8bs_grouped_gemm_tg128_nt", "fp8bs_grouped_wgrad", "fp8bs_swiglu_quantize_tg128",
                     "fp8bs_swiglu_backward_quantize_tg128"}
    for n in names:
        assert hasattr(lib, n), n
        assert hasattr(fp8bs, n[len("fp8bs_"):]), n


def test_quantize_tg128_refusals():
    q = binding.quantize_tg128_raw
    assert q(A16, 0, 64, A16, A4) == OK and q(A16, 5, 0, A16, A4) == OK
    assert q(None, 0, 64, None, None) == OK
    assert q(A16, -1, 64, A16, A4) == EINVAL and q(A16, 1, -16, A16, A4) == EINVAL
    assert q(A16, 4, 40, A16, A4) == ESHAPE
    assert q(A16, BIG + 1, 64, A16, A4) == ESHAPE and q(A16, 4, BIG + 16, A16, A4) == ESHAPE
    for bad in [(None, A16, A4), (A16, None, A4), (A16, A16, None)]:
        assert q(bad[0], 4, 64, bad[1], bad[2]) == EINVAL
    for bad in [(A16 + 8, A16, A4), (A16, A16 + 4, A4), (A16, A16, A4 + 2)]:
        assert q(bad[0], 4, 64, bad[1], bad[2]) == EALIGN


def test_quantize_b128_refusals():
    q = binding.quantize_b128_raw
    assert q(A16, 2, 0, 64, A16, A4, None, None) == OK and q(A16, 2, 64, 0, A16, A4, None, None) == OK
    assert q(A16, 0, 64, 64, A16, A4, None, None) == EINVAL
    assert q(A16, 1, -1, 64, A16, A4, None, None) == EINVAL
    assert q(A16, 1, 64, 64, A16, A4, A16, None) == EINVAL      # qt without its scales
    assert q(A16, 1, 64, 64, A16, A4, None, A4) == EINVAL
    assert q(A16, 1, 64, 40, A16, A4, None, None) == ESHAPE
    assert q(A16, 1, 40, 64, A16, A4, A16, A4) == ESHAPE        # rows % 16 with the transpose
    assert q(A16, 1, BIG, BIG, A16, A4, None, None) == ESHAPE   # too many blocks
    assert q(A16, BIG, BIG, 16, A16, A4, None, None) == ESHAPE
    for bad in [(None, A16, A4), (A16, None, A4), (A16, A16, None)]:
        assert q(bad[0], 1, 64, 64, bad[1], bad[2], None, None) == EINVAL
    assert q(A16 + 8, 1, 64, 64, A16, A4, None, None) == EALIGN
    assert q(A16, 1, 64, 64, A16, A4 + 1, None, None) == EALIGN
    assert q(A16, 1, 64, 64, A16, A4, A16 + 8, A4) == EALIGN
    assert q(A16, 1, 64, 64, A16, A4, A16, A4 + 1) == EALIGN


def test_gemm_refusals():
    g = binding.gemm_tg128_nt_raw
    assert g(None, None, None, None, None, 0, 64, 64) == OK and g(A16, A4, A16, A4, A16, 4, 0, 64) == OK
    assert g(A16, A4, A16, A4, A16, -4, 64, 64) == EINVAL
    assert g(A16, A4, A16, A4, A16, 4, 40, 64) == ESHAPE and g(A16, A4, A16, A4, A16, 4, 64, 40) == ESHAPE
    assert g(A16, A4, A16, A4, A16, BIG + 1, 64, 64) == ESHAPE
    assert g(A16, A4, A16, A4, A16, 4, BIG + 16, 64) == ESHAPE
    assert g(A16, A4, A16, A4, A16, 4, 64, (1 << 22) + 16) == ESHAPE
    for i in range(5):
        p = [A16, A4, A16, A4, A16]
        p[i] = None
        assert g(*p, 4, 64, 64) == EINVAL
    for i in range(5):
        p = [A16, A4, A16, A4, A16]
        p[i] += 2
        assert g(*p, 4, 64, 64) == EALIGN


def test_grouped_gemm_refusals():
    g = binding.grouped_gemm_tg128_nt_raw
    assert g(A16, A4, A16, A4, A4, 0, A16, 64, 64, 64) == EINVAL
    assert g(A16, A4, A16, A4, A4, 1025, A16, 64, 64, 64) == EINVAL
    assert g(A16, A4, A16, A4, None, 2, A16, 64, 64, 64) == EINVAL
    assert g(A16, A4, A16, A4, A4 + 1, 2, A16, 64, 64, 64) == EALIGN
    assert g(A16, A4, A16, A4, A4, 2, A16, 0, 64, 64) == OK
    assert g(A16, A4, A16, A4, A4, 2, A16, 64, 0, 64) == OK
    assert g(A16, A4, A16, A4, A4, 2, A16, 5, 40, 64) == ESHAPE
    assert g(A16, A4, A16, A4, A4, 2, A16, -5, 64, 64) == EINVAL
    assert g(A16, A4, A16, A4, A4, 2, None, 5, 64, 64) == EINVAL
    assert g(A16, A4, A16 + 4, A4, A4, 2, A16, 5, 64, 64) == EALIGN


def test_wgrad_refusals():
    g = binding.grouped_wgrad_raw
    assert g(A16, A16, A4, 0, A16, 0, 5, 64, 64) == EINVAL
    assert g(A16, A16, A4, 1025, A16, 0, 5, 64, 64) == EINVAL
    assert g(A16, A16, None, 2, A16, 0, 5, 64, 64) == EINVAL
    assert g(A16, A16, A4 + 2, 2, A16, 0, 5, 64, 64) == EALIGN
    assert g(A16, A16, A4, 2, A16, 0, 5, 0, 64) == OK and g(A16, A16, A4, 2, A16, 0, 5, 64, 0) == OK
    assert g(A16, A16, A4, 2, A16, 0, 5, 40, 64) == ESHAPE and g(A16, A16, A4, 2, A16, 0, 5, 64, 40) == ESHAPE
    assert g(A16, A16, A4, 2, A16, 0, 5, (1 << 22) + 16, 64) == ESHAPE
    assert g(A16, A16, A4, 2, A16, 0, -5, 64, 64) == EINVAL
    assert g(A16, A16, A4, 2, None, 0, 5, 64, 64) == EINVAL
    assert g(None, A16, A4, 2, A16, 0, 5, 64, 64) == EINVAL
    assert g(A16, None, A4, 2, A16, 0, 5, 64, 64) == EINVAL
    for i in (0, 1, 4):
        p = [A16, A16, A4, 2, A16, 0, 5, 64, 64]
        p[i] += 8
        assert g(*p) == EALIGN


def test_swiglu_refusals():
    f = binding.swiglu_quantize_tg128_raw
    assert f(A16, 0, 64, A16, A4, None) == OK and f(A16, 4, 0, A16, A4, None) == OK
    assert f(A16, -1, 64, A16, A4, None) == EINVAL
    assert f(A16, 4, 40, A16, A4, None) == ESHAPE and f(A16, 4, (1 << 29) + 16, A16, A4, None) == ESHAPE
    assert f(None, 4, 64, A16, A4, None) == EINVAL and f(A16, 4, 64, None, A4, None) == EINVAL
    assert f(A16, 4, 64, A16, None, None) == EINVAL
    assert f(A16, 4, 64, A16, A4, A16 + 8) == EALIGN and f(A16 + 8, 4, 64, A16, A4, None) == EALIGN
    b = binding.swiglu_backward_quantize_tg128_raw
    assert b(A16, A16, 0, 64, A16, A16, A4, None) == OK
    assert b(A16, A16, 4, 40, A16, A16, A4, None) == ESHAPE
    assert b(A16, A16, -4, 64, A16, A16, A4, None) == EINVAL
    for i in (0, 1, 4, 5, 6):
        p = [A16, A16, 4, 64, A16, A16, A4, None]
        p[i] = None
        assert b(*p) == EINVAL
        p[i] = A4 + 2
        assert b(*p) == EALIGN
    assert b(A16, A16, 4, 64, A16, A16, A4, A16 + 8) == EALIGN


def test_tensor_api_rejects_bad_inputs_without_gpu():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fp8bs.quantize_tg128(x.float())
    with pytest.raises(ValueError):
        fp8bs.quantize_tg128(x)                     # not on a GPU
    with pytest.raises(ValueError):
        fp8bs.quantize_tg128(x.t())                 # not contiguous
    with pytest.raises(ValueError):
        fp8bs.quantize_b128(x[0])                   # one dimension
    with pytest.raises(ValueError):
        fp8bs.swiglu_quantize_tg128(x)
