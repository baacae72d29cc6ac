"""The entry points of include/fp8bs_layer.h are exported and refuse bad arguments on the host before any launch
(CPU only: no GPU call is made)."""

import ctypes
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
    text = open(os.path.join(ROOT, "include", "fp8bs_layer.h")).read()
    names = set(re.findall(r"^(?:fp8bs_status|int64_t) (fp8bs_[a-z0-9_]+)\(", text, re.M))
    assert "fp8bs_clip_grad_norm" in names
    for n in names:
        assert hasattr(lib, n), n
        if not n.endswith("_workspace"):
            assert hasattr(fp8bs, n[len("fp8bs_"):]), n


def test_layernorm_refusals():
    f = binding.layernorm_quantize_tg128_raw
    ok = [A16, A16, A16, A16, 1e-5, 4, 64, A16, A16, A4, A16, A4, A4]

    def with_(**at):
        p = list(ok)
        for i, v in at.items():
            p[int(i[1:])] = v
        return f(*p)

    assert with_(_5=0) == OK and with_(_6=0) == OK and with_(_5=0, _0=None, _2=None, _8=None, _9=None) == OK
    assert with_(_5=-1) == EINVAL and with_(_6=-16) == EINVAL
    for eps in (-1e-9, float("nan"), float("inf")):
        assert with_(_4=eps) == EINVAL
    assert with_(_6=40) == ESHAPE and with_(_6=16400) == ESHAPE and with_(_5=BIG + 1) == ESHAPE
    for i in (0, 2, 8, 9, 11, 12):
        assert with_(**{f"_{i}": None}) == EINVAL
    for i in (0, 1, 2, 3, 7, 8, 10):
        assert with_(**{f"_{i}": A16 + 8}) == EALIGN
    for i in (9, 11, 12):
        assert with_(**{f"_{i}": A4 + 2}) == EALIGN
    g = binding.layernorm_raw
    assert g(A16, None, A16, None, 1e-5, 0, 64, None, A16, None, None) == OK
    assert g(A16, None, A16, None, 1e-5, 4, 64, None, None, None, None) == EINVAL
    assert g(A16, None, A16, None, 1e-5, 4, 64, None, A16, A4, None) == EINVAL
    assert g(A16, None, A16, None, 1e-5, 4, 65, None, A16, None, None) == ESHAPE


def test_layernorm_backward_refusals():
    lib = binding.load_library()
    size = lib.fp8bs_layernorm_backward_workspace(4, 64)
    assert size > 0 and lib.fp8bs_layernorm_backward_workspace(0, 64) == 0
    assert lib.fp8bs_layernorm_backward_workspace(-1, 64) == 0
    assert lib.fp8bs_layernorm_backward_workspace(4, 16400) == 0
    ok = [A16, A16, A16, A4, A4, A16, 4, 64, A16, A4, A4, 0, A16, size]

    def with_(**at):
        p = list(ok)
        for i, v in at.items():
            p[int(i[1:])] = v
        return binding.layernorm_backward_raw(*p)

    assert with_(_7=0) == OK
    assert with_(_6=-1) == EINVAL and with_(_7=-16) == EINVAL
    assert with_(_7=24) == ESHAPE and with_(_7=16400) == ESHAPE and with_(_6=BIG + 1) == ESHAPE
    for i in (0, 1, 2, 3, 4, 8, 12):
        assert with_(**{f"_{i}": None}) == EINVAL
    assert with_(_13=size - 1) == EINVAL
    for i in (0, 1, 2, 5, 8, 12):
        assert with_(**{f"_{i}": A16 + 8}) == EALIGN
    for i in (3, 4, 9, 10):
        assert with_(**{f"_{i}": A4 + 2}) == EALIGN


def _changed(call, ok):
    def with_(**at):
        p = list(ok)
        for i, v in at.items():
            p[int(i[1:])] = v
        return call(*p)
    return with_


def test_epilogue_refusals():
    with_ = _changed(binding.gemm_tg128_nt_epilogue_raw, [A16, A4, A16, A4, A16, 2, A16, A16, A16, 4, 64, 64])
    assert with_(_9=0) == OK and with_(_10=0) == OK and with_(_9=0, _0=None, _7=None) == OK
    assert with_(_5=-1) == EINVAL and with_(_5=5) == EINVAL
    assert with_(_9=-1) == EINVAL and with_(_10=40) == ESHAPE and with_(_11=40) == ESHAPE
    assert with_(_9=BIG + 1) == ESHAPE and with_(_11=(1 << 22) + 16) == ESHAPE
    for i in (0, 1, 2, 3, 7):
        assert with_(**{f"_{i}": None}) == EINVAL
    for i in (0, 2, 4, 6, 7, 8):
        assert with_(**{f"_{i}": A16 + 8}) == EALIGN
    for i in (1, 3):
        assert with_(**{f"_{i}": A4 + 2}) == EALIGN

    for same in (A16 + 256, A16 + 512):  # z stored over the result or over the residual
        assert with_(_6=A16 + 256, _7=A16 + 512, _8=same) == EINVAL


def test_epilogue_backward_refusals():
    lib = binding.load_library()
    size = lib.fp8bs_epilogue_backward_workspace(4, 64)
    assert size >= 256 and lib.fp8bs_epilogue_backward_workspace(0, 64) == 0
    assert lib.fp8bs_epilogue_backward_workspace(4, -16) == 0
    with_ = _changed(binding.epilogue_backward_quantize_tg128_raw,
                     [A16, A16, 2, 4, 64, A16, A16, A4, A4, 0, A16, size])
    assert with_(_4=0) == OK
    assert with_(_2=-1) == EINVAL and with_(_2=5) == EINVAL and with_(_3=-1) == EINVAL and with_(_4=-16) == EINVAL
    assert with_(_4=24) == ESHAPE and with_(_3=BIG + 1) == ESHAPE and with_(_4=BIG + 16) == ESHAPE
    for i in (0, 1, 6, 7, 10):
        assert with_(**{f"_{i}": None}) == EINVAL
    assert with_(_11=size - 1) == EINVAL
    for i in (0, 1, 5, 6, 10):
        assert with_(**{f"_{i}": A16 + 8}) == EALIGN
    for i in (7, 8):
        assert with_(**{f"_{i}": A4 + 2}) == EALIGN


def test_moe_refusals():
    lib = binding.load_library()
    size = lib.fp8bs_moe_decode_b128_workspace(3, 2, 4, 64, 64)
    assert size > 0
    for bad in ((-1, 2, 4, 64, 64), (3, 0, 4, 64, 64), (3, 2, 0, 64, 64), (3, 2, 1025, 64, 64), (3, 2, 4, 64, 0),
                (3, 2, 4, 64, 24), (3, 2, 4, 24, 64), (257, 2, 4, 64, 64), (1 << 40, 1 << 40, 4, 64, 64),
                (0, 2, 4, 64, 64)):
        assert lib.fp8bs_moe_decode_b128_workspace(*bad) == 0
    ok = [A16, A4, A4, A16, A4, A16, A4, A16, A16, 3, 2, 4, 64, 64, A16, size]
    with_ = _changed(binding.moe_decode_b128_raw, ok)
    assert with_(_9=0) == OK and with_(_12=0) == OK
    assert with_(_9=-1) == EINVAL and with_(_10=0) == EINVAL and with_(_11=0) == EINVAL and with_(_11=1025) == EINVAL
    assert with_(_12=-16) == EINVAL and with_(_13=-16) == EINVAL
    assert with_(_9=257) == ESHAPE and with_(_10=513) == ESHAPE and with_(_9=1 << 40, _10=1 << 40) == ESHAPE
    assert with_(_12=40) == ESHAPE and with_(_13=40) == ESHAPE and with_(_13=0) == ESHAPE
    assert with_(_12=32784) == ESHAPE and with_(_13=32784) == ESHAPE
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 14):
        assert with_(**{f"_{i}": None}) == EINVAL
    assert with_(_15=size - 1) == EINVAL
    for i in (0, 3, 5, 7, 8, 14):
        assert with_(**{f"_{i}": A16 + 8}) == EALIGN
    for i in (1, 2, 4, 6):
        assert with_(**{f"_{i}": A4 + 2}) == EALIGN


# ---- gradients ---------------------------------------------------------------------------
def _arrays(pointers, counts, types):
    n = len(pointers)
    return (ctypes.c_void_p * n)(*pointers), (ctypes.c_int64 * n)(*counts), (ctypes.c_int32 * n)(*types)


def _norm(pointers, counts, types, norm=A4, ws=A16, size=None, n=None):
    p, c, t = _arrays(pointers, counts, types)
    n = len(pointers) if n is None else n
    size = binding.load_library().fp8bs_grad_norm_workspace(n) if size is None else size
    return binding.grad_norm_raw(p, c, t, n, norm, ws, size)


def _clip(pointers, outs, counts, types, max_norm=1.0, eps=1e-6, norm=A4, ws=A16, size=1 << 20):
    p, c, t = _arrays(pointers, counts, types)
    o = (ctypes.c_void_p * len(outs))(*outs)
    both = binding.clip_grad_norm_raw(p, o, c, t, len(pointers), max_norm, eps, norm, ws, size)
    if ws == A16 and size == 1 << 20:
        assert binding.clip_grads_raw(p, o, c, t, len(pointers), norm, max_norm, eps) == both
    return both


def test_grad_norm_refusals():
    assert _norm([A16], [4], [0], n=-1) == EINVAL and _norm([A16], [4], [0], n=65537) == EINVAL
    assert _norm([A16], [-1], [0]) == EINVAL and _norm([A16], [4], [2]) == EINVAL and _norm([A16], [4], [-1]) == EINVAL
    assert _norm([None], [4], [0]) == EINVAL and _norm([A16], [4], [0], norm=None) == EINVAL
    assert _norm([A16], [4], [0], ws=None) == EINVAL and _norm([A16], [4], [0], size=64) == EINVAL
    assert _norm([A16 + 2], [4], [0]) == EALIGN and _norm([A16 + 1], [4], [1]) == EALIGN
    assert _norm([A16], [4], [0], norm=A4 + 2) == EALIGN and _norm([A16], [4], [0], ws=A16 + 8) == EALIGN
    assert _norm([A16], [(1 << 36) + 1], [0]) == ESHAPE
    lib = binding.load_library()
    assert lib.fp8bs_grad_norm(None, None, None, 1, A4, A16, 1 << 20, None) == EINVAL
    assert lib.fp8bs_grad_norm_workspace(1) <= lib.fp8bs_grad_norm_workspace(1000)


def test_clip_refusals():
    far = A16 + (1 << 20)
    for bad in (-1.0, float("nan"), float("inf")):
        assert _clip([A16], [A16], [4], [0], max_norm=bad) == EINVAL
        assert _clip([A16], [A16], [4], [0], eps=bad) == EINVAL
    assert _clip([A16], [None], [4], [0]) == EINVAL and _clip([A16], [far + 2], [4], [0]) == EALIGN
    assert _clip([A16], [A16], [4], [0], norm=None) == EINVAL
    assert _clip([A16], [A16], [4], [0], ws=None) == EINVAL and _clip([A16], [A16], [4], [0], size=8) == EINVAL
    # the same tensor twice, tensors that overlap, outputs over another gradient or over each other
    assert _clip([A16, A16], [A16, A16], [4, 4], [0, 0]) == EINVAL
    assert _clip([A16, A16 + 8], [A16, A16 + 8], [4, 4], [0, 0]) == EINVAL
    assert _clip([A16 + 8, A16], [A16 + 8, A16], [4, 4], [0, 1 - 1]) == EINVAL
    assert _clip([A16], [A16 + 4], [4], [0]) == EINVAL
    assert _clip([A16, far], [far, far + 64], [4, 4], [0, 0]) == EINVAL
    assert _clip([A16, A16 + 16], [far, far + 8], [4, 4], [0, 0]) == EINVAL


def test_norm_inside_a_gradient_is_refused():
    for norm in (A16, A16 + 12):
        assert _clip([A16], [A16], [4], [0], norm=norm) == EINVAL
        assert _clip([A16 + 64], [A16], [4], [0], norm=norm) == EINVAL
    p, c, t = _arrays([A16], [4], [0])
    o = (ctypes.c_void_p * 1)(A16 + 64)
    assert binding.clip_grad_norm_raw(p, o, c, t, 1, 1.0, 0.0, A16 + 4, A16, 1 << 20) == EINVAL  # written, and read


def test_gradient_lists_are_checked_without_gpu():
    x = torch.zeros(4, 32)
    for call in (fp8bs.grad_norm, lambda g: fp8bs.clip_grad_norm(g, 1.0)):
        with pytest.raises(ValueError):
            call([])
        with pytest.raises(ValueError):
            call([x])                       # not on a GPU
        with pytest.raises(TypeError):
            call([x.half()])
        with pytest.raises(TypeError):
            call([1.0])
