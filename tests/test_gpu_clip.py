"""The norm over many gradients and their clipping, against 64-bit numpy.

Bounds: the norm's squares and sums are 64-bit, so it is off by its rounding to fp32 (2^-24) and by less than
2^-40 of 64-bit arithmetic.  A clipped value is off by the rounding of the factor (2^-24), of the fp32 product
(2^-24) and, for bf16, of the result (2^-8), and by half the smallest subnormal."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -150, BF16: 2.0 ** -134}


def make(seed, sizes, types, std=0.01):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(types[i % len(types)]).to(DEV) for i, n in enumerate(sizes)]


def np64(t):
    return t.cpu().double().numpy()


def norm64(grads):
    return np.sqrt(sum(float((np64(g) ** 2).sum()) for g in grads))


def check_norm(norm, grads):
    ref = norm64(grads)
    assert norm.dtype == F32 and norm.dim() == 0
    assert abs(float(norm) - ref) <= ref * (2.0 ** -24 + 2.0 ** -40)


def check_clipped(got, grads, max_norm, eps=1e-6, norm=None):
    factor = min(1.0, max_norm / ((norm64(grads) if norm is None else norm) + eps))
    for a, g in zip(got, grads):
        ref = np64(g) * factor
        assert a.dtype == g.dtype
        tol = np.abs(ref) * (2 * 2.0 ** -24 + (HALF[BF16] if g.dtype == BF16 else 0.0) + 2.0 ** -40) + TINY[g.dtype]
        assert (np.abs(np64(a) - ref) <= tol).all()


SIZES = [[1], [0], [3, 0, 1, 70000], [8192] * 5, [16384, 1, 8191, 8193, 5], list(range(0, 300)),
         [1 << 20, 7, 12345, 1 << 18, 3 * 2731 * 97]]


@pytest.mark.parametrize("types", [(F32,), (BF16,), (F32, BF16, F32)])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_norm_and_clip(sizes, types):
    say(f"clip {sizes[:6]} {types}")
    grads = make(len(sizes), sizes, types)
    check_norm(fp8bs.grad_norm(grads), grads)
    ref = norm64(grads)
    for max_norm in (0.37 * ref + 0.01, 2.0 * ref + 1.0):
        out = [torch.full_like(g, 9.0) for g in grads]
        norm = fp8bs.clip_grad_norm(grads, max_norm, out=out)
        check_norm(norm, grads)
        check_clipped(out, grads, max_norm)
        here = [g.clone() for g in grads]
        fp8bs.clip_grad_norm(here, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(here, out))
        fp8bs.clip_grads(grads, norm, max_norm, out=out)
        check_clipped(out, grads, max_norm, norm=float(norm))
        if max_norm > ref:
            assert all(torch.equal(a, b) for a, b in zip(here, grads))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lead", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("n", [1, 2, 9, 16383, 16384, 40007])
def test_tensors_that_start_anywhere(dtype, lead, n):
    """Slices of a larger buffer: what lies before and behind them is not counted and not changed, and outputs may
    start at other places inside 16 bytes than their gradients."""
    whole = make(n + lead, [n + 64], (dtype,))[0]
    g = whole[lead:lead + n]
    say(f"slice {dtype} {lead} {n}")
    check_norm(fp8bs.grad_norm([g]), [g])
    for at in (lead, 0, 3):
        out = torch.full((n + 64,), 7.0, dtype=dtype, device=DEV)
        fp8bs.clip_grad_norm([g], 0.001, out=[out[at:at + n]])
        check_clipped([out[at:at + n]], [g], 0.001)
        assert (out[:at] == 7.0).all() and (out[at + n:] == 7.0).all()
    old = whole.clone()
    fp8bs.clip_grad_norm([g], 0.001)
    check_clipped([g], [old[lead:lead + n]], 0.001)
    assert torch.equal(whole[:lead], old[:lead]) and torch.equal(whole[lead + n:], old[lead + n:])


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e15, 1e18])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_squares_beyond_fp32(scale, dtype):
    grads = make(3, [5000, 77], (dtype,), std=scale)
    say(f"scale {scale} {dtype}")
    check_norm(fp8bs.grad_norm(grads), grads)
    out = [torch.empty_like(g) for g in grads]
    fp8bs.clip_grad_norm(grads, scale, out=out, eps=0.0)
    check_clipped(out, grads, scale, eps=0.0)


def test_many_values_of_one_size():
    """2^24 equal values: a 32-bit running sum would stop growing."""
    g = torch.full((1 << 24,), 0.1, device=DEV)
    say("2^24 equal values")
    check_norm(fp8bs.grad_norm([g]), [g])


def test_not_finite():
    say("not finite")
    for bad in (float("inf"), float("-inf"), float("nan")):
        grads = make(5, [100, 40000], (F32, BF16))
        grads[1][39999] = bad
        norm = fp8bs.clip_grad_norm(grads, 1.0)
        if bad != bad:
            assert torch.isnan(norm) and all(torch.isnan(g).all() for g in grads)
        else:
            assert float(norm) == float("inf") and (grads[0] == 0).all()
            assert (grads[1][:-1] == 0).all() and torch.isnan(grads[1][-1])  # 0 * inf


def test_zero_gradients_and_zero_limit():
    say("zeros")
    grads = [torch.zeros(100, device=DEV), torch.zeros(0, device=DEV)]
    assert float(fp8bs.clip_grad_norm(grads, 1.0)) == 0.0 and (grads[0] == 0).all()
    grads = make(6, [1000], (F32,))
    fp8bs.clip_grad_norm(grads, 0.0)
    assert (grads[0] == 0).all()


def test_the_same_bits_every_time_and_in_a_graph():
    """Replays with other values in the same tensors, eager work between them, and a second stream."""
    sizes = [70001, 33, 1 << 20, 5, 8192]
    grads = make(7, sizes, (F32, BF16))
    out = [torch.empty_like(g) for g in grads]
    say("graph")
    fp8bs.clip_grad_norm(grads, 0.5, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = fp8bs.clip_grad_norm(grads, 0.5, out=out)
    for seed in (8, 9, 10):
        for g, new in zip(grads, make(seed, sizes, (F32, BF16))):
            g.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        eager = [torch.empty_like(g) for g in grads]
        want = fp8bs.clip_grad_norm(grads, 0.5, out=eager)
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, eager))
        check_norm(norm, grads)
    say("second stream")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = fp8bs.clip_grad_norm(grads, 0.5, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, want) and all(torch.equal(a, b) for a, b in zip(out, eager))


def test_outputs_over_gradients_are_refused():
    g = torch.ones(100, device=DEV)
    for grads, out in (([g, g], None), ([g[:60], g[40:]], None), ([g[:50]], [g[10:60]])):
        with pytest.raises(fp8bs.Fp8bsError):
            fp8bs.clip_grad_norm(grads, 1.0, out=out)
    assert (g == 1).all()
    assert abs(float(fp8bs.grad_norm([g, g])) - np.sqrt(200.0)) < 1e-5  # a norm may count a tensor twice
    one = torch.full((3, 5), 2.0, device=DEV)  # a tensor by itself
    check_norm(fp8bs.clip_grad_norm(one, 1.0), [torch.full((3, 5), 2.0)])
    with pytest.raises(ValueError):
        fp8bs.clip_grad_norm([torch.ones(4, 6, device=DEV).t()], 1.0)
    with pytest.raises(ValueError):
        fp8bs.clip_grad_norm([g], 1.0, out=[g[:50]])
