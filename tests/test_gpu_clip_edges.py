"""Norm and clipping of lists beyond 8 MB, whose chunks are larger: the first and last values of tensors that start and
end anywhere, one at a time, and every clipped value, bit for bit; what lies around the tensors is left alone."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# (values, type, first value's place in its buffer); a chunk is 32 KB: 8192 values of 32 bits, 16384 of 16
PARTS = [(8192, F32, 0), (8193, F32, 1), (3 * 8192 - 1, F32, 3), (16384, BF16, 0), (16385, BF16, 7), (40001, BF16, 5),
         (1, BF16, 1), (5, F32, 2), (0, F32, 0), (16384 * 3, BF16, 4), (8192 * 4, F32, 2)]
# what the lists are filled up to: below 192 MB, above it (clipping past the caches), above 512 MB (the norm too)
FILL = [(3_000_017, F32, 1), (60_000_001, F32, 2), (300_000_007, BF16, 3)]


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def buffers(fill, value):
    whole = [torch.full((n + 64,), value, dtype=t, device=DEV) for n, t, _ in PARTS + [fill]]
    return whole, [w[at:at + n] for w, (n, _, at) in zip(whole, PARTS + [fill])]


def edges(n):
    """Places next to a tensor's ends, to its chunks' and to what a thread reads at once."""
    near = {0, 1, 2, 3, 7, 8, n - 1, n - 2, n - 8, n - 9, n // 2}
    for chunk in (8192, 16384):
        for k in (chunk, n // chunk * chunk):
            near |= set(range(k - 9, k + 2))
    return sorted(p for p in near if 0 <= p < n)


@pytest.mark.parametrize("fill", FILL, ids=str)
def test_every_edge_is_in_the_norm(fill):
    whole, grads = buffers(fill, 0.0)
    for w, (n, _, at) in zip(whole, PARTS + [fill]):
        w[:at] = 3.0  # around the tensors: not counted
        w[at + n:] = 5.0
    say(f"edges {fill}")
    assert float(fp8bs.grad_norm(grads)) == 0.0
    for i, g in enumerate(grads):
        for p in edges(g.numel()):
            g[p] = -1.5
            assert float(fp8bs.grad_norm(grads)) == 1.5, (i, p)
            g[p] = 0.0


@pytest.mark.parametrize("fill", FILL, ids=str)
@pytest.mark.parametrize("shift", [0, 1])
def test_every_clipped_value(fill, shift):
    """In place (shift 0), and into tensors that start elsewhere inside 16 bytes."""
    whole, grads = buffers(fill, 9.0)
    gen = torch.Generator(device=DEV).manual_seed(1)
    for g in grads:
        g.copy_(torch.randn(g.numel(), generator=gen, device=DEV))
    norm = torch.tensor(7.3, device=DEV)
    factor = np.float32(min(1.0, 2.1 / (float(norm) + 1e-6)))
    say(f"clip values {fill} {shift}")
    want = [(g.float() * torch.tensor(factor, device=DEV)).to(g.dtype) for g in grads]
    if shift:
        old = [w.clone() for w in whole]
        there = [torch.full((w.numel() + 8,), 9.0, dtype=w.dtype, device=DEV) for w in whole]
        out = [t[at + shift:at + shift + n] for t, (n, _, at) in zip(there, PARTS + [fill])]
        fp8bs.clip_grads(grads, norm, 2.1, out=out)
        assert all(torch.equal(a, b) for a, b in zip(whole, old))
    else:
        there, out = whole, grads
        fp8bs.clip_grads(grads, norm, 2.1)
    for t, o, w, (n, _, at) in zip(there, out, want, PARTS + [fill]):
        assert torch.equal(o, w)
        assert (t[:at + shift] == 9.0).all() and (t[at + shift + n:] == 9.0).all()
