"""Norm and clipping of lists so long that their partial sums are joined by a launch of their own (more than 4096 of
them; here each tensor with values has one, seven in eight), up to the most tensors of a call.

Values are small whole numbers, so every square and sum is exact in 64 bits; a norm is off by its square root and its
rounding to fp32 (2^-24 and 2^-53 of it)."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def lists(n, seed):
    """n tensors of 0 to 7 values, fp32 and bf16 in turn, slices of two buffers; what lies between them is large."""
    g = torch.Generator().manual_seed(seed)
    counts = torch.randint(0, 8, (n,), generator=g).tolist()
    whole = [torch.full((8 * n,), 1000.0, dtype=t, device=DEV) for t in (torch.float32, torch.bfloat16)]
    values = torch.randint(-9, 10, (8 * n,), generator=g)
    held = torch.zeros(8 * n, dtype=torch.bool)
    for i, c in enumerate(counts):
        held[8 * i:8 * i + c] = True
    kind = torch.arange(8 * n) // 8 % 2
    for t, w in enumerate(whole):
        w.copy_(torch.where(held & (kind == t), values, torch.full_like(values, 1000)).to(w.dtype))
    grads = [whole[i % 2][8 * i:8 * i + c] for i, c in enumerate(counts)]
    return whole, grads, held, kind, values


def norm_of(held, values):
    return float(np.sqrt((values[held].double() ** 2).sum().numpy()))


@pytest.mark.parametrize("n", [4097, 6001, 65536])
def test_long_lists(n):
    whole, grads, held, kind, values = lists(n, n)
    want = norm_of(held, values)
    say(f"clip {n} tensors")
    norm = fp8bs.grad_norm(grads)
    assert abs(float(norm) - want) <= (2.0 ** -24 + 2.0 ** -50) * want
    both = fp8bs.clip_grad_norm(grads, want / 4, eps=0.0)
    assert torch.equal(both, norm)
    # a factor of a quarter or its neighbour: the norm's own last bit of 64
    for t, w in enumerate(whole):
        mine = held & (kind == t)
        got = w.cpu().double()
        assert (got[~mine] == 1000.0).all()
        off = (got[mine] - values[mine] / 4.0).abs()
        assert (off <= (2 * 2.0 ** -24 + (2.0 ** -8 if t else 0.0)) * values[mine].abs() / 4.0).all()
    again = fp8bs.clip_grad_norm(grads, 1e30)
    assert abs(float(again) - want / 4) <= 2.0 ** -7 * want


def test_a_long_list_in_a_graph():
    n = 5000
    whole, grads, held, kind, values = lists(n, 1)
    out = [torch.empty_like(g) for g in grads]
    say("long list in a graph")
    fp8bs.clip_grad_norm(grads, 1.0, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = fp8bs.clip_grad_norm(grads, 1.0, out=out)
    for seed in (2, 3, 4):
        values = torch.randint(-9, 10, (8 * n,), generator=torch.Generator().manual_seed(seed))
        for t, w in enumerate(whole):
            w.copy_(torch.where(held & (kind == t), values, torch.full_like(values, 1000)).to(w.dtype))
        graph.replay()
        torch.cuda.synchronize()
        kept, kept_norm = [o.clone() for o in out], norm.clone()
        want = norm_of(held, values)
        assert abs(float(kept_norm) - want) <= (2.0 ** -24 + 2.0 ** -50) * want
        again = fp8bs.clip_grad_norm(grads, 1.0, out=out)
        assert torch.equal(again, kept_norm) and all(torch.equal(a, b) for a, b in zip(kept, out))


def test_one_more_than_the_most_is_refused():
    g = torch.zeros(4, device=DEV)
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.grad_norm([g] * 65537)
