"""A mixture-of-experts layer for a few tokens against float64 on the dequantized weights.

Tolerance.  u = 2^-24.  A product's sum has exact products and at most d additions in a row: 128 within a K-block
(the matrix instruction's own order is not stated), one fused multiply-add per K-block and the joining of at most four
parts: off by (K + 8) u of sum |w x|, bounded here by n u with n = K + 8 of the larger K.  To first order h moves y
by |slope u| dg + |silu| du; y adds 8 u and its two parts 2^-17; the second product (I + 8) u of its magnitudes, the
weighted sum (top + 2) u, then bf16's half step.  So |out - ref| <= c size + 2^-8 (|ref| + c size) with
c = (H + I + top + 24) u + 2^-17, size as oracle.moe_layer gives it; the second order is below a factor 1.01."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def normal(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(DEV)


def layer(seed, E, H, inner):
    q1, s1 = fp8bs.quantize_b128(normal(seed, E, 2 * inner, H, std=1.5 / H ** 0.5))
    q2, s2 = fp8bs.quantize_b128(normal(seed + 1, E, H, inner, std=1.0 / inner ** 0.5))
    return q1, s1, q2, s2


def dequantized(q, s):
    return np.stack([oracle.dequantize_g128(a, b, 128) for a, b in zip(q.cpu().numpy(), s.cpu().numpy())])


def choices(seed, T, k, E, spread=0.0, repeat=False):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) + spread * torch.randn(E, generator=g)
    if repeat:
        ids = torch.multinomial(torch.softmax(logits, 1), k, replacement=True, generator=g)
    else:
        ids = logits.topk(k, 1).indices
    w = torch.rand(T, k, generator=g)
    return ids.to(torch.int32).to(DEV), (w / w.sum(1, keepdim=True)).to(DEV)


def check(out, x, ids, weights, weights_of, residual=None):
    q1, s1, q2, s2 = weights_of
    H, inner, top = x.shape[1], q2.shape[2], ids.shape[1]
    ref, size = oracle.moe_layer(x.cpu().double().numpy(), ids.cpu().numpy(), weights.cpu().double().numpy(),
                                 dequantized(q1, s1), dequantized(q2, s2))
    off = 1.01 * ((H + inner + top + 24) * U + 2.0 ** -17) * size
    if residual is not None:
        ref = ref + residual.cpu().double().numpy()
        off = off + U * (np.abs(ref) + off)
    err = np.abs(out.cpu().double().numpy() - ref)
    assert (err <= off + 2.0 ** -8 * (np.abs(ref) + off) + 2.0 ** -134).all()


CASES = [(1, 1, 1, 16, 16), (1, 2, 4, 48, 80), (3, 2, 4, 144, 272), (5, 1, 7, 1040, 528), (17, 2, 3, 272, 144),
         (1, 8, 64, 512, 640), (33, 4, 8, 128, 256), (64, 8, 16, 256, 128), (61, 8, 12, 400, 1168), (2, 6, 300, 64, 48),
         (64, 2, 2, 128, 2576), (100, 5, 9, 64, 64), (512, 1, 3, 32, 16), (1, 512, 5, 64, 32), (256, 2, 1024, 16, 16),
         (25, 2, 8, 80, 4112), (61, 2, 8, 8272, 48), (40, 3, 8, 144, 4176)]


@pytest.mark.parametrize("T,k,E,H,inner", CASES)
def test_layer(T, k, E, H, inner):
    say(f"moe {T} {k} {E} {H} {inner}")
    w = layer(T + E, E, H, inner)
    x = normal(7, T, H)
    ids, weights = choices(8, T, k, E, repeat=k > E)
    out = fp8bs.moe_decode_b128(x, ids, weights, *w)
    check(out, x, ids, weights, w)
    res = normal(9, T, H)
    added = fp8bs.moe_decode_b128(x, ids, weights, *w, residual=res)
    check(added, x, ids, weights, w, res)
    here = res.clone()
    assert fp8bs.moe_decode_b128(x, ids, weights, *w, residual=here, out=here) is here
    assert torch.equal(here.view(torch.int16), added.view(torch.int16))
    again = fp8bs.moe_decode_b128(x, ids, weights, *w)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_choices_of_every_kind():
    """Ids outside the experts (held elsewhere, padding), the largest and smallest numbers, a token without any
    expert, an expert named several times by one token, all tokens on one expert."""
    T, k, E, H, inner = 40, 4, 6, 144, 272
    w = layer(3, E, H, inner)
    x = normal(4, T, H)
    ids, weights = choices(5, T, k, E)
    ids[3] = -1
    ids[4, 1:] = E
    ids[5] = torch.tensor([2, 2, 2, 2])
    ids[6] = torch.tensor([2, -7, 2, 2 ** 31 - 1])
    ids[7, 0] = -2 ** 31
    weights[3] = float("nan")  # not used
    say("choices")
    out = fp8bs.moe_decode_b128(x, ids, weights, *w)
    weights[3] = 0.0
    check(out, x, ids, weights, w)
    assert (out[3].view(torch.int16) == 0).all()
    res = normal(6, T, H)
    added = fp8bs.moe_decode_b128(x, ids, weights, *w, residual=res)
    assert torch.equal(added[3].view(torch.int16), res[3].view(torch.int16))
    ids[:] = 5
    check(fp8bs.moe_decode_b128(x, ids, weights, *w), x, ids, weights, w)
    ids[:] = -1
    assert (fp8bs.moe_decode_b128(x, ids, weights, *w) == 0).all()


@pytest.mark.parametrize("E,k", [(8, 2), (200, 3)])
def test_tokens_do_not_depend_on_the_batch(E, k):
    T, H, inner = 50, 528, 1040
    w = layer(13, E, H, inner)
    x, res = normal(14, T, H), normal(15, T, H)
    ids, weights = choices(16, T, k, E, spread=1.0)
    say(f"moe invariance {E}")
    full = fp8bs.moe_decode_b128(x, ids, weights, *w, residual=res)
    for a, b in ((0, 1), (49, 50), (7, 30), (20, 40)):
        part = fp8bs.moe_decode_b128(x[a:b], ids[a:b], weights[a:b], *w, residual=res[a:b])
        assert torch.equal(part.view(torch.int16), full[a:b].view(torch.int16)), (a, b)
    order = torch.randperm(T).to(DEV)
    mixed = fp8bs.moe_decode_b128(x[order], ids[order], weights[order], *w, residual=res[order])
    assert torch.equal(mixed.view(torch.int16), full[order].view(torch.int16))


@pytest.mark.parametrize("T,k,E,H,inner", [(25, 2, 8, 80, 4112), (61, 2, 8, 8272, 48)])
def test_a_token_alone_where_tiles_are_large(T, k, E, H, inner):
    say(f"moe invariance {T} {H} {inner}")
    w = layer(31, E, H, inner)
    x = normal(32, T, H)
    ids, weights = choices(33, T, k, E)
    out = fp8bs.moe_decode_b128(x, ids, weights, *w)
    for t in (0, 7, T - 1):
        at = slice(t, t + 1)
        one = fp8bs.moe_decode_b128(x[at], ids[at], weights[at], *w)
        assert torch.equal(one.view(torch.int16), out[at].view(torch.int16)), t


def test_not_finite_reaches_its_token_only():
    T, k, E, H, inner = 20, 2, 3, 144, 80
    q1, s1, q2, s2 = layer(23, E, H, inner)
    x = normal(24, T, H)
    ids, weights = choices(25, T, k, E)
    say("not finite")
    good = fp8bs.moe_decode_b128(x, ids, weights, q1, s1, q2, s2)
    x[4, 100] = float("nan")
    x[9, 0] = float("inf")
    weights[11, 1] = float("inf")
    out = fp8bs.moe_decode_b128(x, ids, weights, q1, s1, q2, s2)
    keep = [t for t in range(T) if t not in (4, 9, 11)]
    assert torch.equal(out[keep], good[keep])
    assert torch.isnan(out[4]).all() and not torch.isfinite(out[9].float()).any()
    assert not torch.isfinite(out[11].float()).any()
    x[4, 100], x[9, 0], weights[11, 1] = 0.0, 0.0, 0.0
    q2[1, 33, 5] = 0x7F  # a NaN weight: that column of the tokens that take expert 1
    out = fp8bs.moe_decode_b128(x, ids, weights, q1, s1, q2, s2)
    takes = (ids == 1).any(1)
    assert torch.isnan(out[takes][:, 33]).all() and int(torch.isnan(out).sum()) == int(takes.sum())


def test_refusals():
    say("refusals")
    w = layer(33, 2, 64, 32)
    x = normal(1, 3, 64)
    ids, weights = choices(2, 3, 2, 2)
    q1, s1, q2, s2 = w
    for bad in ((x[:2], ids, weights, *w), (x, ids[:, :1], weights, *w), (x, ids, weights[:2], *w),
                (x, ids, weights, q1[:, :62], s1, q2, s2), (x, ids, weights, q1, s1[:, :0], q2, s2),
                (x, ids, weights, q1, s1, q2[:1], s2), (x, ids, weights, q1, s1, q2, s2[:1])):
        with pytest.raises(ValueError):
            fp8bs.moe_decode_b128(*bad)
    with pytest.raises(TypeError):
        fp8bs.moe_decode_b128(x, ids.long(), weights, *w)
    with pytest.raises(TypeError):
        fp8bs.moe_decode_b128(x, ids, weights.to(torch.bfloat16), *w)
    many = torch.zeros(300, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.moe_decode_b128(normal(3, 300, 64), many, torch.zeros(300, 2, device=DEV), *w)
    assert fp8bs.moe_decode_b128(x[:0], ids[:0], weights[:0], *w).shape == (0, 64)


def test_graph_follows_the_choices_and_second_stream():
    T, k, E, H, inner = 9, 3, 20, 272, 400
    w = layer(43, E, H, inner)
    x = normal(44, T, H)
    ids, weights = choices(45, T, k, E)
    say("graph")
    fp8bs.moe_decode_b128(x, ids, weights, *w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8bs.moe_decode_b128(x, ids, weights, *w)
    for seed in (50, 51, 52, 53):
        x.copy_(normal(seed, T, H))
        new, given = choices(seed + 10, T, k, E)
        if seed == 52:
            new[2:] = -1
        ids.copy_(new)
        weights.copy_(given)
        graph.replay()
        torch.cuda.synchronize()
        kept = out.clone()
        want = fp8bs.moe_decode_b128(x, ids, weights, *w)
        assert torch.equal(kept.view(torch.int16), want.view(torch.int16)), seed
        check(kept, x, ids, weights, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = fp8bs.moe_decode_b128(x, ids, weights, *w)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(there.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("k,E,H,inner", [(1, 8, 144, 272), (1, 1, 5152, 16), (2, 8, 5136, 528), (2, 3, 48, 4112),
                                         (3, 64, 4112, 144), (3, 5, 8208, 16), (4, 16, 4096, 1040), (4, 9, 5136, 80),
                                         (4, 9, 4080, 80), (5, 9, 4112, 272)])
def test_one_token_of_few_choices(k, E, H, inner):
    """A token alone (its choices' sums joined in the second kernel, where there are few): in its bound, and the bits
    that it has in a batch; skipped and repeated choices, weights that are not used, the residual in place."""
    say(f"moe one token {k} {E} {H} {inner}")
    w = layer(51, E, H, inner)
    x, res = normal(52, 2, H), normal(53, 2, H)
    ids, weights = choices(54, 2, k, E)
    for kind in ("all", "skipped", "repeated", "none"):
        if kind == "skipped":
            ids[0, k - 1] = -1 if k < 3 else E
            weights[0, k - 1] = float("nan")  # not used
        elif kind == "repeated":
            ids[0] = E - 1
            weights[0] = torch.arange(1, k + 1, device=DEV) * 0.25
        elif kind == "none":
            ids[0] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31, -7][:k])
        for residual in (None, res):
            one = residual[:1].clone() if residual is not None else None
            both = fp8bs.moe_decode_b128(x, ids, weights, *w, residual=residual)
            out = fp8bs.moe_decode_b128(x[:1], ids[:1], weights[:1], *w, residual=one, out=one)
            assert torch.equal(out.view(torch.int16), both[:1].view(torch.int16)), kind
            used = torch.where((ids[:1] >= 0) & (ids[:1] < E), weights[:1], torch.zeros_like(weights[:1]))
            check(out, x[:1], ids[:1], used, w, None if residual is None else residual[:1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8bs.moe_decode_b128(x[:1], ids[:1], weights[:1], *w)
    for seed in (55, 56, 57):
        new, given = choices(seed, 2, k, E)
        ids.copy_(new)
        weights.copy_(given)
        graph.replay()
        torch.cuda.synchronize()
        want = fp8bs.moe_decode_b128(x, ids, weights, *w)[:1]
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), seed
