"""The operators between the products run together, as a program runs them: a feed-forward block's training step
(layer norm, product with gelu, product with residual, their backward passes, weight gradients, clipping), and a
decode step (layer norm, experts for few tokens, the residual stream).  Each step is held to its own bound against
float64 on what the step before it left; captured and on another stream the run gives the same bits."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

import test_gpu_clip as clip
import test_gpu_epilogue as epilogue
import test_gpu_layernorm as norm
import test_gpu_moe as moe
import test_gpu_g128_training as training
from gpu_util import DEV, i32_dev, say

pytestmark = pytest.mark.gpu
EPS = 1e-5


class Block:
    """A pre-norm feed-forward block, M rows of d columns, f columns inside."""

    def __init__(self, M, d, f):
        self.x, self.stream = norm.normal(1, M, d), norm.normal(2, M, d, shift=0.25)
        self.dout = norm.normal(3, M, d, std=0.01)
        self.gamma, self.beta = norm.normal(4, d, std=0.1, shift=1.0), norm.normal(5, d, std=0.1)
        self.b1, self.b2 = norm.normal(6, f, std=0.1), norm.normal(7, d, std=0.1)
        self.w1 = fp8bs.quantize_b128(norm.normal(8, f, d, std=d ** -0.5), transposed=True)
        self.w2 = fp8bs.quantize_b128(norm.normal(9, d, f, std=f ** -0.5), transposed=True)
        self.rows = i32_dev([0, M])
        self.h = torch.empty_like(self.x)

    def step(self):
        s = {"h": self.h}
        s["qy"], s["sy"], s["y"], s["mean"], s["rstd"] = fp8bs.layernorm_quantize_tg128(
            self.x, self.gamma, self.beta, EPS, residual=self.stream, h=self.h, want_y=True, want_stats=True)
        s["a"], s["pre"] = fp8bs.gemm_tg128_nt_epilogue(s["qy"], s["sy"], *self.w1[:2], bias=self.b1,
                                                        activation="gelu", want_pre=True)
        s["qa"], s["sa"] = fp8bs.quantize_tg128(s["a"])
        s["out"] = fp8bs.gemm_tg128_nt_epilogue(s["qa"], s["sa"], *self.w2[:2], bias=self.b2, residual=self.h)
        _, s["qd"], s["sd"], s["db2"] = fp8bs.epilogue_backward_quantize_tg128(self.dout, None)
        s["da"] = fp8bs.gemm_tg128_nt(s["qd"], s["sd"], *self.w2[2:])
        s["dz"], s["qz"], s["sz"], s["db1"] = fp8bs.epilogue_backward_quantize_tg128(s["da"], s["pre"], "gelu")
        s["dy"] = fp8bs.gemm_tg128_nt(s["qz"], s["sz"], *self.w1[2:])
        s["dx"], s["dgamma"], s["dbeta"] = fp8bs.layernorm_backward(s["dy"], self.h, self.gamma, s["mean"], s["rstd"],
                                                                    dresidual=self.dout)
        s["dw2"] = fp8bs.grouped_wgrad(self.dout, s["a"], self.rows)
        s["dw1"] = fp8bs.grouped_wgrad(s["dz"], s["y"], self.rows)
        grads = [s[n] for n in ("dw1", "dw2", "db1", "db2", "dgamma", "dbeta")]
        s["clipped"] = [torch.empty_like(g) for g in grads]
        s["norm"] = fp8bs.clip_grad_norm(grads, 0.05, out=s["clipped"])
        return s


def flat(s):
    return [t for v in s.values() for t in (v if isinstance(v, list) else [v])]


def same(a, b):
    return all(torch.equal(x.reshape(-1).view(torch.uint8), y.reshape(-1).view(torch.uint8))
               for x, y in zip(flat(a), flat(b)))


def host(*ts):
    return [t.cpu().numpy() for t in ts]


@pytest.mark.parametrize("M,d,f", [(77, 272, 528), (130, 512, 1040)])
def test_training_step_of_a_block(M, d, f):
    say(f"block {M} {d} {f}")
    b = Block(M, d, f)
    s = b.step()
    torch.cuda.synchronize()
    _, _, ref, off = norm.reference(s["h"], b.gamma, b.beta, EPS)
    norm.check_codes(s["qy"], s["sy"], ref, off)
    every = (np.arange(M), np.arange(f))
    epilogue.check(s["a"], s["pre"], host(s["qy"], s["sy"], *b.w1[:2]), b.b1, "gelu", None, *every)
    epilogue.check(s["out"], None, host(s["qa"], s["sa"], *b.w2[:2]), b.b2, "none", s["h"], np.arange(M), np.arange(d))
    epilogue.check_backward(b.dout, None, "none", (b.dout, s["qd"], s["sd"], s["db2"]))
    epilogue.check_backward(s["da"], s["pre"], "gelu", (s["dz"], s["qz"], s["sz"], s["db1"]))
    for got, q, sc, w in (("da", "qd", "sd", b.w2), ("dy", "qz", "sz", b.w1)):
        ref, bound = oracle.gemm_g128_bound(*host(s[q], s[sc], *w[2:]))
        assert (np.abs(norm.np64(s[got]) - ref) <= bound).all(), got
    norm.check_backward(s["dy"], s["h"], b.gamma, s["mean"], s["rstd"], b.dout, (s["dx"], s["dgamma"], s["dbeta"]))
    training.check_wgrad(s["dw2"], b.dout, s["a"], [0, M])
    training.check_wgrad(s["dw1"], s["dz"], s["y"], [0, M])
    grads = [s[n] for n in ("dw1", "dw2", "db1", "db2", "dgamma", "dbeta")]
    clip.check_norm(s["norm"], grads)
    clip.check_clipped(s["clipped"], grads, 0.05)

    say("captured, with new inputs")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = b.step()
    for seed in (30, 31, 32):
        b.x.copy_(norm.normal(seed, M, d))
        b.dout.copy_(norm.normal(seed + 10, M, d, std=0.01))
        graph.replay()
        torch.cuda.synchronize()
        kept = {k: [t.clone() for t in v] if isinstance(v, list) else v.clone() for k, v in held.items()}
        want = b.step()
        assert same(kept, want), seed
    say("another stream")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = b.step()
    torch.cuda.current_stream().wait_stream(side)
    assert same(there, want)


def test_two_blocks_on_two_streams_at_once():
    """Calls that overlap in time have workspaces of their own."""
    blocks = [Block(130, 512, 1040), Block(77, 272, 528)]
    want = [b.step() for b in blocks]
    torch.cuda.synchronize()
    say("two streams at once")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for b, st in zip(blocks, streams):
            with torch.cuda.stream(st):
                got.append([b.step() for _ in range(4)][-1])
        torch.cuda.synchronize()
        for a, w in zip(got, want):
            assert same(a, w)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_decode_step(T):
    E, k, H, inner = 12, 3, 272, 400
    w = moe.layer(60, E, H, inner)
    x, stream = norm.normal(61, T, H), norm.normal(62, T, H)
    gamma, beta = norm.normal(63, H, std=0.1, shift=1.0), norm.normal(64, H, std=0.1)
    ids, weights = moe.choices(65, T, k, E)
    h = torch.empty_like(x)

    def step():
        y = fp8bs.layernorm(x, gamma, beta, EPS, residual=stream, h=h)
        return y, fp8bs.moe_decode_b128(y, ids, weights, *w, residual=h)

    say(f"decode step {T}")
    y, out = step()
    _, _, ref, off = norm.reference(h, gamma, beta, EPS)
    assert (np.abs(norm.np64(y) - ref) <= off + 2.0 ** -8 * (np.abs(ref) + off) + 2.0 ** -134).all()
    moe.check(out, y, ids, weights, w, h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (70, 71, 72):
        x.copy_(norm.normal(seed, T, H))
        new, given = moe.choices(seed, T, k, E)
        ids.copy_(new)
        weights.copy_(given)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in held]
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(kept, step()))


def test_the_experts_layer_is_what_its_parts_compute():
    """moe_decode_b128 against the same layer by products of quantized activations.  Between them lie the codes of x
    and of y: half an E4M3 step each, 2^-4 of a value (beside 2^-19 of its group's largest), which moves y and then
    out by at most 2^-4 of the magnitudes; and bf16 roundings of h and of the parts, 2^-8 each, within the rest."""
    T, k, E, H, inner = 24, 2, 6, 512, 640
    q1, s1, q2, s2 = moe.layer(80, E, H, inner)
    x = norm.normal(81, T, H)
    ids, weights = moe.choices(82, T, k, E)
    say("parts")
    out = fp8bs.moe_decode_b128(x, ids, weights, q1, s1, q2, s2)
    order = ids.flatten().long().argsort(stable=True)
    offsets = torch.cat([torch.zeros(1, device=DEV), torch.bincount(ids.flatten().long(), minlength=E).cumsum(0)])
    offsets = offsets.to(torch.int32)
    rows = x[order // k].contiguous()
    gu = fp8bs.grouped_gemm_tg128_nt(*fp8bs.quantize_tg128(rows), q1, s1, offsets)
    part = fp8bs.grouped_gemm_tg128_nt(*fp8bs.swiglu_quantize_tg128(gu), q2, s2, offsets)
    slots = torch.empty(T * k, H, device=DEV)
    slots[order] = part.float()
    want = (slots.view(T, k, H) * weights[:, :, None]).sum(1)
    _, size = oracle.moe_layer(x.cpu().double().numpy(), ids.cpu().numpy(), weights.cpu().double().numpy(),
                               moe.dequantized(q1, s1), moe.dequantized(q2, s2))
    assert (np.abs(norm.np64(out) - norm.np64(want)) <= (2 * 2.0 ** -4 + 2.0 ** -6) * size).all()
