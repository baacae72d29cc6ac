"""Products with bias, activation and residual in their epilogue, and the epilogue's backward pass.

Tolerances.  u = 2^-24 is fp32's half step, 2^-8 bf16's.  The product itself is within the bound of
oracle.gemm_g128_bound, B before it is rounded; z = product + bias adds u|z|.  No activation's slope exceeds 1.13,
so act(z) moves by 1.13 (B + u|z|); the header states 2^-15 of the result and 2^-118 for the activation itself; the
residual's addition adds u and the result's rounding 2^-8."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, f32_dev, say, u8_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ACTS = list(fp8bs.ACTIVATIONS)


def np64(t):
    return t.cpu().double().numpy()


def normal(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(DEV)


def operands(seed, M, N, K):
    rng = np.random.default_rng(seed)
    nk, nn = -(-K // 128), -(-N // 128)

    def codes(*shape):
        return oracle.encode_e4m3(np.clip(rng.normal(size=shape) * 140, -448, 448).astype(np.float32))
    return (codes(M, K), np.exp(rng.normal(size=(M, nk))).astype(np.float32) * np.float32(0.01), codes(N, K),
            np.exp(rng.normal(size=(nn, nk))).astype(np.float32) * np.float32(1e-3))


def dev(ops):
    return u8_dev(ops[0]), f32_dev(ops[1]), u8_dev(ops[2]), f32_dev(ops[3])


def check(out, pre, ops, bias, act, res, rows, cols):
    ref, bound = oracle.gemm_g128_bound(ops[0][rows], ops[1][rows], ops[2], ops[3])
    ref, bound = ref[:, cols], bound[:, cols]
    B = bound - 2.0 ** -8 * np.abs(ref)
    z = ref + (0.0 if bias is None else np64(bias)[cols][None, :])
    B = B + U * (np.abs(z) + B)
    if pre is not None:
        assert (np.abs(np64(pre)[rows][:, cols] - z) <= B + 2.0 ** -8 * (np.abs(z) + B) + 2.0 ** -134).all()
    a, _, _ = oracle.activation_parts(z, act)
    off = 1.13 * B + (0.0 if act in ("none", "relu") else 2.0 ** -15 * (np.abs(a) + 1.13 * B) + 2.0 ** -118)
    want = a + (0.0 if res is None else np64(res)[rows][:, cols])
    off = off + U * (np.abs(want) + off)
    err = np.abs(np64(out)[rows][:, cols] - want)
    assert (err <= off + 2.0 ** -8 * (np.abs(want) + off) + 2.0 ** -134).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (3, 272, 144), (17, 16, 528), (64, 80, 272), (130, 272, 400)])
@pytest.mark.parametrize("with_bias,with_res,with_pre",
                         [(True, True, True), (False, False, False), (True, False, True)])
def test_within_the_bound(M, N, K, act, with_bias, with_res, with_pre):
    say(f"epilogue {M}x{N}x{K} {act} {with_bias} {with_res}")
    ops = operands(M * 7 + N + K, M, N, K)
    bias = normal(1, N) if with_bias else None
    res = normal(2, M, N) if with_res else None
    got = fp8bs.gemm_tg128_nt_epilogue(*dev(ops), bias=bias, activation=act, residual=res, want_pre=with_pre)
    out, pre = got if with_pre else (got, None)
    check(out, pre, ops, bias, act, res, np.arange(M), np.arange(N))
    if act == "none" and not with_bias and not with_res:
        plain = fp8bs.gemm_tg128_nt(*dev(ops))
        assert torch.equal(out.view(torch.int16), plain.view(torch.int16))


# One size for each tile that the dispatch can take, ragged both ways, with whole lines of C and without.
SIZES = [(9, 1040), (16, 4096), (20, 2064), (40, 1040), (13, 8208), (30, 10256), (50, 16528), (100, 4112), (500, 3600),
         (1000, 2320), (1000, 4624), (1000, 9232), (400, 7184), (1700, 4112), (3500, 4112),
         (1000, 2368), (1000, 9280), (400, 7232), (1700, 4160), (3500, 4160)]


@pytest.mark.parametrize("M,N", SIZES)
def test_every_tile(M, N):
    """Every tile gives a row the bits that the row has alone; the values are checked at sampled rows."""
    K = 400
    ops = operands(M + N, M, N, K)
    a, sa, bt, sbt = dev(ops)
    bias, res = normal(3, N), normal(4, M, N)
    for act in ("gelu", "silu", "relu"):
        say(f"epilogue tile {M}x{N} {act}")
        out, pre = fp8bs.gemm_tg128_nt_epilogue(a, sa, bt, sbt, bias=bias, activation=act, residual=res, want_pre=True)
        rows = sorted({0, 1, M // 2, M - 1})
        for r in rows:
            one = slice(r, r + 1)
            o, p = fp8bs.gemm_tg128_nt_epilogue(a[one], sa[one], bt, sbt, bias=bias, activation=act, residual=res[one],
                                                want_pre=True)
            assert torch.equal(o[0].view(torch.int16), out[r].view(torch.int16)), (act, r)
            assert torch.equal(p[0].view(torch.int16), pre[r].view(torch.int16)), (act, r)
        # in place on the residual, without pre
        here = res.clone()
        assert fp8bs.gemm_tg128_nt_epilogue(a, sa, bt, sbt, bias=bias, activation=act, residual=here, out=here) is here
        assert torch.equal(here.view(torch.int16), out.view(torch.int16))
        # the epilogue is what it is of the product: pre is the rounded sum, and no residual is no addition
        bare = fp8bs.gemm_tg128_nt_epilogue(a, sa, bt, sbt, bias=bias)
        assert torch.equal(bare.view(torch.int16), pre.view(torch.int16))
        rows = np.unique(np.linspace(0, M - 1, 10).astype(int))
        if act == "gelu":
            at = torch.from_numpy(rows).to(DEV)
            cols = np.unique(np.r_[0:8, N // 2:N // 2 + 8, N - 8:N])
            check(out[at], pre[at], (ops[0][rows], ops[1][rows], ops[2], ops[3]), bias, act, res[at],
                  np.arange(len(rows)), cols)


def every_bf16():
    """All finite bf16 values."""
    bits = torch.arange(65536, dtype=torch.int32)
    keep = (bits & 0x7F80) != 0x7F80
    return bits[keep].to(torch.int16).view(torch.bfloat16)


@pytest.mark.parametrize("act", ACTS)
def test_activation_of_every_bf16_value(act):
    """K = 0: the result is act(bias) + residual."""
    z = every_bf16()
    N = z.numel()
    say(f"every bf16 {act}")
    empty = (torch.zeros(3, 0, dtype=torch.uint8, device=DEV), torch.zeros(3, 0, device=DEV),
             torch.zeros(N, 0, dtype=torch.uint8, device=DEV), torch.zeros(-(-N // 128), 0, device=DEV))
    out, pre = fp8bs.gemm_tg128_nt_epilogue(*empty, bias=z.to(DEV), activation=act, want_pre=True)
    assert torch.equal(pre[2].cpu().float(), z.float())
    want = oracle.activation_parts(z.double().numpy(), act)[0]
    # z + 0 is exact, the activation as the header has it, then the rounding
    tol = (0.0 if act in ("none", "relu") else 2.0 ** -15 * np.abs(want) + 2.0 ** -118)
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134
    got = np64(out)
    assert (np.abs(got - want) <= tol).all(), act
    assert not ((want == 0) & np.signbit(got)).any()  # (a value below 2^-134 rounds to a zero of its sign)
    res = normal(5, 3, N)
    out = fp8bs.gemm_tg128_nt_epilogue(*empty, bias=z.to(DEV), activation=act, residual=res)
    want = want + np64(res)
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert (np.abs(np64(out) - want) <= tol).all(), act


def test_not_finite_stays_in_its_column():
    say("not finite")
    ops = dev(operands(5, 70, 272, 144))
    bias = normal(6, 272)
    bias[100], bias[200] = float("nan"), float("inf")
    for act in ACTS:
        out, pre = fp8bs.gemm_tg128_nt_epilogue(*ops, bias=bias, activation=act, want_pre=True)
        keep = [n for n in range(272) if n not in (100, 200)]
        assert torch.isnan(out[:, 100]).all() and (out[:, 200] == float("inf")).all(), act
        assert torch.isfinite(out[:, keep].float()).all() and torch.isnan(pre[:, 100]).all()


def test_minus_infinity():
    """relu and gelu have their limit 0, the products z sigma(z) a NaN; what stands beside is left alone."""
    say("-inf")
    ops = dev(operands(9, 21, 272, 144))
    bias = normal(7, 272)
    bias[33] = float("-inf")
    for act in ACTS:
        out, pre = fp8bs.gemm_tg128_nt_epilogue(*ops, bias=bias, activation=act, want_pre=True)
        assert (pre[:, 33] == float("-inf")).all(), act
        if act == "none":
            assert (out[:, 33] == float("-inf")).all()
        elif act in ("relu", "gelu"):
            assert (out[:, 33].view(torch.int16) == 0).all(), act
        else:
            assert torch.isnan(out[:, 33]).all(), act
        assert torch.isfinite(out[:, [n for n in range(272) if n != 33]].float()).all(), act


def test_refusals_and_empty():
    say("refusals")
    a, sa, bt, sbt = dev(operands(7, 5, 32, 64))
    for bad in ({"bias": normal(1, 16)}, {"residual": normal(1, 5, 16)}, {"activation": "tanh"},
                {"residual": normal(1, 32, 5).t()}, {"pre": normal(1, 4, 32)}):
        with pytest.raises(ValueError):
            fp8bs.gemm_tg128_nt_epilogue(a, sa, bt, sbt, **bad)
    with pytest.raises(TypeError):
        fp8bs.gemm_tg128_nt_epilogue(a, sa, bt, sbt, bias=torch.zeros(32, device=DEV))
    assert fp8bs.gemm_tg128_nt_epilogue(a[:0], sa[:0], bt, sbt, activation="gelu").shape == (0, 32)
    d = normal(2, 5, 32)
    with pytest.raises(ValueError):
        fp8bs.epilogue_backward_quantize_tg128(d, None, "gelu")
    with pytest.raises(ValueError):
        fp8bs.epilogue_backward_quantize_tg128(d, d[:4], "gelu")
    with pytest.raises(ValueError):
        fp8bs.epilogue_backward_quantize_tg128(d, d, "gelu", accumulate=True)
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.epilogue_backward_quantize_tg128(normal(3, 5, 24), None, "none")


# ---- backward ----------------------------------------------------------------------------
@pytest.mark.parametrize("act", ACTS)
def test_slope_of_every_bf16_value(act):
    """One value to a row of 128: the scale times 448 is |act'| with fp32's digits.  16 u of the magnitudes that it
    is made of (each part is within 8 ulp by the errors of its steps), and the scale's own rounding."""
    z = every_bf16()
    n = z.numel() // 16 * 16
    z = z[:n]
    pre = torch.zeros(n, 128, dtype=torch.bfloat16)
    pre[:, 77] = z
    dout = torch.zeros(n, 128, dtype=torch.bfloat16)
    dout[:, 77] = 1.0
    say(f"slopes {act}")
    dz, q, s, dbias = fp8bs.epilogue_backward_quantize_tg128(dout.to(DEV), pre.to(DEV), act)
    _, slope, size = oracle.activation_parts(z.double().numpy(), act)
    got = np64(s)[:, 0] * 448.0 * np.where(np.signbit(np64(dz)[:, 77]), -1.0, 1.0)
    tol = 16 * U * size + 2 * U * np.abs(slope) + 448 * 2.0 ** -148
    bad = np.abs(got - slope) > tol
    assert not bad.any(), (act, z[torch.from_numpy(bad)][:5], (np.abs(got - slope) / (U * size))[bad].max())
    assert (np.abs(np64(dz)[:, 77] - slope) <= tol + 2.0 ** -8 * (np.abs(slope) + tol) + 2.0 ** -134).all()
    assert (np64(dz)[:, :77] == 0).all() and (np64(dz)[:, 78:] == 0).all()
    total = np.zeros(128)
    total[77] = slope.sum()
    assert (np.abs(np64(dbias) - total) <= (n * U * np.abs(slope).sum() + tol.sum())).all()


def check_backward(dout, pre, act, got, old=None):
    dz, q, s, dbias = got
    rows, n = dout.shape
    _, slope, size = oracle.activation_parts(np64(pre) if pre is not None else np.zeros((rows, n)), act)
    ref = np64(dout) * slope
    off = np.abs(np64(dout)) * 16 * U * size + 2 * U * np.abs(ref) + 2.0 ** -140
    if act == "none":
        off = off * 0
        assert torch.equal(dz.view(torch.int16), dout.view(torch.int16))
    assert (np.abs(np64(dz) - ref) <= off + 2.0 ** -8 * (np.abs(ref) + off) + 2.0 ** -134).all()
    q, s = q.cpu().numpy(), np64(s)
    for b in range(s.shape[1]):
        at = slice(128 * b, min(n, 128 * b + 128))
        amax, slack = np.abs(ref[:, at]).max(1), off[:, at].max(1)
        assert (np.abs(s[:, b] - amax / 448) <= slack / 448 + 2 * U * amax / 448 + 2.0 ** -149).all()
        sc = s[:, b:b + 1]
        t = np.where(sc > 0, ref[:, at] / np.where(sc > 0, sc, 1), 0)
        loose = np.where(sc > 0, off[:, at] / np.where(sc > 0, sc, 1), 0) + 2 * U * np.abs(t)
        half = oracle.e4m3_half_step(np.minimum(np.abs(t) + loose, 448))
        assert (np.abs(oracle.decode_e4m3(q[:, at]) - t) <= half + loose).all()
    want, mag = ref.sum(0), np.abs(ref).sum(0)
    tol = (rows + 2) * U * mag + off.sum(0)
    if old is not None:
        want = want + np64(old)
        tol = tol + U * (np.abs(want) + tol)
    assert (np.abs(np64(dbias) - want) <= tol).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,n", [(1, 16), (3, 128), (5, 272), (33, 1040), (130, 4096), (7, 8208), (2100, 144),
                                    (9000, 16)])
def test_backward(rows, n, act):
    say(f"epilogue_backward {rows}x{n} {act}")
    dout, pre = normal(1, rows, n, std=0.01), normal(2, rows, n, std=1.7)
    got = fp8bs.epilogue_backward_quantize_tg128(dout, None if act == "none" else pre, act)
    check_backward(dout, pre, act, got)
    again = fp8bs.epilogue_backward_quantize_tg128(dout, pre, act)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, again))
    old = torch.randn(n, device=DEV)
    sums = old.clone()
    more = fp8bs.epilogue_backward_quantize_tg128(dout, pre, act, dbias=sums, accumulate=True)
    assert more[3] is sums
    check_backward(dout, pre, act, more, old)


def test_backward_rows_and_special_values():
    say("special rows")
    rows, n = 40, 528
    dout, pre = normal(1, rows, n), normal(2, rows, n)
    dout[3] = 0
    pre[4] = float("-inf")
    pre[5] = -100.0
    dout[6] = 1e30
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        dz, q, s, dbias = fp8bs.epilogue_backward_quantize_tg128(dout, pre, act)
        assert (dz[3] == 0).all() and (s[3] == 0).all() and (q[3] & 0x7F == 0).all()
        assert (dz[4] == 0).all() and torch.isfinite(dbias).all(), act
        for a, b in ((0, 1), (39, 40), (2, 9)):
            part = fp8bs.epilogue_backward_quantize_tg128(dout[a:b], pre[a:b], act)
            assert torch.equal(part[0].view(torch.int16), dz[a:b].view(torch.int16))
            assert torch.equal(part[1], q[a:b]) and torch.equal(part[2], s[a:b])
        pre[7, 100] = float("nan")
        dz, _, _, dbias = fp8bs.epilogue_backward_quantize_tg128(dout, pre, act)
        assert torch.isnan(dz[7, 100]) and torch.isnan(dbias[100]) and int(torch.isnan(dz).sum()) == 1
        pre[7, 100] = 0.0
    z = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    assert (fp8bs.epilogue_backward_quantize_tg128(z, z, "gelu")[3] == 0).all()


def test_graph_and_second_stream():
    M, N, K = 300, 1040, 528
    a, sa, bt, sbt = dev(operands(1, M, N, K))
    bias, res, dout = normal(2, N), normal(3, M, N), normal(4, M, N)

    def step():
        out, pre = fp8bs.gemm_tg128_nt_epilogue(a, sa, bt, sbt, bias=bias, activation="gelu", residual=res,
                                                want_pre=True)
        return (out, pre) + fp8bs.epilogue_backward_quantize_tg128(dout, pre, "gelu")

    say("graph")
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (20, 21, 22):
        res.copy_(normal(seed, M, N))
        dout.copy_(normal(seed + 10, M, N))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        want = step()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(kept, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(there, want))
