"""The weight gradients of ragged groups, silu(gate) * up with its gradient, and a
run of an expert layer forward and backward."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, i32_dev, say

pytestmark = pytest.mark.gpu


def normal(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(DEV)


def np64(t):
    return t.cpu().double().numpy()


# ---- weight gradients ----------------------------------------------------------------------
def check_wgrad(dw, dy, x, offsets, old=None):
    """|dw - exact| <= (R + 2) 2^-23 sum |dy x| (+ the rounding of the addition to `old`): at most R additions of
    exact products, each off by at most one fp32 step of a partial sum."""
    dy, x, dw = np64(dy), np64(x), np64(dw)
    for g in range(len(offsets) - 1):
        r = slice(offsets[g], offsets[g + 1])
        ref, mag = dy[r].T @ x[r], np.abs(dy[r]).T @ np.abs(x[r])
        tol = (r.stop - r.start + 2) * 2.0 ** -23 * mag + 1e-300
        if old is not None:
            ref = ref + np64(old[g])
            tol = tol + 2.0 ** -23 * np.abs(ref)
        assert (np.abs(dw[g] - ref) <= tol).all(), g


@pytest.mark.parametrize("sizes", [[1], [0], [31, 0, 32, 33], [100, 1, 0, 65], [0, 0, 300]])
@pytest.mark.parametrize("N,K", [(16, 16), (144, 272), (272, 80)])
def test_wgrad(sizes, N, K):
    say(f"wgrad {sizes} {N}x{K}")
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(int)
    M = int(off[-1]) + 3
    dy, x = normal(1, M, N), normal(2, M, K)
    dw = fp8bs.grouped_wgrad(dy, x, i32_dev(off))
    check_wgrad(dw, dy, x, off)
    old = torch.randn(len(sizes), N, K, device=DEV)
    out = old.clone()
    assert fp8bs.grouped_wgrad(dy, x, i32_dev(off), out, accumulate=True) is out
    check_wgrad(out, dy, x, off, old)
    for g, n in enumerate(sizes):
        if n == 0:
            assert (dw[g] == 0).all() and torch.equal(out[g], old[g])


def test_wgrad_large_tiles():
    """Enough tiles for the large form, with ranges inside the rows."""
    off = np.array([3, 203, 203, 500, 640, 641, 900, 933, 1001])
    dy, x = normal(3, 1010, 2064), normal(4, 1010, 2000)
    say("wgrad large")
    check_wgrad(fp8bs.grouped_wgrad(dy, x, i32_dev(off)), dy, x, off)


@pytest.mark.parametrize("G,M,N,K", [(16, 6500, 2064, 2000), (4, 2000, 2048, 2064), (1, 8000, 2048, 2000),
                                     (3, 1500, 2048, 2000), (8, 333, 1040, 528), (1, 5000, 272, 144)])
def test_wgrad_every_tile(G, M, N, K):
    """Sizes that reach every tile, uneven ranges, against fp64 on the GPU; replacing and adding."""
    rng = np.random.default_rng(G * M)
    off = np.sort(rng.integers(0, M + 1, G + 1))
    off[0], off[-1] = 0, M
    dy, x = normal(3, M, N), normal(4, M, K)
    say(f"wgrad {G} {M} {N}x{K}")
    old = torch.randn(G, N, K, device=DEV)
    dw = fp8bs.grouped_wgrad(dy, x, i32_dev(off))
    added = fp8bs.grouped_wgrad(dy, x, i32_dev(off), old.clone(), accumulate=True)
    for g in range(G):
        r = slice(int(off[g]), int(off[g + 1]))
        a, b = dy[r].double(), x[r].double()
        ref, mag = a.t() @ b, a.abs().t() @ b.abs()
        tol = (r.stop - r.start + 2) * 2.0 ** -23 * mag + 1e-300
        assert ((dw[g] - ref).abs() <= tol).all(), g
        # the sum again, added once in fp32
        assert torch.equal(added[g], old[g] + dw[g]), g


def test_wgrad_not_finite_rows_of_other_groups():
    """Rows past a range's end are another range's: an infinity or a NaN there stays there."""
    off = [0, 5, 40]
    dy, x = normal(5, 45, 48), normal(6, 45, 32)
    good = fp8bs.grouped_wgrad(dy, x, i32_dev(off))
    x[7, 3] = float("nan")
    dy[41, 0] = float("inf")          # outside every range
    x[44, 0] = float("inf")
    dw = fp8bs.grouped_wgrad(dy, x, i32_dev(off))
    assert torch.equal(dw[0], good[0])
    assert torch.isnan(dw[1][:, 3]).all()
    keep = [k for k in range(32) if k != 3]
    assert torch.equal(dw[1][:, keep], good[1][:, keep])


def test_wgrad_no_rows_and_bad_tables():
    e = torch.empty(0, 32, dtype=torch.bfloat16, device=DEV)
    out = torch.full((2, 32, 32), 7.0, device=DEV)
    fp8bs.grouped_wgrad(e, e, i32_dev([0, 0, 0]), out, accumulate=True)
    assert (out == 7.0).all()
    fp8bs.grouped_wgrad(e, e, i32_dev([0, 0, 0]), out)
    assert (out == 0.0).all()
    dy, x = normal(7, 20, 32), normal(8, 20, 32)
    check_wgrad(fp8bs.grouped_wgrad(dy, x, i32_dev([-5, 10, 1000])), dy, x, [0, 10, 20])
    assert (fp8bs.grouped_wgrad(dy, x, i32_dev([10, 2, 2])) == 0).all()
    with pytest.raises(ValueError):
        fp8bs.grouped_wgrad(dy, x, i32_dev([0, 20]), accumulate=True)
    with pytest.raises(ValueError):
        fp8bs.grouped_wgrad(dy, x, i32_dev([0]))
    with pytest.raises(ValueError):
        fp8bs.grouped_wgrad(dy, x[:5].clone(), i32_dev([0, 20]))


# ---- silu(gate) * up --------------------------------------------------------------------------
# fp32 steps: t = -g log2(e) in two parts, exp2 (1 ulp) and its correction, 1 + e, the reciprocal with a Newton step,
# at most four products: within 16 half steps (2^-24) of the value, 2^-20.  1 - sigma and 1 + g (1 - sigma) may cancel:
# there the error is 2^-20 of the terms, at most dy u sigma (1 + |g|).
REL = 2.0 ** -20


def grids(seed, rows, d, std):
    return normal(seed, rows, 2 * d, std=std), normal(seed + 1, rows, d)


def check_codes(q, s, exact, tol):
    """Scales within the error of the values they are taken from, values within half a code's step of the exact ones."""
    q, s = q.cpu().numpy(), s.cpu().numpy()
    R, C = exact.shape
    off = np.zeros_like(s, np.float64)
    amax = np.zeros_like(s, np.float64)
    for b in range(s.shape[1]):
        at = np.s_[:, b * 128:(b + 1) * 128]
        off[:, b], amax[:, b] = tol[at].max(1), np.abs(exact[at]).max(1)
    assert (np.abs(s - amax / 448) <= off / 448 + 2.0 ** -23 * amax / 448 + 2.0 ** -149).all()
    full = np.repeat(s.astype(np.float64), 128, 1)[:, :C]
    value = oracle.decode_e4m3(q) * full
    t = np.abs(exact) / np.where(full > 0, full, 1)
    step = np.where(full > 0, oracle.e4m3_half_step(np.minimum(t * (1 + 2.0 ** -18), 448)) * full, 0)
    assert (np.abs(value - exact) <= step * (1 + 2.0 ** -18) + tol + 2.0 ** -22 * np.abs(exact) + 2.0 ** -140).all()


@pytest.mark.parametrize("rows,d", [(1, 16), (3, 128), (5, 144), (70, 400), (33, 1024), (1300, 5120 + 16)])
@pytest.mark.parametrize("std", [0.1, 1.5, 20.0])
def test_swiglu(rows, d, std):
    say(f"swiglu {rows}x{d} {std}")
    gu, _ = grids(11, rows, d, std)
    q, s, y = fp8bs.swiglu_quantize_tg128(gu, want_y=True)
    exact = oracle.swiglu(np64(gu))
    tol = REL * np.abs(exact) + 2.0 ** -140
    assert (np.abs(np64(y) - exact) <= tol + 2.0 ** -8 * np.abs(exact) + 2.0 ** -133).all()
    check_codes(q, s, exact, tol)
    q2, s2 = fp8bs.swiglu_quantize_tg128(gu)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("rows,d", [(1, 16), (3, 128), (5, 144), (70, 400), (33, 1024), (700, 5120), (700, 5120 + 16)])
@pytest.mark.parametrize("std", [0.1, 1.5, 20.0])
def test_swiglu_backward(rows, d, std):
    say(f"swiglu backward {rows}x{d} {std}")
    gu, dy = grids(13, rows, d, std)
    dgu, q, s, y = fp8bs.swiglu_backward_quantize_tg128(gu, dy, want_y=True)
    gu64, dy64 = np64(gu), np64(dy)
    exact = oracle.swiglu_grad(gu64, dy64)
    g, u = gu64[:, :d], gu64[:, d:]
    terms = np.abs(np.concatenate([dy64 * u * (1 + np.abs(g)) / (1 + np.exp(-g)), exact[:, d:]], 1))
    tol = REL * np.maximum(terms, np.abs(exact)) + 2.0 ** -140
    assert (np.abs(np64(dgu) - exact) <= tol + 2.0 ** -8 * np.abs(exact) + 2.0 ** -133).all()
    check_codes(q, s, exact, tol)
    forward = fp8bs.swiglu_quantize_tg128(gu, want_y=True)[2]
    assert torch.equal(y, forward)
    again = fp8bs.swiglu_backward_quantize_tg128(gu, dy)
    assert len(again) == 3 and all(torch.equal(a, b) for a, b in zip(again, (dgu, q, s)))


def test_swiglu_far_gates():
    """Gates beyond exp's range: sigma is 0 or 1, no NaN from finite inputs."""
    far = [3e38, -3e38, 1e30, -1e30, 200.0, -200.0, 95.0, -95.0, 88.0, -88.0, 0.0, -0.0, 1e-38, -1e-38, 30.0, -30.0]
    gu = torch.tensor([far + [1.0] * 16, far + [-0.5] * 16], device=DEV).to(torch.bfloat16)
    y = fp8bs.swiglu_quantize_tg128(gu, want_y=True)[2]
    with np.errstate(over="ignore"):
        exact = oracle.swiglu(np64(gu))
        grad = oracle.swiglu_grad(np64(gu), np.ones((2, 16)))
    assert (np.abs(np64(y) - exact) <= 2.0 ** -8 * np.abs(exact) * (1 + REL) + 2.0 ** -126).all()
    dgu = fp8bs.swiglu_backward_quantize_tg128(gu, torch.ones(2, 16, dtype=torch.bfloat16, device=DEV))[0]
    terms = np.concatenate([np.abs(np64(gu)[:, :16]) * (np.abs(grad[:, :16]) > 0), np.zeros((2, 16))], 1)
    assert (np.abs(np64(dgu) - grad) <= 2.0 ** -8 * np.abs(grad) * (1 + REL) + REL * terms + 2.0 ** -120).all()


def test_swiglu_zero_rows_and_empty():
    gu = torch.zeros(6, 288, dtype=torch.bfloat16, device=DEV)
    q, s = fp8bs.swiglu_quantize_tg128(gu)
    assert (q == 0).all() and (s == 0).all()
    dgu, q, s = fp8bs.swiglu_backward_quantize_tg128(gu, torch.zeros(6, 144, dtype=torch.bfloat16, device=DEV))
    assert (q == 0).all() and (s == 0).all() and (dgu == 0).all()
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    assert fp8bs.swiglu_quantize_tg128(e)[0].shape == (0, 32)
    with pytest.raises(ValueError):
        fp8bs.swiglu_backward_quantize_tg128(gu, gu)


# ---- an expert layer ---------------------------------------------------------------------------
class Layer:
    """Weights laid out once; forward and backward as a training step calls them."""

    def __init__(self, G, d, h, seed=21):
        self.up = fp8bs.quantize_b128(normal(seed, G, 2 * h, d, std=0.05), transposed=True)
        self.down = fp8bs.quantize_b128(normal(seed + 1, G, d, h, std=0.05), transposed=True)

    def step(self, x, dout, offsets):
        qx, sx = fp8bs.quantize_tg128(x)
        gu = fp8bs.grouped_gemm_tg128_nt(qx, sx, *self.up[:2], offsets)
        qy, sy = fp8bs.swiglu_quantize_tg128(gu)
        out = fp8bs.grouped_gemm_tg128_nt(qy, sy, *self.down[:2], offsets)
        qo, so = fp8bs.quantize_tg128(dout)
        dy = fp8bs.grouped_gemm_tg128_nt(qo, so, *self.down[2:], offsets)
        dgu, qg, sg, y = fp8bs.swiglu_backward_quantize_tg128(gu, dy, want_y=True)
        dx = fp8bs.grouped_gemm_tg128_nt(qg, sg, *self.up[2:], offsets)
        dw_down = fp8bs.grouped_wgrad(dout, y, offsets)
        dw_up = fp8bs.grouped_wgrad(dgu, x, offsets)
        return {"gu": gu, "qy": qy, "sy": sy, "out": out, "dy": dy, "dgu": dgu, "dx": dx, "y": y, "qg": qg, "sg": sg,
                "dw_down": dw_down, "dw_up": dw_up, "qx": qx, "sx": sx, "qo": qo, "so": so}


def value(q, s):
    return oracle.dequantize_g128(q.cpu().numpy(), s.cpu().numpy(), 1)


def weight(q, s, g):
    return oracle.dequantize_g128(q[g].cpu().numpy(), s[g].cpu().numpy(), 128)


def close(c, a, w):
    """bf16 result of a product of exact operands: half a bf16 step, and 2^-10 of the magnitude sum for what the
    instruction cuts and fp32 rounds (the products' own bound is tested above)."""
    ref = a @ w.T
    return (np.abs(np64(c) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * (np.abs(a) @ np.abs(w).T)).all()


def test_expert_layer_forward_and_backward():
    """Each step against fp64 on the values that the step before it left, for every expert; one has no rows."""
    G, d, h = 4, 272, 400
    off = [0, 37, 37, 150, 151]
    offsets = i32_dev(off)
    x, dout = normal(31, 151, d), normal(32, 151, d)
    layer = Layer(G, d, h)
    r = layer.step(x, dout, offsets)
    ax, ay, ao, ag = value(r["qx"], r["sx"]), value(r["qy"], r["sy"]), value(r["qo"], r["so"]), value(r["qg"], r["sg"])
    for g in range(G):
        at = slice(off[g], off[g + 1])
        up, down = weight(*layer.up[:2], g), weight(*layer.down[:2], g)
        assert np.array_equal(up.T, weight(*layer.up[2:], g)) and np.array_equal(down.T, weight(*layer.down[2:], g))
        if at.start == at.stop:
            continue
        assert close(r["gu"][at], ax[at], up) and close(r["out"][at], ay[at], down)
        assert close(r["dy"][at], ao[at], down.T) and close(r["dx"][at], ag[at], up.T)
    check_wgrad(r["dw_down"], dout, r["y"], off)
    check_wgrad(r["dw_up"], r["dgu"], x, off)


def test_expert_layer_captured_into_a_graph():
    """The step captured once and replayed with other inputs and other group sizes, with eager work between the
    replays: every replay is the eager step's bits."""
    G, d, h, M = 5, 256, 384, 300
    layer = Layer(G, d, h)
    x, dout = normal(41, M, d), normal(42, M, d)
    offsets = i32_dev([0, 60, 60, 200, 299, 300])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, dout, offsets)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer.step(x, dout, offsets)
    for i, table in enumerate([[0, 60, 60, 200, 299, 300], [0, 0, 0, 300, 300, 300], [0, 1, 2, 3, 4, 300]]):
        x.copy_(normal(50 + i, M, d))
        dout.copy_(normal(60 + i, M, d))
        offsets.copy_(i32_dev(table))
        graph.replay()
        torch.cuda.synchronize()
        eager = layer.step(x, dout, offsets)
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(held[k], eager[k]), (i, k)


def test_two_streams_at_once():
    """Two steps of different layers on two streams: the results of each alone."""
    layers = [Layer(3, 256, 256, 71), Layer(3, 144, 272, 81)]
    xs = [(normal(91 + i, 200, d), normal(95 + i, 200, d)) for i, d in enumerate((256, 144))]
    offsets = i32_dev([0, 100, 101, 200])
    alone = [layer.step(*x, offsets) for layer, x in zip(layers, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    together = [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                together[i] = layers[i].step(*xs[i], offsets)
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        assert all(torch.equal(a[k], b[k]) for k in a)
