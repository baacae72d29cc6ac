"""The operators between the products on what is larger than the caches, and past 32-bit offsets: rows are the bits that
they have in a small call, sums are held against float64."""

import pytest
import torch

import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
EPS = 1e-5
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def rows_of(rows, d, seed, std=1.0):
    """bf16 rows from 4096 random ones, each times a power of two that goes by its number (quick to make)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    some = (torch.randn(4096, d, generator=g, device=DEV) * std).to(torch.bfloat16)
    out = torch.empty(rows, d, dtype=torch.bfloat16, device=DEV)
    for i, at in enumerate(range(0, rows, 4096)):
        n = min(4096, rows - at)
        out[at:at + n] = some[:n] * 2.0 ** (i % 3)
    return out


def equal(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def sum64(rows, of, step=1 << 14):
    """Sum over the rows, and of the magnitudes, in float64."""
    total = size = None
    for at in range(0, rows, step):
        t = of(slice(at, min(rows, at + step)))
        total, size = (t.sum(0), t.abs().sum(0)) if total is None else (total + t.sum(0), size + t.abs().sum(0))
    return total, size


@pytest.mark.parametrize("rows,d", [(6001, 16384), (50003, 2064), (270001, 16384)])
def test_layernorm(rows, d):
    say(f"layernorm {rows}x{d}")
    x, r = rows_of(rows, d, 1), rows_of(rows, d, 2)
    gamma, beta = rows_of(1, d, 3)[0], rows_of(1, d, 4)[0]
    q, s, y, mean, rstd = fp8bs.layernorm_quantize_tg128(x, gamma, beta, EPS, residual=r, h=x, want_y=True,
                                                         want_stats=True)  # the sum over x
    small = [slice(0, 3), slice(rows // 2, rows // 2 + 2), slice(rows - 3, rows)]
    for at in small:
        x1 = (rows_of(rows, d, 1)[at] if rows < 100000 else None)
        if x1 is not None:
            one = fp8bs.layernorm_quantize_tg128(x1.clone(), gamma, beta, EPS, residual=r[at].clone(), want_y=True,
                                                 want_stats=True)
        else:  # the sum is there
            one = fp8bs.layernorm_quantize_tg128(x[at].clone(), gamma, beta, EPS, want_y=True, want_stats=True)
        assert all(equal(a, b[at]) for a, b in zip(one, (q, s, y, mean, rstd))), at
    del q, s, y
    dy = rows_of(rows, d, 5, std=0.01)
    dx, dgamma, dbeta = fp8bs.layernorm_backward(dy, x, gamma, mean, rstd, dresidual=r)
    for at in small:
        one = fp8bs.layernorm_backward(dy[at].clone(), x[at].clone(), gamma, mean[at].clone(), rstd[at].clone(),
                                       dresidual=r[at].clone())[0]
        assert equal(one, dx[at]), at
    del dx
    # rows / 256 additions of a workgroup, 16 rows or fewer at a time, then 256 partial sums: each off by U
    steps = rows / 256 + 300
    for got, of in ((dgamma, lambda at: dy[at].double() * ((x[at].double() - mean[at, None].double())
                                                           * rstd[at, None].double())),
                    (dbeta, lambda at: dy[at].double())):
        want, size = sum64(rows, of)
        assert ((got.double() - want).abs() <= (steps + 4) * U * size).all()


@pytest.mark.parametrize("rows,n,act", [(8001, 16384, "gelu"), (30001, 4112, "silu"), (140001, 32768, "gelu_tanh")])
def test_epilogue_backward(rows, n, act):
    say(f"epilogue_backward {rows}x{n} {act}")
    dout, pre = rows_of(rows, n, 1, std=0.01), rows_of(rows, n, 2)
    dz, q, s, dbias = fp8bs.epilogue_backward_quantize_tg128(dout, pre, act)
    for at in (slice(0, 3), slice(rows // 2, rows // 2 + 2), slice(rows - 3, rows)):
        one = fp8bs.epilogue_backward_quantize_tg128(dout[at].clone(), pre[at].clone(), act)
        assert all(equal(a, b[at]) for a, b in zip(one, (dz, q, s))), at
    del q, s, dout, pre
    # against the sums of the rounded dz: half a bf16 step of each, and the additions of a slab's and the slabs' sums
    want, size = sum64(rows, lambda at: dz[at].double())
    slabs = max(1, 8192 // (-(-n // 128)))
    assert ((dbias.double() - want).abs() <= (2.0 ** -8 + (rows / 4 / slabs + slabs + 8) * U) * size).all()


@pytest.mark.parametrize("rows,n", [(3, 64 * 65536 + 80), (1, (1 << 28) + 2064)])
def test_sums_over_many_columns(rows, n):
    say(f"epilogue_backward {rows}x{n}")
    dout = rows_of(n // 16, 16, 1).view(1, n).repeat(rows, 1)
    old = torch.ones(n, device=DEV)
    dbias = fp8bs.epilogue_backward_quantize_tg128(dout, None, dbias=old, accumulate=True)[3]
    want = dout[0].float() * rows  # exact: at most three times eight bits; the addition of 1 rounds
    assert torch.equal(dbias, want + 1.0)


@pytest.mark.parametrize("M,N", [(66001, 65552)])
def test_product_with_epilogue_past_32_bits(M, N):
    K = 16
    say(f"epilogue {M}x{N}x{K}")
    a, sa = fp8bs.quantize_tg128(rows_of(M, K, 1))
    bt, sbt = fp8bs.quantize_b128(rows_of(N, K, 2))
    bias = rows_of(1, N, 3)[0]
    res = rows_of(M, N, 4)
    out, pre = fp8bs.gemm_tg128_nt_epilogue(a, sa, bt, sbt, bias=bias, activation="silu", residual=res, want_pre=True)
    for r in (0, M // 2, M - 1):
        at = slice(r, r + 1)
        one = fp8bs.gemm_tg128_nt_epilogue(a[at], sa[at], bt, sbt, bias=bias, activation="silu", residual=res[at],
                                           want_pre=True)
        assert equal(one[0], out[at]) and equal(one[1], pre[at]), r


@pytest.mark.parametrize("M,N", [(3500, 4160), (2600, 16400)])
def test_no_k_in_the_large_tile(M, N):
    say(f"epilogue {M}x{N}x0")
    empty = (torch.zeros(M, 0, dtype=torch.uint8, device=DEV), torch.zeros(M, 0, device=DEV),
             torch.zeros(N, 0, dtype=torch.uint8, device=DEV), torch.zeros(-(-N // 128), 0, device=DEV))
    bias, res = rows_of(1, N, 1)[0], rows_of(M, N, 2)
    out, pre = fp8bs.gemm_tg128_nt_epilogue(*empty, bias=bias, activation="gelu", residual=res, want_pre=True)
    assert equal(pre, bias.expand(M, N))
    for r in (0, 300, M - 1):
        one = fp8bs.gemm_tg128_nt_epilogue(empty[0][:1], empty[1][:1], *empty[2:], bias=bias, activation="gelu",
                                           residual=res[r:r + 1])
        assert equal(one, out[r:r + 1]), r


@pytest.mark.parametrize("sizes", [[60_000_000, 7, 100_000_001], [200_000_003, 1, 12345], [(1 << 32) + 1001]])
def test_clip(sizes):
    say(f"clip {sizes}")
    grads = []
    for i, n in enumerate(sizes):
        g = torch.empty(n, device=DEV).uniform_(-1, 1, generator=torch.Generator(device=DEV).manual_seed(i))
        grads.append(g.to(torch.bfloat16) if i == 1 else g)
    want = sum(float(p.double().square().sum()) for g in grads for p in g.split(1 << 28)) ** 0.5
    assert abs(float(fp8bs.grad_norm(grads)) - want) <= (2.0 ** -24 + 2.0 ** -40) * want
    parts = [(g, at) for g in grads for at in (slice(0, 1000), slice(max(0, g.numel() - 1000), g.numel()))]
    old = [g[at].clone() for g, at in parts]
    norm = fp8bs.clip_grad_norm(grads, want / 3)
    assert abs(float(norm) - want) <= (2.0 ** -24 + 2.0 ** -40) * want
    factor = (want / 3) / (want + 1e-6)
    for (g, at), o in zip(parts, old):
        ref = o.double() * factor
        tol = (2 * U + (2.0 ** -8 if g.dtype == torch.bfloat16 else 0.0) + 2.0 ** -40) * ref.abs() + 2.0 ** -134
        assert ((g[at].double() - ref).abs() <= tol).all()
