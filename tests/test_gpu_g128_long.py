"""The 128-value forms over long sums: products whose K passes every buffer of staged scales, in every tile, and
weight gradients whose fp32 accumulation shows."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, i32_dev, say

pytestmark = pytest.mark.gpu


# ---- products ------------------------------------------------------------------------------
# Scales of A are staged eight K-blocks at a time in two buffers, a weight's 64 at a time: 18 blocks read each buffer
# again, 66 fetch the weight's again; both K end in a partial block.  One size for each tile the dispatch takes, with
# a ragged last tile both ways and every wave of a whole tile live.  The last of both lists has more tiles than the
# large form has workgroups.
LONG_K = [2192, 8336]
DENSE = [(9, 1040), (20, 2064), (30, 10256), (50, 16528), (500, 3600), (1000, 2320), (1000, 4624), (1000, 9232),
         (400, 7184), (3500, 4112), (4500, 4160)]
RANGED = [(7, 60, 1040), (7, 60, 3600), (5, 300, 1808), (5, 300, 4112), (5, 300, 5200), (3, 1000, 4368),
          (3, 1000, 3472), (3, 1000, 7200), (4, 8000, 1296), (6, 4000, 4160)]


def operands(seed, M, N, K, *lead):
    """Finite codes of both signs and scales on the device."""
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def codes(*shape):
        c = torch.randint(0, 256, shape, generator=gen, device=DEV, dtype=torch.uint8)
        return torch.where((c & 0x7F) == 0x7F, c - 1, c)

    def scales(*shape):
        return torch.rand(*shape, generator=gen, device=DEV) + 0.5
    KB, NB = -(-K // 128), -(-N // 128)
    return codes(M, K), scales(M, KB), codes(*lead, N, K), scales(*lead, NB, KB)


def rows_are_right(c, rows, a, sa, bt, sbt):
    """Rows of c: bit for bit the one-row call's, and within the bound in the columns of three weight blocks' ends."""
    N = bt.shape[0]
    for r in rows:
        one = fp8bs.gemm_tg128_nt(a[r:r + 1].clone(), sa[r:r + 1].clone(), bt, sbt)
        assert torch.equal(one[0].view(torch.int16), c[r].view(torch.int16)), r
    at = torch.tensor(rows, device=DEV)
    host = [t.cpu().numpy() for t in (c[at].double(), a[at], sa[at])]
    for c0 in (0, N // 256 * 128 + 120, N - 8):
        w = slice(c0, c0 + 8)
        ref, bound = oracle.gemm_g128_bound(host[1], host[2], bt[w].cpu().numpy(),
                                            sbt[c0 // 128:c0 // 128 + 1].cpu().numpy())
        assert (np.abs(host[0][:, w] - ref) <= bound).all(), c0


@pytest.mark.parametrize("K", LONG_K)
@pytest.mark.parametrize("M,N", DENSE)
def test_long_k(M, N, K):
    say(f"gemm_tg128_nt {M}x{N}x{K}")
    ops = operands(M + N + K, M, N, K)
    c = fp8bs.gemm_tg128_nt(*ops)
    rows_are_right(c, sorted({0, M // 3, M - 150 if M > 300 else M // 2, M - 1}), *ops)


@pytest.mark.parametrize("K", LONG_K)
@pytest.mark.parametrize("G,M,N", RANGED)
def test_long_k_of_ranges(G, M, N, K):
    say(f"grouped {G} {M} {N} {K}")
    cuts = np.sort(np.random.default_rng(G + M).integers(0, M + 1, G + 1)).astype(np.int32)
    a, sa, bt, sbt = operands(G + N, M, N, K, G)
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    fp8bs.grouped_gemm_tg128_nt(a, sa, bt, sbt, i32_dev(cuts), out)
    for g in range(G):
        b, e = int(cuts[g]), int(cuts[g + 1])
        if b < e:
            rows_are_right(out, sorted({b, (b + e) // 2, e - 1}), a, sa, bt[g], sbt[g])
    assert (out[:cuts[0]] == 3.0).all() and (out[cuts[-1]:] == 3.0).all()


# ---- weight gradients --------------------------------------------------------------------------
# One size for each tile that the dispatch takes.
GRADIENTS = [(16, 6500, 2064, 2000), (4, 2000, 2048, 2064), (1, 8000, 2048, 2000), (8, 1010, 2064, 2000),
             (8, 333, 1040, 528), (1, 8000, 272, 144)]


def ranges(G, M):
    off = np.sort(np.random.default_rng(G * M).integers(0, M + 1, G + 1))
    if G == 1:
        off[0], off[1] = 5, M - 3
    return off


@pytest.mark.parametrize("G,M,N,K", GRADIENTS)
def test_wgrad_of_integers_is_exact(G, M, N, K):
    """Operands of [-40, 40] and at most 8000 rows: every partial sum is a whole number below 8000 * 1600 = 12.8e6, with
    the old values of at most 10^6 below 2^24, which fp32 holds: the result is the sum itself, in whatever order.  A row
    that is left out, taken twice or taken from elsewhere shows, and so does a sum held in fewer bits."""
    say(f"wgrad of integers {G} {M} {N}x{K}")
    gen = torch.Generator(device=DEV).manual_seed(G + M)
    dy = torch.randint(-40, 41, (M, N), generator=gen, device=DEV).bfloat16()
    x = torch.randint(-40, 41, (M, K), generator=gen, device=DEV).bfloat16()
    old = torch.randint(-10 ** 6, 10 ** 6 + 1, (G, N, K), generator=gen, device=DEV).float()
    off = ranges(G, M)
    dw = fp8bs.grouped_wgrad(dy, x, i32_dev(off))
    added = fp8bs.grouped_wgrad(dy, x, i32_dev(off), old.clone(), accumulate=True)
    for g in range(G):
        r = slice(int(off[g]), int(off[g + 1]))
        ref = dy[r].double().t() @ x[r].double()
        assert torch.equal(dw[g].double(), ref), g
        assert torch.equal(added[g].double(), ref + old[g].double()), g


@pytest.mark.parametrize("G,M,N,K", [(1, 8000, 2048, 2000), (2, 4000, 2048, 2064), (1, 8000, 272, 144)])
def test_wgrad_against_its_running_sums(G, M, N, K):
    """32 rows enter at a time, by at most 32 additions, each within 2^-23 of a value that is at most the sum before
    them and the magnitudes of the 32 products."""
    say(f"wgrad running sums {G} {M} {N}x{K}")
    gen = torch.Generator(device=DEV).manual_seed(M + N)
    dy = torch.randn(M, N, generator=gen, device=DEV).bfloat16()
    x = torch.randn(M, K, generator=gen, device=DEV).bfloat16()
    off = ranges(G, M)
    dw = fp8bs.grouped_wgrad(dy, x, i32_dev(off))
    for g in range(G):
        ref = torch.zeros(N, K, dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(ref)
        for b in range(int(off[g]), int(off[g + 1]), 32):
            r = slice(b, min(b + 32, int(off[g + 1])))
            p, q = dy[r].double(), x[r].double()
            tol += 32 * 2.0 ** -23 * (ref.abs() + p.abs().t() @ q.abs())
            ref += p.t() @ q
        assert ((dw[g] - ref).abs() <= tol).all(), g
