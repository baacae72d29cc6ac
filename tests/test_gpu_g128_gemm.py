"""E4M3 products with scales of 128 values: within the derived bound of the fp64
result, bitwise the same whatever M, the row's place or the grouping, rows
outside every range untouched."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, f32_dev, i32_dev, say, u8_dev

pytestmark = pytest.mark.gpu


def codes(rng, *shape, spread=1.0):
    """Codes of normal values scaled to the whole range, as a quantizer leaves them."""
    v = np.clip(rng.normal(size=shape) * 140 * np.exp(rng.normal(size=shape) * spread), -448, 448)
    return oracle.encode_e4m3(v.astype(np.float32))


def operands(seed, M, N, K, groups=None):
    rng = np.random.default_rng(seed)
    lead = () if groups is None else (groups,)
    nk, nn = -(-K // 128), -(-N // 128)
    return (codes(rng, M, K), np.exp(rng.normal(size=(M, nk))).astype(np.float32),
            codes(rng, *lead, N, K), np.exp(rng.normal(size=lead + (nn, nk))).astype(np.float32) * np.float32(1e-3))


def f64(c):
    return c.float().cpu().numpy().astype(np.float64)


def dev(ops):
    return u8_dev(ops[0]), f32_dev(ops[1]), u8_dev(ops[2]), f32_dev(ops[3])


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 16, 128), (1, 128, 1040), (3, 272, 144), (16, 144, 256),
                                   (17, 16, 2064), (33, 48, 400), (64, 80, 272), (65, 144, 384), (127, 64, 128),
                                   (130, 272, 1152)])
def test_within_the_bound(M, N, K):
    say(f"gemm_tg128_nt {M}x{N}x{K}")
    ops = operands(M * 7 + N + K, M, N, K)
    c = f64(fp8bs.gemm_tg128_nt(*dev(ops)))
    ref, bound = oracle.gemm_g128_bound(*ops)
    assert (np.abs(c - ref) <= bound).all(), float((np.abs(c - ref) / bound).max())


def rows_of(ops, rows):
    a, sa, bt, sbt = ops
    return a[rows], sa[rows], bt, sbt


@pytest.mark.parametrize("N,K", [(4112, 1040), (8192, 2048), (272, 528)])
def test_rows_do_not_depend_on_m(N, K):
    """The same rows alone, in small batches and in large ones (every kernel): the same bits, and those bits within
    the bound at sampled columns."""
    ops = operands(N, 4352, N, K)
    a, sa, bt, sbt = dev(ops)
    full = fp8bs.gemm_tg128_nt(a, sa, bt, sbt)
    at = np.r_[0:8, N // 2 - 8:N // 2 + 8, N - 16:N]
    cols = np.unique(at)
    for r in (0, 700, 4351):
        ref, bound = oracle.gemm_g128_bound(ops[0][r:r + 1], ops[1][r:r + 1], ops[2], ops[3])
        off = np.abs(f64(full[r:r + 1]) - ref)[:, cols]
        assert (off <= bound[:, cols]).all()
    for M in (1, 2, 16, 17, 32, 33, 64, 65, 100, 129, 256, 300, 700, 1500, 2600):
        for first in (0, 4352 - M):
            say(f"M={M} first={first}")
            part = fp8bs.gemm_tg128_nt(a[first:first + M].clone(), sa[first:first + M].clone(), bt, sbt)
            assert torch.equal(part.view(torch.int16), full[first:first + M].view(torch.int16)), (M, first)


# One size for each tile that the dispatch can take, with a ragged last tile both ways and a partial last K-block;
# where waves have 64 columns, one with N a multiple of that as well.
DENSE = [(9, 1040), (20, 2064), (40, 1040), (13, 8208), (30, 10256), (50, 16528), (100, 4112), (500, 3600),
         (1000, 2320), (1000, 4624), (1000, 9232), (400, 7184), (1700, 4112), (3500, 4112),
         (1000, 2368), (1000, 9280), (400, 7232), (1700, 4160), (3500, 4160)]
RANGED = [(7, 60, 1040), (7, 60, 3600), (5, 300, 1808), (5, 300, 4112), (5, 300, 5200), (3, 1000, 4368),
          (3, 1000, 3472), (3, 1000, 7200), (4, 2000, 3600), (4, 8000, 1296), (4, 8000, 1344),
          (5, 300, 5248), (3, 1000, 7232)]


@pytest.mark.parametrize("K", [400, 1168])
@pytest.mark.parametrize("M,N", DENSE)
def test_every_tile(M, N, K):
    say(f"gemm_tg128_nt {M}x{N}x{K}")
    ops = operands(M + N + K, M, N, K)
    a, sa, bt, sbt = dev(ops)
    c = fp8bs.gemm_tg128_nt(a, sa, bt, sbt)
    for r in sorted({0, M // 2, M - 1}):
        one = fp8bs.gemm_tg128_nt(a[r:r + 1].clone(), sa[r:r + 1].clone(), bt, sbt)
        assert torch.equal(one[0].view(torch.int16), c[r].view(torch.int16)), r
    cols = np.unique(np.r_[0:8, N // 2:N // 2 + 8, N - 8:N])
    rows = np.unique(np.linspace(0, M - 1, 12).astype(int))
    ref, bound = oracle.gemm_g128_bound(ops[0][rows], ops[1][rows], ops[2], ops[3])
    assert (np.abs(f64(c[torch.from_numpy(rows).to(DEV)]) - ref)[:, cols] <= bound[:, cols]).all()


@pytest.mark.parametrize("K", [400, 1168])
@pytest.mark.parametrize("G,M,N", RANGED)
def test_every_tile_of_ranges(G, M, N, K):
    rng = np.random.default_rng(G + M)
    cuts = np.sort(rng.integers(0, M + 1, G + 1)).astype(np.int32)
    a, sa, bt, sbt = dev(operands(G + N, M, N, K, G))
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    say(f"grouped {G} {M} {N} {K}")
    fp8bs.grouped_gemm_tg128_nt(a, sa, bt, sbt, i32_dev(cuts), out)
    for g in range(G):
        r = slice(int(cuts[g]), int(cuts[g + 1]))
        if r.start < r.stop:
            one = fp8bs.gemm_tg128_nt(a[r].clone(), sa[r].clone(), bt[g].clone(), sbt[g].clone())
            assert torch.equal(out[r].view(torch.int16), one.view(torch.int16)), g
    assert (out[:cuts[0]] == 3.0).all() and (out[cuts[-1]:] == 3.0).all()


def test_k_zero_and_empty():
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    f = lambda *s: torch.zeros(*s, device=DEV)                     # noqa: E731
    out = torch.full((5, 32), 7.0, dtype=torch.bfloat16, device=DEV)
    fp8bs.gemm_tg128_nt(z(5, 0), f(5, 0), z(32, 0), f(1, 0), out)
    assert (out.view(torch.int16) == 0).all()
    assert fp8bs.gemm_tg128_nt(z(0, 64), f(0, 1), z(32, 64), f(1, 1)).shape == (0, 32)
    assert fp8bs.gemm_tg128_nt(z(5, 64), f(5, 1), z(0, 64), f(0, 1)).shape == (5, 0)


def test_not_finite_reaches_its_row_or_column_only():
    ops = operands(3, 200, 272, 400)
    good = fp8bs.gemm_tg128_nt(*dev(ops))
    a, sa, bt, sbt = (x.copy() for x in ops)
    a[70, 399] = 0x7F
    sa[150, 2] = np.inf
    bt[131, 0] = 0xFF
    c = fp8bs.gemm_tg128_nt(*dev((a, sa, bt, sbt)))
    assert torch.isnan(c[70]).all() and torch.isnan(c[:, 131]).all()
    assert not torch.isfinite(c[150]).any()
    keep_r = [r for r in range(200) if r not in (70, 150)]
    keep_c = [n for n in range(272) if n != 131]
    assert torch.equal(c[keep_r][:, keep_c], good[keep_r][:, keep_c])


def test_zero_is_stored_as_plus_zero():
    ops = list(operands(4, 70, 32, 256))
    ops[0][:] = 0x80
    c = fp8bs.gemm_tg128_nt(*dev(ops))
    assert (c.view(torch.int16) == 0).all()


# ---- groups --------------------------------------------------------------------------------
GROUPS = [[5], [0], [1, 0, 3], [0, 0, 130, 1, 0], [33, 64, 2, 17], [300, 1, 0, 257], [1] * 70,
          [0] * 40 + [9] + [0] * 90, [1] * 20 + [700] + [0, 3] * 12,
          [64, 65, 63, 0, 66, 20, 31], [20] * 3 + [200], [0] * 1000 + [5] + [0] * 23]


@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: f"{len(s)}x{sum(s)}")
@pytest.mark.parametrize("N,K", [(144, 272)])
def test_groups_are_the_single_products(sizes, N, K):
    say(f"grouped {sizes[:8]}")
    G, M = len(sizes), sum(sizes) + 5          # five rows behind the last range
    a, sa, bt, sbt = dev(operands(G, M, N, K, G))
    off = np.concatenate([[0], np.cumsum(sizes)])
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    fp8bs.grouped_gemm_tg128_nt(a, sa, bt, sbt, i32_dev(off), out)
    for g in range(G):
        r = slice(int(off[g]), int(off[g + 1]))
        if r.start < r.stop:
            one = fp8bs.gemm_tg128_nt(a[r].clone(), sa[r].clone(), bt[g].clone(), sbt[g].clone())
            assert torch.equal(out[r].view(torch.int16), one.view(torch.int16)), g
    assert (out[off[-1]:] == 3.0).all()


@pytest.mark.parametrize("G,M,N,K", [(3, 2000, 1040, 528), (16, 4000, 4096, 272), (40, 4000, 2048, 144)])
def test_large_groups(G, M, N, K):
    """Sizes that reach the large tiles, ranges that start after row 0 and end before the last."""
    rng = np.random.default_rng(G)
    cuts = np.sort(rng.integers(10, M - 10, G + 1)).astype(np.int32)
    a, sa, bt, sbt = dev(operands(G + 1, M, N, K, G))
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    say(f"grouped {G} {M} {N} {K}")
    fp8bs.grouped_gemm_tg128_nt(a, sa, bt, sbt, i32_dev(cuts), out)
    for g in range(G):
        r = slice(int(cuts[g]), int(cuts[g + 1]))
        if r.start < r.stop:
            one = fp8bs.gemm_tg128_nt(a[r].clone(), sa[r].clone(), bt[g].clone(), sbt[g].clone())
            assert torch.equal(out[r].view(torch.int16), one.view(torch.int16)), g
    assert (out[:cuts[0]] == 3.0).all() and (out[cuts[-1]:] == 3.0).all()


@pytest.mark.parametrize("table", [[0, -4, 7, 20], [5, 3, 2, 1], [0, 100, 1 << 30, 9], [-9, 0, 40, 1000]])
def test_bad_tables_stay_inside(table):
    """Entries outside [0, M] and ranges that run backwards: nothing outside the rows is written, and a well-formed
    clamped range still gets its product."""
    M, N, K = 40, 32, 144
    a, sa, bt, sbt = dev(operands(9, M, N, K, 3))
    whole = torch.full((M + 64, N), 3.0, dtype=torch.bfloat16, device=DEV)
    out = whole[:M]
    fp8bs.grouped_gemm_tg128_nt(a, sa, bt, sbt, i32_dev(table), out)
    assert (whole[M:] == 3.0).all()
    clamped = [min(max(t, 0), M) for t in table]
    if all(x <= y for x, y in zip(clamped, clamped[1:])):
        for g in range(3):
            r = slice(clamped[g], clamped[g + 1])
            if r.start < r.stop:
                one = fp8bs.gemm_tg128_nt(a[r].clone(), sa[r].clone(), bt[g].clone(), sbt[g].clone())
                assert torch.equal(out[r], one)


def test_refusals_on_the_device():
    a, sa, bt, sbt = dev(operands(1, 8, 32, 64))
    with pytest.raises(ValueError):
        fp8bs.gemm_tg128_nt(a, sa[:, :0], bt, sbt)
    with pytest.raises(ValueError):
        fp8bs.gemm_tg128_nt(a, sa, bt, sbt, torch.empty(8, 16, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        fp8bs.gemm_tg128_nt(a[:, :48].contiguous(), sa, bt, sbt)
    with pytest.raises(ValueError):
        fp8bs.gemm_tg128_nt(a.t(), sa, bt, sbt)
    with pytest.raises(TypeError):
        fp8bs.gemm_tg128_nt(a, sa.double(), bt, sbt)
    with pytest.raises(fp8bs.Fp8bsError):   # K not a multiple of 16
        fp8bs.gemm_tg128_nt(a[:, :40].contiguous(), sa, bt[:, :40].contiguous(), sbt)
    off = i32_dev([0, 8])
    with pytest.raises(ValueError):
        fp8bs.grouped_gemm_tg128_nt(a, sa, bt[None], sbt[None], i32_dev([0, 4, 8]))
    with pytest.raises(TypeError):
        fp8bs.grouped_gemm_tg128_nt(a, sa, bt[None], sbt[None], off.long())
    with pytest.raises(ValueError):
        fp8bs.grouped_gemm_tg128_nt(a, sa, bt[None], sbt[None], off.cpu())
