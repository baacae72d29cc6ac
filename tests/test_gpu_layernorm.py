"""Residual add + layer norm + row quantizer, and the backward pass, against float64.

Tolerances.  u = 2^-24 is fp32's half step, 2^-8 bf16's.

Forward: a row's sums of d values run over a lane's columns (at most 32), six levels of a butterfly and at most
eight waves: at most n = 46 additions deep, each off by u.
- mean: m is off by at most n u sum|h|/d; delta repairs it but for n u sum|h - m|/d and u |m| of rounding.
- var: off by n u of itself (sums of squares), a few u more for its products; rstd then by half of that and 4 u.
- y: the deviation is off by 2 u of |h - m| and of |delta| and by delta's own error; the product by 3 u more:
      |y - ref| <= |gamma| rstd (|dev| (n/2 + 8) u + (n + 4) u mean|h - mu|) + 2 u |y|, then bf16's half step.
Codes: the scale is off as y is, the code may be the neighbour's where the quotient is that near to a border:
      |q s - ref| <= half an E4M3 step of the quotient + what y and the scale are off by.

Backward: the kernel's formula on the same mean and rstd, sums as above:
      dx: c1 and c2 are off by (n + 3) u of mean|g| and mean|g xh|; every product by a few u.
      dgamma, dbeta: at most rows additions, each off by u of a partial sum, bounded by sum|terms|."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U, N = 2.0 ** -24, 46
EPS = 1e-5


def np64(t):
    return t.cpu().double().numpy()


def normal(seed, *shape, std=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + shift).to(torch.bfloat16).to(DEV)


def reference(h, gamma, beta, eps):
    h = np64(h)
    mean = h.mean(1, keepdims=True)
    var = ((h - mean) ** 2).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (h - mean) * rstd * np64(gamma) + (0.0 if beta is None else np64(beta))
    dev = np.abs(h - mean)
    off = np.abs(np64(gamma)) * rstd * (dev * (N / 2 + 8) * U + (N + 4) * U * dev.mean(1, keepdims=True)
                                        + 2 * U * U * np.abs(mean) * N) + 2 * U * np.abs(y)
    return mean[:, 0], rstd[:, 0], y, off


def check_codes(q, s, y, off):
    """Codes and scales of values that are within `off` of y."""
    q, s = q.cpu().numpy(), s.cpu().double().numpy()
    d = y.shape[1]
    for b in range(s.shape[1]):
        at = slice(128 * b, min(d, 128 * b + 128))
        amax, slack = np.abs(y[:, at]).max(1), off[:, at].max(1)
        ref = amax / 448.0
        tol = slack / 448.0 + 2 * U * ref + 2.0 ** -149
        assert (np.abs(s[:, b] - ref) <= tol).all(), b
        sc = s[:, b:b + 1]
        t = np.where(sc > 0, y[:, at] / np.where(sc > 0, sc, 1.0), 0.0)
        loose = np.where(sc > 0, off[:, at] / np.where(sc > 0, sc, 1.0), 0.0) + 2 * U * np.abs(t)
        code = oracle.decode_e4m3(q[:, at])
        half = oracle.g128.e4m3_half_step(np.minimum(np.abs(t) + loose, 448.0))
        assert (np.abs(code - t) <= half + loose).all(), b


def run_forward(x, gamma, beta, residual, eps=EPS, label=""):
    say(f"layernorm {tuple(x.shape)} {label}")
    rows, d = x.shape
    h = torch.empty_like(x) if residual is not None else None
    q, s, y, mean, rstd = fp8bs.layernorm_quantize_tg128(x, gamma, beta, eps, residual=residual, h=h, want_y=True,
                                                         want_stats=True)
    if residual is not None:
        assert torch.equal(h.view(torch.int16), (x.float() + residual.float()).to(torch.bfloat16).view(torch.int16))
    else:
        h = x
    mu, rs, ref, off = reference(h, gamma, beta, eps)
    habs = np.abs(np64(h))
    assert (np.abs(np64(mean) - mu) <= 2 * U * np.abs(mu) + N * U * np.abs(np64(h) - mu[:, None]).mean(1)
            + N * N * U * U * habs.mean(1) + 2.0 ** -149).all()
    assert (np.abs(np64(rstd) - rs) <= (N / 2 + 6) * U * rs).all()
    assert (np.abs(np64(y) - ref) <= (off + 2.0 ** -8 * (np.abs(ref) + off) + 2.0 ** -134)).all()
    check_codes(q, s, ref, off)
    # every other choice of outputs gives the same bits
    q2, s2 = fp8bs.layernorm_quantize_tg128(x, gamma, beta, eps, residual=None if residual is None
                                            else residual.clone())
    assert torch.equal(q, q2) and torch.equal(s, s2)
    y2, mean2, rstd2 = fp8bs.layernorm(x, gamma, beta, eps, residual=None if residual is None else residual.clone(),
                                       want_stats=True)
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16))
    assert torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    return h, q, s, y, mean, rstd


SHAPES = [(1, 16), (5, 48), (33, 128), (7, 496), (3, 512), (9, 528), (2, 1024), (6, 1040), (17, 2048), (5, 2064),
          (4, 4096), (3, 4112), (11, 7168), (2, 8192), (3, 8208), (2, 16384), (1, 16368)]


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("with_residual,with_beta", [(True, True), (False, False)])
def test_forward(rows, d, with_residual, with_beta):
    x = normal(d + rows, rows, d, shift=0.3)
    gamma, beta = normal(1, d, std=0.1, shift=1.0), normal(2, d, std=0.2)
    run_forward(x, gamma, beta if with_beta else None, normal(3, rows, d, std=2.0) if with_residual else None)


def test_forward_more_rows_than_workgroups():
    x, r = normal(5, 5001, 2064), normal(6, 5001, 2064)
    run_forward(x, normal(1, 2064, shift=1.0), normal(2, 2064), r)


@pytest.mark.parametrize("d", [256, 2048, 8192])
def test_rows_far_from_zero_and_special_rows(d):
    """A mean a thousand times the deviation, tiny and huge rows, a zero row, a constant row, one value alone."""
    x = normal(7, 8, d)
    x[0] = (torch.randn(d) + 1000.0).to(torch.bfloat16)
    x[1] = normal(8, d, std=1e-18)
    x[2] = normal(9, d, std=1e15)
    x[3] = 0
    x[4] = 3.0
    x[5] = 0
    x[5, d // 2] = 100.0
    gamma, beta = normal(1, d, std=0.1, shift=1.0), normal(2, d, std=0.2)
    gamma[:16] = 0
    h, q, s, y, mean, rstd = run_forward(x, gamma, beta, None, label="special")
    assert torch.equal(y[3].view(torch.int16), y[4].view(torch.int16))  # both are beta
    assert torch.equal(mean[3:5].cpu(), torch.tensor([0.0, 3.0]))


@pytest.mark.parametrize("d", [528, 4096, 8192, 16384])
def test_rows_do_not_depend_on_the_batch(d):
    x, r = normal(10, 70, d), normal(11, 70, d)
    gamma, beta = normal(1, d, shift=1.0), normal(2, d)
    say(f"invariance {d}")
    full = fp8bs.layernorm_quantize_tg128(x, gamma, beta, EPS, residual=r.clone(), want_y=True, want_stats=True)
    for a, b in ((0, 1), (69, 70), (3, 20)):
        part = fp8bs.layernorm_quantize_tg128(x[a:b], gamma, beta, EPS, residual=r[a:b].clone(), want_y=True,
                                              want_stats=True)
        for p, f in zip(part, full):
            assert torch.equal(p.view(torch.uint8), f[a:b].view(torch.uint8))


def test_sum_written_in_place_or_apart():
    x, r = normal(12, 9, 272), normal(13, 9, 272)
    gamma = normal(1, 272, shift=1.0)
    say("in place")
    want = (x.float() + r.float()).to(torch.bfloat16)
    a, b, c = r.clone(), r.clone(), x.clone()
    qa, _ = fp8bs.layernorm_quantize_tg128(x, gamma, None, EPS, residual=a)
    h = torch.empty_like(x)
    qb, _ = fp8bs.layernorm_quantize_tg128(x, gamma, None, EPS, residual=b, h=h)
    qc, _ = fp8bs.layernorm_quantize_tg128(c, gamma, None, EPS, residual=b, h=c)
    assert torch.equal(a, want) and torch.equal(h, want) and torch.equal(b, r) and torch.equal(c, want)
    assert torch.equal(qa, qb) and torch.equal(qa, qc)
    with pytest.raises(ValueError):
        fp8bs.layernorm(x, gamma, None, EPS, h=h)
    with pytest.raises(ValueError):
        fp8bs.layernorm(x, gamma[:256], None, EPS)
    with pytest.raises(ValueError):
        fp8bs.layernorm(x[:, :256], gamma[:256], None, EPS)  # not contiguous
    with pytest.raises(TypeError):
        fp8bs.layernorm(x.float(), gamma, None, EPS)
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.layernorm(x, gamma, None, -1.0)


# ---- backward ----------------------------------------------------------------------------
def check_backward(dy, h, gamma, mean, rstd, dres, got, old=None):
    dx, dgamma, dbeta = (np64(t) for t in got)
    dy, h, gamma = np64(dy), np64(h), np64(gamma)
    mean, rstd = np64(mean)[:, None], np64(rstd)[:, None]
    xh = (h - mean) * rstd
    g = dy * gamma
    c1, c2 = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * xh).mean(1, keepdims=True)
    ref = rstd * (g - c1 - xh * c2)
    # xh: off by 2 u; the sums by n + 3 u of the mean of magnitudes; then four roundings
    off = rstd * (8 * U * (np.abs(g) + np.abs(c1) + np.abs(xh * c2)) + (N + 6) * U * (a1 + np.abs(xh) * a2))
    if dres is not None:
        ref = ref + np64(dres)
        off = off + U * np.abs(ref)
    assert (np.abs(dx - ref) <= off + 2.0 ** -8 * (np.abs(ref) + off) + 2.0 ** -134).all()
    rows = dy.shape[0]
    for name, value, terms, more in (("dgamma", dgamma, dy * xh, 2), ("dbeta", dbeta, dy, 0)):
        want, size = terms.sum(0), np.abs(terms).sum(0)
        tol = (rows + 2 + more) * U * size + 2.0 ** -149
        if old is not None:
            want = want + np64(old[name])
            tol = tol + U * (np.abs(want) + tol)
        assert (np.abs(value - want) <= tol).all(), name


BACK_SHAPES = [(1, 16), (3, 48), (40, 512), (17, 528), (50, 1024), (9, 1040), (33, 2048), (7, 2064), (31, 4096),
               (5, 4112), (513, 8192), (3, 8208), (258, 16384), (1, 16368), (4500, 272), (1030, 4096)]


@pytest.mark.parametrize("rows,d", BACK_SHAPES)
@pytest.mark.parametrize("stream", [True, False])
def test_backward(rows, d, stream):
    say(f"layernorm_backward {rows}x{d} {stream}")
    h, dy = normal(1, rows, d, shift=0.5), normal(2, rows, d, std=0.01)
    gamma = normal(3, d, std=0.2, shift=1.0)
    dres = normal(4, rows, d, std=0.01) if stream else None
    _, mean, rstd = fp8bs.layernorm(h, gamma, None, EPS, want_stats=True)
    got = fp8bs.layernorm_backward(dy, h, gamma, mean, rstd, dresidual=dres)
    check_backward(dy, h, gamma, mean, rstd, dres, got)
    # the same bits again, and added to what was there
    again = fp8bs.layernorm_backward(dy, h, gamma, mean, rstd, dresidual=dres)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, again))
    old = {"dgamma": torch.randn(d, device=DEV), "dbeta": torch.randn(d, device=DEV)}
    sums = {k: v.clone() for k, v in old.items()}
    more = fp8bs.layernorm_backward(dy, h, gamma, mean, rstd, dresidual=dres, accumulate=True, **sums)
    assert more[1] is sums["dgamma"]
    check_backward(dy, h, gamma, mean, rstd, dres, more, old)


def test_backward_of_no_rows():
    say("no rows")
    z = torch.zeros(0, 256, dtype=torch.bfloat16, device=DEV)
    f = torch.zeros(0, device=DEV)
    gamma = normal(1, 256)
    dx, dgamma, dbeta = fp8bs.layernorm_backward(z, z, gamma, f, f)
    assert dx.shape == (0, 256) and (dgamma == 0).all() and (dbeta == 0).all()
    ones = torch.ones(256, device=DEV)
    fp8bs.layernorm_backward(z, z, gamma, f, f, dgamma=ones, dbeta=ones.clone(), accumulate=True)
    assert (ones == 1).all()
    q, s = fp8bs.layernorm_quantize_tg128(z, gamma, None, EPS)
    assert q.shape == (0, 256) and s.shape == (0, 2)


def test_backward_rows_do_not_depend_on_the_batch():
    rows, d = 300, 1040
    h, dy, dres = normal(1, rows, d), normal(2, rows, d), normal(3, rows, d)
    gamma = normal(4, d, shift=1.0)
    _, mean, rstd = fp8bs.layernorm(h, gamma, None, EPS, want_stats=True)
    say("backward invariance")
    full = fp8bs.layernorm_backward(dy, h, gamma, mean, rstd, dresidual=dres)[0]
    for a, b in ((0, 1), (299, 300), (10, 50)):
        part = fp8bs.layernorm_backward(dy[a:b], h[a:b], gamma, mean[a:b], rstd[a:b], dresidual=dres[a:b])[0]
        assert torch.equal(part.view(torch.int16), full[a:b].view(torch.int16))


def test_sums_of_many_rows_keep_their_digits():
    """2^17 rows of equal gradients: the sums stay within the rounding of a few hundred additions of partial sums of
    a few hundred rows each."""
    rows, d = 1 << 17, 64
    h = normal(1, 1, d).expand(rows, d).contiguous()
    dy = torch.full((rows, d), 0.1, dtype=torch.bfloat16, device=DEV)
    gamma = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    say("many rows")
    _, mean, rstd = fp8bs.layernorm(h, gamma, None, EPS, want_stats=True)
    _, dgamma, dbeta = fp8bs.layernorm_backward(dy, h, gamma, mean, rstd)
    xh = (np64(h[0]) - float(mean[0])) * float(rstd[0])
    one = float(dy[0, 0])
    assert (np.abs(np64(dbeta) - rows * one) <= 1024 * U * rows * one).all()
    assert (np.abs(np64(dgamma) - rows * one * xh) <= 1024 * U * rows * one * np.abs(xh) + 2.0 ** -100).all()


def test_graph_and_second_stream():
    rows, d = 700, 2064
    x, r, dy = normal(1, rows, d), normal(2, rows, d), normal(3, rows, d)
    gamma, beta = normal(4, d, shift=1.0), normal(5, d)
    h = torch.empty_like(x)

    def step():
        q, s, mean, rstd = fp8bs.layernorm_quantize_tg128(x, gamma, beta, EPS, residual=r, h=h, want_stats=True)
        return (q, s, mean, rstd) + fp8bs.layernorm_backward(dy, h, gamma, mean, rstd, dresidual=dy)

    say("graph")
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (20, 21, 22):
        x.copy_(normal(seed, rows, d))
        dy.copy_(normal(seed + 10, rows, d))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        want = step()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(kept, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(there, want))


@pytest.mark.parametrize("rows,d", [(5, 64), (5, 1040), (3, 2064), (5, 8192), (3, 16384)])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_a_row_that_is_not_finite(rows, d, bad):
    """Its own results are NaN, as the formula has them, and no other row's change."""
    say(f"layernorm {rows}x{d} {bad}")
    x, gamma, beta, dy = normal(1, rows, d), normal(2, d), normal(3, d), normal(4, rows, d)
    good = fp8bs.layernorm_quantize_tg128(x, gamma, beta, EPS, want_y=True, want_stats=True)
    good_dx = fp8bs.layernorm_backward(dy, x, gamma, *good[3:])[0]
    x[1, d // 2] = float(bad)
    got = fp8bs.layernorm_quantize_tg128(x, gamma, beta, EPS, want_y=True, want_stats=True)
    y, rstd = got[2], got[4]
    assert torch.isnan(y[1]).all() and torch.isnan(rstd[1])
    assert torch.equal(got[0][1:2], fp8bs.quantize_tg128(y[1:2].contiguous())[0])
    keep = [r for r in range(rows) if r != 1]
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, good))
    dx, dgamma, dbeta = fp8bs.layernorm_backward(dy, x, gamma, *got[3:])
    assert torch.isnan(dx[1]).all() and torch.equal(dx[keep], good_dx[keep])
    assert torch.isnan(dgamma).all() and torch.isfinite(dbeta).all()
