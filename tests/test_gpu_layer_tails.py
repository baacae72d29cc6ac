"""Sums over rows where inputs are beyond the caches: every row is in them, those of the first and the last turns too.

Some rows (the first, the last, every 997th) are 2^12 times as large as the others, so that any of them would be missed:
the test says so itself of each.  Sampled columns, against the formula in float64.  U = 2^-24.

Tolerance of dbias of an epilogue: a lane adds ceil(sets / slabs) rows of its slab, two exchanges join four rows, a
wave of the second launch adds ceil(slabs / 16) sums and sixteen are joined; each addition rounds by U of what is
added up.  A term is off by 16 U of the magnitudes that the derivative is made of (as in test_gpu_epilogue.py) and by U
of the product.  Of dgamma and dbeta of a layer norm: a lane adds ceil(sets / grid) rows, at most sixteen rows are
joined, then as above; a term of dgamma is off by 3 U (a difference, a product, the fused one has none of its own)."""

import math

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
WHERE = ["first", "last", "spread"]


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def rows_of(rows, d, seed, std=1.0):
    """bf16 rows from 4096 random ones, each block turned by its number."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    some = (torch.randn(4096, d, generator=g, device=DEV) * std).to(torch.bfloat16)
    out = torch.empty(rows, d, dtype=torch.bfloat16, device=DEV)
    for i, at in enumerate(range(0, rows, 4096)):
        n = min(4096, rows - at)
        out[at:at + n] = some.roll(31 * i, 0)[:n]
    return out


def enlarged(dy, where, turn_rows):
    """Makes some rows large, in place: those of all workgroups' first or last turn and a few beside, or
    single ones throughout.  Their numbers."""
    rows = dy.shape[0]
    n = min(rows, turn_rows + 5)
    at = {"first": np.arange(n), "last": np.arange(rows - n, rows), "spread": np.arange(0, rows, 997)}[where]
    dy[torch.from_numpy(at).to(DEV)] *= 2.0 ** 12
    return at


def columns(n):
    """Sampled columns: the ends, and throughout."""
    return np.unique(np.r_[0:8, n - 8:n, np.linspace(0, n - 1, 112).astype(int)])


def sampled(t, cols):
    return t[:, torch.from_numpy(cols).to(DEV)].cpu().double().numpy()


def check(got, terms, off, additions, at):
    """Sums over the rows within their bound, which would show each of the rows `at` missing in some column."""
    size = np.abs(terms).sum(0)
    tol = additions * U * size + off.sum(0) + 2.0 ** -149
    assert (np.abs(got - terms.sum(0)) <= tol).all()
    assert (np.abs(terms[at]) > 2 * tol).any(1).all()


@pytest.mark.parametrize("rows,n,act", [(8001, 16384, "gelu"), (30001, 4112, "silu"), (140001, 32768, "gelu_tanh"),
                                        (60003, 2064, "relu"), (120003, 1040, "none")])
def test_bias_gradient(rows, n, act):
    sets, nb = -(-rows // 4), -(-n // 128)
    slabs = min((sets + 7) // 8, max(1, 8192 // nb))
    cols = columns(n)
    dout, pre = rows_of(rows, n, 1, std=0.01), rows_of(rows, n, 2)
    assert rows * n * (2 if act == "none" else 4) > 192 << 20  # past the caches
    _, slope, size = oracle.activation_parts(sampled(pre, cols), act)
    for where in WHERE:
        say(f"epilogue_backward {rows}x{n} {act} {where}")
        at = enlarged(dout, where, min(4 * slabs, 512))
        dbias = fp8bs.epilogue_backward_quantize_tg128(dout, None if act == "none" else pre, act)[3]
        d = sampled(dout, cols)
        terms = d * slope
        off = 0.0 * terms if act == "none" else np.abs(d) * 16 * U * size + 2 * U * np.abs(terms) + 2.0 ** -140
        check(dbias.cpu().double().numpy()[cols], terms, off, -(-sets // slabs) + 2 + -(-slabs // 16) + 16, at)
        dout[torch.from_numpy(at).to(DEV)] *= 2.0 ** -12


@pytest.mark.parametrize("rows,d", [(6001, 16384), (50003, 2064), (30007, 4096), (90001, 1040), (200003, 512)])
@pytest.mark.parametrize("stream", [False, True])
def test_weight_and_bias_gradients(rows, d, stream):
    cols = columns(d)
    h, dy = rows_of(rows, d, 1), rows_of(rows, d, 2, std=0.01)
    dres = rows_of(rows, d, 3, std=0.01) if stream else None
    gamma = rows_of(1, d, 4)[0]
    assert rows * d * (6 if stream else 4) > 192 << 20  # past the caches
    _, mean, rstd = fp8bs.layernorm(h, gamma, None, EPS, want_stats=True)
    m, r = (t.cpu().double().numpy()[:, None] for t in (mean, rstd))
    xh = (sampled(h, cols) - m) * r
    for where in WHERE:
        say(f"layernorm_backward {rows}x{d} {stream} {where}")
        at = enlarged(dy, where, 256)
        _, dgamma, dbeta = fp8bs.layernorm_backward(dy, h, gamma, mean, rstd, dresidual=dres)
        terms = sampled(dy, cols)
        # 256 workgroups at most, 128 at least, of at least one row a set
        additions = math.ceil(rows / 128) + 16 + 16 + 16
        check(dbeta.cpu().double().numpy()[cols], terms, 0.0 * terms, additions, at)
        check(dgamma.cpu().double().numpy()[cols], terms * xh, 3 * U * np.abs(terms * xh), additions, at)
        dy[torch.from_numpy(at).to(DEV)] *= 2.0 ** -12
