"""The layer norm's gradient of a row whose incoming gradient is infinite in one column: every result is the formula's,
an infinity or a NaN, wherever that column is and whatever the row's length leaves of the last piece."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
EPS = 1e-5


def normal(seed, *shape, std=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + shift).to(torch.bfloat16).to(DEV)


def host(t):
    return t.cpu().double().numpy()


@pytest.mark.parametrize("d", [16, 64, 496, 512, 528, 1040, 2064, 4096, 4112, 8208, 16368])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("stream", [False, True])
def test_an_infinite_gradient(d, bad, stream):
    rows = 5
    h, dy, gamma = normal(1, rows, d), normal(2, rows, d), normal(3, d, std=0.1, shift=1.0)
    dres = normal(4, rows, d) if stream else None
    _, mean, rstd = fp8bs.layernorm(h, gamma, None, EPS, want_stats=True)
    say(f"layernorm_backward {rows}x{d} {bad} {stream}")
    good = fp8bs.layernorm_backward(dy, h, gamma, mean, rstd, dresidual=dres)
    for col in (0, d // 2, d - 1):
        off = dy.clone()
        off[2, col] = bad
        dx, dgamma, dbeta = fp8bs.layernorm_backward(off, h, gamma, mean, rstd, dresidual=dres)
        with np.errstate(invalid="ignore"):
            want = oracle.layernorm_grad(host(off), host(h), host(gamma), host(mean), host(rstd))[0][2]
        assert not np.isfinite(want).any() and not np.isnan(want).all()
        np.testing.assert_array_equal(host(dx)[2], want)  # (NaN where the formula's is)
        keep = [r for r in range(rows) if r != 2]
        assert torch.equal(dx[keep], good[0][keep])
        there = [c for c in range(d) if c != col]
        assert torch.equal(dgamma[there], good[1][there]) and torch.equal(dbeta[there], good[2][there])
        assert torch.isinf(dgamma[col]) and float(dbeta[col]) == bad
