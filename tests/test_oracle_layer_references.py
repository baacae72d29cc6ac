"""What the GPU tests of layer norm hold the kernels to is the oracle's layer norm, which is held to differences: their
formulas are the same, their checks pass on the oracle's results and fail on planted mistakes (CPU only)."""

import numpy as np
import pytest
import torch

import oracle
import test_gpu_layernorm as norm

EPS = 1e-5


def rows(seed, *shape, std=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + shift).to(torch.bfloat16)


def host(t):
    return t.double().numpy()


@pytest.mark.parametrize("R,d", [(1, 16), (7, 272), (5, 2064)])
@pytest.mark.parametrize("with_beta", [True, False])
def test_the_forward_reference(R, d, with_beta):
    h, gamma = rows(1, R, d, shift=0.3), rows(2, d, std=0.1, shift=1.0)
    beta = rows(3, d) if with_beta else None
    mean, rstd, y, off = norm.reference(h, gamma, beta, EPS)
    want = oracle.layernorm(host(h), host(gamma), None if beta is None else host(beta), EPS)
    for got, ref in zip((mean, rstd, y), want):
        assert got.shape == ref.shape and np.abs(got - ref).max() <= 1e-13 * np.abs(ref).max()
    assert (off > 0).all() and (off <= 64 * norm.U * (np.abs(y) + np.abs(y).max())).all()


def results(R, d, stream):
    """Inputs, and the oracle's gradients rounded as the kernels round theirs."""
    h, dy, gamma = rows(1, R, d, shift=0.5), rows(2, R, d, std=0.01), rows(3, d, std=0.2, shift=1.0)
    dres = rows(4, R, d, std=0.01) if stream else None
    mean, rstd, _ = oracle.layernorm(host(h), host(gamma), None, EPS)
    mean, rstd = (torch.from_numpy(v).float() for v in (mean, rstd))
    dx, dg, db = oracle.layernorm_grad(host(dy), host(h), host(gamma), host(mean), host(rstd))
    if stream:
        dx = dx + host(dres)
    got = (torch.from_numpy(dx).to(torch.bfloat16), torch.from_numpy(dg.sum(0)).float(),
           torch.from_numpy(db.sum(0)).float())
    return (dy, h, gamma, mean, rstd, dres), got


@pytest.mark.parametrize("R,d", [(1, 16), (7, 272), (40, 1040)])
@pytest.mark.parametrize("stream", [True, False])
def test_the_gradients_check(R, d, stream):
    inputs, got = results(R, d, stream)
    norm.check_backward(*inputs, got)


@pytest.mark.parametrize("stream", [True, False])
def test_the_gradients_check_sees_mistakes(stream):
    inputs, (dx, dgamma, dbeta) = results(40, 1040, stream)
    dy, h, gamma, mean, rstd, dres = inputs
    xh = (host(h) - host(mean)[:, None]) * host(rstd)[:, None]
    g = host(dy) * host(gamma)
    one_more = torch.from_numpy(host(dx) + host(rstd)[:, None] * g.mean(1, keepdims=True)).to(torch.bfloat16)
    unweighted = torch.from_numpy(host(dx) / host(gamma)).to(torch.bfloat16)
    for wrong in ((one_more, dgamma, dbeta), (unweighted, dgamma, dbeta),
                  (dx, dgamma - torch.from_numpy(host(dy)[-1] * xh[-1]).float(), dbeta),  # without the last row
                  (dx, dgamma, dbeta - dy[-1].float()), (dx, dbeta, dgamma)):
        with pytest.raises(AssertionError):
            norm.check_backward(*inputs, wrong)
