"""Pins of the oracle's activations and layer norm: closed forms, torch in fp64, differences."""

import math

import numpy as np
import pytest
import torch

import oracle

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
TORCH = {"none": lambda z: z, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"), "silu": torch.nn.functional.silu}


@pytest.mark.parametrize("act", ACTS)
def test_activation_is_torchs(act):
    z = np.concatenate([np.linspace(-30, 30, 6001), [0.0, 1e-30, -1e-30]])
    got = oracle.activation_parts(z, act)[0]
    want = TORCH[act](torch.from_numpy(z)).numpy()
    assert np.abs(got - want).max() < 1e-13


@pytest.mark.parametrize("act", ACTS)
def test_slope_against_differences(act):
    z = np.linspace(-8, 8, 4001) + 1e-4
    h = 1e-5
    diff = (oracle.activation_parts(z + h, act)[0] - oracle.activation_parts(z - h, act)[0]) / (2 * h)
    value, slope, size = oracle.activation_parts(z, act)
    assert np.abs(diff - slope).max() < 1e-8 and (size >= np.abs(slope) - 1e-15).all()


@pytest.mark.parametrize("act", ACTS)
def test_far_values_are_finite_and_exact(act):
    with np.errstate(over="ignore", invalid="ignore"):
        value, slope, _ = oracle.activation_parts(np.array([3e38, 200.0, -200.0, -3e38]), act)
    low = 0.0 if act != "none" else None
    assert value[0] == 3e38 and value[1] == 200.0 and slope[0] == 1.0 and abs(slope[1] - 1.0) < 1e-15
    if low is not None:
        assert abs(value[2]) < 1e-80 and abs(value[3]) < 1e-80 and abs(slope[2]) < 1e-80 and abs(slope[3]) < 1e-80


def test_gelu_closed_forms():
    value, slope, _ = oracle.activation_parts(np.array([0.0, 1.0, -1.0]), "gelu")
    phi1 = 0.5 * (1 + math.erf(1 / math.sqrt(2)))
    assert value[0] == 0.0 and abs(value[1] - phi1) < 1e-15 and abs(value[2] + (1 - phi1)) < 1e-15
    dens = math.exp(-0.5) / math.sqrt(2 * math.pi)
    assert slope[0] == 0.5 and abs(slope[1] - (phi1 + dens)) < 1e-15 and abs(slope[2] - (1 - phi1 - dens)) < 1e-15


def test_layernorm_is_torchs_and_its_gradient_that_of_differences():
    rng = np.random.default_rng(0)
    h, gamma, beta = rng.normal(size=(5, 48)) + 2, rng.normal(size=48), rng.normal(size=48)
    dy = rng.normal(size=(5, 48))
    mean, rstd, y = oracle.layernorm(h, gamma, beta, 1e-3)
    t = [torch.from_numpy(v).requires_grad_() for v in (h, gamma, beta)]
    want = torch.nn.functional.layer_norm(t[0], (48,), t[1], t[2], 1e-3)
    assert np.abs(want.detach().numpy() - y).max() < 1e-13
    want.backward(torch.from_numpy(dy))
    dx, dgamma, dbeta = oracle.layernorm_grad(dy, h, gamma, mean, rstd)
    for got, leaf in ((dx, t[0]), (dgamma.sum(0), t[1]), (dbeta.sum(0), t[2])):
        assert np.abs(got - leaf.grad.numpy()).max() < 1e-12
    step = 1e-5
    for i, j in ((0, 0), (2, 17), (4, 47)):
        up, down = h.copy(), h.copy()
        up[i, j] += step
        down[i, j] -= step
        diff = ((oracle.layernorm(up, gamma, beta, 1e-3)[2] - oracle.layernorm(down, gamma, beta, 1e-3)[2]) * dy).sum()
        assert abs(diff / (2 * step) - dx[i, j]) < 1e-7
