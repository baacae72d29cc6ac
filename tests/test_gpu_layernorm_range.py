"""The range of layer norm's fp32 sums as the header states it: rows whose squared deviations add up to just below
2^128, and rows of tiny deviations with eps = 0, are within the ordinary bounds."""

import math

import pytest
import torch

import test_gpu_layernorm as norm
from gpu_util import DEV

pytestmark = pytest.mark.gpu


def rows_of(size, d, shift=0.0):
    """Rows of deviations of either sign, between half of `size` and all of it."""
    g = torch.Generator().manual_seed(d)
    sign = torch.randint(0, 2, (4, d), generator=g) * 2.0 - 1.0
    part = 0.5 + 0.5 * torch.rand(4, d, generator=g)
    return ((sign * part + shift) * size).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("d", [16, 512, 2064, 4096, 16384])
def test_large_deviations(d):
    size = 2.0 ** math.floor((128 - math.log2(d)) / 2 - 0.25)  # d size^2 <= 2^127.5
    gamma, beta = norm.normal(1, d, std=0.1, shift=1.0), norm.normal(2, d, std=0.2)
    norm.run_forward(rows_of(size, d), gamma, beta, None, label="large")
    half = rows_of(size / 2, d)
    norm.run_forward(half, gamma, beta, half.clone(), label="large with residual")


@pytest.mark.parametrize("d", [16, 512, 2064, 4096, 16384])
def test_tiny_deviations_without_eps(d):
    gamma, beta = norm.normal(1, d, std=0.1, shift=1.0), norm.normal(2, d, std=0.2)
    norm.run_forward(rows_of(2.0 ** -61, d), gamma, beta, None, eps=0.0, label="tiny")
    norm.run_forward(rows_of(2.0 ** -61, d, shift=1.0), gamma, beta, None, eps=0.0, label="tiny, shifted")
