"""The digits of an epilogue's activation below bf16's: K = 0, the bias runs over every finite bf16 value, and the
residual is minus the rounded result, so that the sum that is rounded is what the leading bits leave.

Tolerance: the activation itself as the header has it, E = 2^-15 |act| + 2^-118; the fp32 sum with the residual
rounds by 2^-24 of itself, the result by 2^-8 of itself or half the smallest step, 2^-134."""

import numpy as np
import pytest
import torch

import oracle
import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

ACTS = ["gelu", "gelu_tanh", "silu"]


def every_bf16():
    """All finite bf16 values."""
    bits = torch.arange(65536, dtype=torch.int32)
    return bits[(bits & 0x7F80) != 0x7F80].to(torch.int16).view(torch.bfloat16)


def exact(act):
    """act(z) of every z in 64 bits, and minus its bf16 rounding (infinities and zeros' signs left out)."""
    want = oracle.activation_parts(every_bf16().double().numpy(), act)[0]
    return want, -torch.from_numpy(want).to(torch.bfloat16)


def allowed(act64, residual):
    off = 2.0 ** -15 * np.abs(act64) + 2.0 ** -118
    left = np.abs(act64 + residual.double().numpy()) + off
    return off + 2.0 ** -24 * left + 2.0 ** -8 * (1 + 2.0 ** -24) * left + 2.0 ** -134


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 70])
def test_low_digits_of_every_value(act, M):
    z = every_bf16()
    N = z.numel()
    act64, residual = exact(act)
    empty = (torch.zeros(M, 0, dtype=torch.uint8, device=DEV), torch.zeros(M, 0, device=DEV),
             torch.zeros(N, 0, dtype=torch.uint8, device=DEV), torch.zeros(-(-N // 128), 0, device=DEV))
    say(f"digits {act} {M}")
    out = fp8bs.gemm_tg128_nt_epilogue(*empty, bias=z.to(DEV), activation=act,
                                       residual=residual.to(DEV).expand(M, N).contiguous())
    got = out.cpu().double().numpy()
    bad = np.abs(got - (act64 + residual.double().numpy())) > allowed(act64, residual)
    assert not bad.any(), (act, z[torch.from_numpy(bad[0])][:8])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("error", [2.0 ** -14, -2.0 ** -14])
def test_an_error_of_twice_what_is_stated_is_seen(act, error):
    """The same check of values that are off by 2^-14 (on the CPU): it fails at nearly every one."""
    act64, residual = exact(act)
    wrong = (act64 * (1 + error)).astype(np.float32) + residual.float().numpy()
    got = torch.from_numpy(wrong).to(torch.bfloat16).double().numpy()
    over = np.abs(got - (act64 + residual.double().numpy())) > allowed(act64, residual)
    curved = (np.abs(act64) > 2.0 ** -100) & np.isfinite(residual.double().numpy())
    assert over[curved].mean() > 0.9
