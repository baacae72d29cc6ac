"""Layer norm and the epilogue's gradient on inputs beyond the caches, for every way in which a row is held and every
activation: rows are the bits that they have in a small call, which the other tests hold to float64."""

import pytest
import torch

import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
EPS = 1e-5
BEYOND = 192 << 20  # bytes of inputs


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


def equal(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def places(rows):
    return [slice(0, 37), slice(rows // 2 - 20, rows // 2 + 21), slice(rows - 37, rows)]


@pytest.mark.parametrize("d", [256, 272, 512, 528, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 16384, 16368])
@pytest.mark.parametrize("with_residual", [True, False])
def test_layernorm(d, with_residual):
    rows = BEYOND // ((4 if with_residual else 2) * d) + 13
    say(f"layernorm {rows}x{d} {with_residual}")
    x = rows_of(rows, d, 1)
    r = rows_of(rows, d, 2) if with_residual else None
    gamma, beta = rows_of(1, d, 3)[0], rows_of(1, d, 4)[0]

    def call(at):
        part = x[at].clone(), None if r is None else r[at].clone()
        h = torch.empty_like(part[0]) if with_residual else None
        out = fp8bs.layernorm_quantize_tg128(part[0], gamma, beta, EPS, residual=part[1], h=h, want_y=True,
                                             want_stats=True)
        return out + ((h,) if with_residual else ())

    whole = call(slice(0, rows))
    for at in places(rows):
        assert all(equal(a, b[at]) for a, b in zip(call(at), whole)), at
    y = fp8bs.layernorm(x, gamma, beta, EPS, residual=None if r is None else r.clone())
    assert equal(y, whole[2])


@pytest.mark.parametrize("n", [2048, 2064, 144])
@pytest.mark.parametrize("act", list(fp8bs.ACTIVATIONS))
def test_epilogue_backward(n, act):
    rows = BEYOND // ((2 if act == "none" else 4) * n) + 13
    say(f"epilogue_backward {rows}x{n} {act}")
    dout = rows_of(rows, n, 1, std=0.01)
    pre = None if act == "none" else rows_of(rows, n, 2, std=1.7)
    whole = fp8bs.epilogue_backward_quantize_tg128(dout, pre, act)
    for at in places(rows):
        one = fp8bs.epilogue_backward_quantize_tg128(dout[at].clone(), None if pre is None else pre[at].clone(), act)
        assert all(equal(a, b[at]) for a, b in zip(one[:3], whole[:3])), at
    again = fp8bs.epilogue_backward_quantize_tg128(dout, pre, act)
    assert all(equal(a, b) for a, b in zip(again, whole))


@pytest.mark.parametrize("d", [256, 512, 528, 1024, 2048, 2064, 4112, 8192, 8208, 16384])
@pytest.mark.parametrize("stream", [True, False])
def test_layernorm_backward(d, stream):
    rows = BEYOND // ((6 if stream else 4) * d) + 13
    say(f"layernorm_backward {rows}x{d} {stream}")
    h, dy = rows_of(rows, d, 1), rows_of(rows, d, 2, std=0.01)
    dres = rows_of(rows, d, 3, std=0.01) if stream else None
    gamma = rows_of(1, d, 4)[0]
    _, mean, rstd = fp8bs.layernorm(h, gamma, None, EPS, want_stats=True)
    whole = fp8bs.layernorm_backward(dy, h, gamma, mean, rstd, dresidual=dres)
    for at in places(rows):
        one = fp8bs.layernorm_backward(dy[at].clone(), h[at].clone(), gamma, mean[at].clone(), rstd[at].clone(),
                                       dresidual=None if dres is None else dres[at].clone())
        assert equal(one[0], whole[0][at]), at
    again = fp8bs.layernorm_backward(dy, h, gamma, mean, rstd, dresidual=dres)
    assert all(equal(a, b) for a, b in zip(again, whole))
