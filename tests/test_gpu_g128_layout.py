"""The 128-value forms where addresses are unusual: tensors that start 16 bytes into a line, and tensors
whose byte or element offsets pass 32 bits.  Each result is the same call's on an ordinary copy, bit for bit."""

import pytest
import torch

import fp8_block_scaled_03_amd as fp8bs

from gpu_util import DEV, i32_dev, say

pytestmark = pytest.mark.gpu


def normal(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).bfloat16()


def code_bytes(seed, *shape):
    """Finite codes of both signs."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
    return torch.where((c & 0x7F) == 0x7F, c - 1, c)


def scale_values(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.rand(*shape, generator=g, device=DEV) + 0.5


def moved(t, by=None):
    """A copy of t that starts 16 bytes (scales and offsets: 4) behind an allocation's start, with marked
    bytes around it, and a function that checks these."""
    size = t.element_size()
    by = (16 if size != 4 or by == 16 else 4) // size
    room = torch.full((t.numel() + by + 64,), 77, dtype=t.dtype, device=DEV)
    view = room[by:by + t.numel()].view(t.shape)
    view.copy_(t)

    def check():
        assert (room[:by] == 77).all() and (room[by + t.numel():] == 77).all()
    return view, check


def same(x, y):
    return torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def all_same(got, want):
    for x, y in zip(got, want):
        assert same(x, y)


@pytest.mark.parametrize("rows,cols", [(16, 128), (130, 272), (64, 1024)])
def test_quantizers_on_moved_tensors(rows, cols):
    say(f"moved quantizers {rows}x{cols}")
    x = normal(1, rows, cols)
    want = fp8bs.quantize_tg128(x)
    out = [moved(torch.zeros_like(t)) for t in want]
    fp8bs.quantize_tg128(moved(x)[0], out[0][0], out[1][0])
    all_same([o[0] for o in out], want)
    rows16 = rows // 16 * 16
    w = normal(2, 2, rows16, cols)
    want = fp8bs.quantize_b128(w, transposed=True)
    outs = [moved(torch.zeros_like(t)) for t in want]
    fp8bs.quantize_b128(moved(w)[0], outs[0][0], outs[1][0], True, outs[2][0], outs[3][0])
    all_same([o[0] for o in outs], want)
    for _, check in out + outs:
        check()


@pytest.mark.parametrize("rows,d", [(3, 16), (130, 272), (64, 512)])
def test_swiglu_on_moved_tensors(rows, d):
    say(f"moved swiglu {rows}x{d}")
    gu, dy = normal(3, rows, 2 * d), normal(4, rows, d)
    want = fp8bs.swiglu_quantize_tg128(gu, want_y=True)
    outs = [moved(torch.zeros_like(t)) for t in want]
    fp8bs.swiglu_quantize_tg128(moved(gu)[0], outs[0][0], outs[1][0], outs[2][0])
    all_same([o[0] for o in outs], want)
    want = fp8bs.swiglu_backward_quantize_tg128(gu, dy, want_y=True)
    back = [moved(torch.zeros_like(t)) for t in want]
    fp8bs.swiglu_backward_quantize_tg128(moved(gu)[0], moved(dy)[0], *[o[0] for o in back])
    all_same([o[0] for o in back], want)
    for _, check in outs + back:
        check()


@pytest.mark.parametrize("M,N,K", [(5, 272, 400), (50, 1040, 272), (700, 528, 400), (3500, 4112, 144),
                                   (3500, 4160, 144)])
def test_products_on_moved_tensors(M, N, K):
    say(f"moved products {M}x{N}x{K}")
    a, sa = code_bytes(5, M, K), scale_values(6, M, -(-K // 128))
    bt, sbt = code_bytes(7, 3, N, K), scale_values(8, 3, -(-N // 128), -(-K // 128))
    off = i32_dev([0, M // 3, M // 3, M])
    want = fp8bs.gemm_tg128_nt(a, sa, bt[0], sbt[0])
    out, check = moved(torch.zeros_like(want))
    ma, msa, mbt, msbt, moff = (moved(t)[0] for t in (a, sa, bt, sbt, off))
    fp8bs.gemm_tg128_nt(ma, msa, mbt[0], msbt[0], out)
    assert same(out, want)
    want = fp8bs.grouped_gemm_tg128_nt(a, sa, bt, sbt, off)
    fp8bs.grouped_gemm_tg128_nt(ma, msa, mbt, msbt, moff, out)
    assert same(out, want)
    check()
    dy, x = normal(9, M, N), normal(10, M, K)
    want = fp8bs.grouped_wgrad(dy, x, off)
    dw, check = moved(torch.zeros_like(want), 16)
    fp8bs.grouped_wgrad(moved(dy)[0], moved(x)[0], moff, dw)
    assert same(dw, want)
    check()


def test_k_zero_in_ranges_leaves_the_other_rows():
    say("grouped K=0")
    out = torch.full((40, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    z = torch.zeros
    fp8bs.grouped_gemm_tg128_nt(z(40, 0, dtype=torch.uint8, device=DEV), z(40, 0, device=DEV),
                                z(2, 64, 0, dtype=torch.uint8, device=DEV), z(2, 1, 0, device=DEV),
                                i32_dev([3, 10, 37]), out)
    assert (out[3:37].view(torch.int16) == 0).all() and (out[:3] == 3.0).all() and (out[37:] == 3.0).all()


# ---- offsets past 32 bits ------------------------------------------------------------------
def test_rows_past_32_bits():
    """4.4e9 codes: the last rows give what they give alone, from a dense call and from ranges."""
    M, N, K = 530016, 48, 8208
    say(f"gemm {M}x{N}x{K}")
    a = torch.empty(M, K, dtype=torch.uint8, device=DEV)
    tail = code_bytes(11, 700, K)
    a[:M - 700] = 0x38
    a[M - 700:] = tail
    sa = torch.ones(M, 65, device=DEV)
    sa[M - 700:] = scale_values(12, 700, 65)
    bt, sbt = code_bytes(13, 2, N, K), scale_values(14, 2, 1, 65)
    want = fp8bs.gemm_tg128_nt(tail, sa[M - 700:].clone(), bt[1], sbt[1])
    c = fp8bs.gemm_tg128_nt(a, sa, bt[1], sbt[1])
    assert same(c[M - 700:], want)
    c = fp8bs.grouped_gemm_tg128_nt(a, sa, bt, sbt, i32_dev([0, M - 700, M]))
    assert same(c[M - 700:], want)


def test_weights_and_gradients_past_32_bits():
    """The last of 40 weights of 1.3e8 codes (5.4e9 in all), and its fp32 gradient 21e9 bytes in."""
    G, N, K = 40, 8192, 16400
    say(f"grouped {G}x{N}x{K}")
    bt = torch.full((G, N, K), 0x38, dtype=torch.uint8, device=DEV)
    bt[G - 1] = code_bytes(15, N, K)
    sbt = scale_values(16, G, 64, 129)
    M = 90
    a, sa = code_bytes(17, M, K), scale_values(18, M, 129)
    off = torch.arange(G + 1, dtype=torch.int32)
    off[G] = M
    c = fp8bs.grouped_gemm_tg128_nt(a, sa, bt, sbt, off.to(DEV))
    r = slice(G - 1, M)
    assert same(c[r], fp8bs.gemm_tg128_nt(a[r].clone(), sa[r].clone(), bt[G - 1].clone(), sbt[G - 1].clone()))
    del bt, c
    dy, x = normal(19, M, N), normal(20, M, K)
    dw = torch.full((G, N, K), 2.0, device=DEV)
    fp8bs.grouped_wgrad(dy, x, off.to(DEV), dw, accumulate=True)
    one = torch.full((1, N, K), 2.0, device=DEV)
    fp8bs.grouped_wgrad(dy[r].clone(), x[r].clone(), i32_dev([0, M - G + 1]), one, accumulate=True)
    assert same(dw[G - 1], one[0])


def test_quantizers_past_32_bits():
    rows, cols = 300001, 16416
    say(f"quantize {rows}x{cols}")
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[rows - 130:] = normal(21, 130, cols)
    want = fp8bs.quantize_tg128(x[rows - 130:].clone())
    q, s = fp8bs.quantize_tg128(x)
    all_same((q[rows - 130:], s[rows - 130:]), want)
    want = fp8bs.swiglu_quantize_tg128(x[rows - 130:].clone(), want_y=True)
    q, s, y = fp8bs.swiglu_quantize_tg128(x, want_y=True)
    all_same((q[rows - 130:], s[rows - 130:], y[rows - 130:]), want)
    dy = torch.ones(rows, cols // 2, dtype=torch.bfloat16, device=DEV)
    want = fp8bs.swiglu_backward_quantize_tg128(x[rows - 130:].clone(), dy[:130].clone())
    got = fp8bs.swiglu_backward_quantize_tg128(x, dy)
    all_same([t[rows - 130:] for t in got], want)
    del q, s, y, dy, got
    w = x[:rows // 16 * 16].view(2, rows // 16 * 8, cols)
    got = fp8bs.quantize_b128(w, transposed=True)
    # block rows counted from the matrix's start, so the last ones start at a multiple of 128
    first = w.shape[1] // 128 * 128
    want = fp8bs.quantize_b128(w[1, first:].clone(), transposed=True)
    assert same(got[0][1, first:], want[0]) and same(got[1][1, first // 128:], want[1])
    assert same(got[2][1, :, first:], want[2]) and same(got[3][1, :, first // 128:], want[3])
