"""Workspace sizes of include/fp8bs_layer.h: 0 for what the call refuses, never less than nothing, and growing with the
sizes (CPU only)."""

import pytest

from fp8_block_scaled_03_amd import binding

MOST = 65536  # tensors of a call


@pytest.mark.parametrize("n", [-1, -2 ** 31, MOST + 1, 2 ** 31 - 96, 2 ** 31 - 95, 2 ** 31 - 1])
def test_no_workspace_for_a_list_that_is_refused(n):
    assert binding.load_library().fp8bs_grad_norm_workspace(n) == 0


def test_a_longer_list_needs_no_less():
    f = binding.load_library().fp8bs_grad_norm_workspace
    sizes = [f(n) for n in range(MOST + 1)]
    assert sizes[0] >= 8 and all(b >= a for a, b in zip(sizes, sizes[1:])) and all(s % 8 == 0 for s in sizes)


@pytest.mark.parametrize("name", ["fp8bs_layernorm_backward_workspace", "fp8bs_epilogue_backward_workspace"])
@pytest.mark.parametrize("rows,cols", [(2 ** 63 - 1, 64), (64, 2 ** 63 - 16), (2 ** 62, 2 ** 62), (-2 ** 63, 16),
                                       (2 ** 30 + 1, 16), (0, 0)])
def test_no_workspace_for_sizes_that_are_refused(name, rows, cols):
    assert getattr(binding.load_library(), name)(rows, cols) == 0


def test_the_largest_sizes_have_a_workspace():
    lib = binding.load_library()
    assert 0 < lib.fp8bs_layernorm_backward_workspace(2 ** 30, 16384) < 2 ** 32
    assert 0 < lib.fp8bs_epilogue_backward_workspace(2 ** 30, 2 ** 30) < 2 ** 40
    assert 0 < lib.fp8bs_moe_decode_b128_workspace(512, 1, 1024, 32768, 32768) < 2 ** 32
