"""Arguments that the headers let be one another (the residual that is the result, the sum that is the residual) are
not promised to the compiler to be apart: the kernels' parameters as clang's front end hands them on (CPU only)."""

import os
import re
import subprocess

import pytest

from fp8_block_scaled_03_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="needs hipcc")


def kernels(source, tmp_path):
    """{kernel's symbol: its parameters} of one source, before any optimisation."""
    out = str(tmp_path / "k.ll")
    r = subprocess.run([build.HIPCC, *build.COMMON_FLAGS, "-Xclang", "-disable-llvm-passes", "-x", "hip",
                        "--cuda-device-only", "-emit-llvm", "-S", os.path.join(build.CSRC, source), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return dict(re.findall(r"^define[^@\n]*amdgpu_kernel[^@\n]*@(\w+)\((.*)\) #\d+ ", open(out).read(), re.M))


def test_the_residual_may_be_the_products_result(tmp_path):
    with_epilogue = plain = 0
    for name, parameters in kernels("gemm_g128.hip", tmp_path).items():
        result = re.findall(r"ptr addrspace\(1\)[^,]*", parameters)[-1]
        if '::Epilogue"' in parameters:
            with_epilogue += 1
            assert "noalias" not in result, name
        else:
            plain += 1
            assert "noalias" in result, name  # nothing else of such a call may be the result
    assert with_epilogue >= 10 and plain >= 10


@pytest.mark.parametrize("source,kernel", [("layernorm.hip", "layernorm_kernel"), ("moe_decode.hip", "moe_join_kernel"),
                                           ("moe_decode.hip", "moe_token_kernel")])
def test_the_residual_may_be_the_sum(source, kernel, tmp_path):
    found = [p for name, p in kernels(source, tmp_path).items() if kernel in name]
    assert found and not any("noalias" in p for p in found)


def test_a_clipped_tensor_may_be_the_gradient(tmp_path):
    """The tensors' addresses are a table's entries; only the norm and the partial sums, which overlap none of them
    (refused otherwise), are parameters of their own."""
    found = [p for name, p in kernels("gradnorm.hip", tmp_path).items() if "clip_kernel" in name]
    assert found and all(p.startswith('ptr addrspace(4) noundef byref(%"struct.fp8bs::GradTable")') for p in found)
