"""The expert layer's kernels hold as many choices as the header allows (CPU only): with another limit in the header
their lists grow with it, or the source does not compile."""

import os
import re
import subprocess

import pytest

from fp8_block_scaled_03_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="needs hipcc")


def compiled(limit, tmp_path):
    """The kernels with the header's limit replaced, as clang's front end hands them on."""
    text = open(os.path.join(build.INCLUDE, "fp8bs_layer.h")).read()
    text, n = re.subn(r"(#define FP8BS_MAX_MOE_CHOICES) \d+", rf"\1 {limit}", text)
    assert n == 1
    (tmp_path / "fp8bs_layer.h").write_text(text)
    out = str(tmp_path / "k.ll")
    r = subprocess.run([build.HIPCC, f"-I{tmp_path}", *build.COMMON_FLAGS, "-Xclang", "-disable-llvm-passes", "-x",
                        "hip", "--cuda-device-only", "-emit-llvm", "-S", os.path.join(build.CSRC, "moe_decode.hip"),
                        "-o", out], capture_output=True, text=True)
    return r.returncode, r.stderr, open(out).read() if r.returncode == 0 else ""


@pytest.mark.parametrize("limit", [512, 1024])
def test_lists_hold_what_the_header_allows(limit, tmp_path):
    code, err, text = compiled(limit, tmp_path)
    assert code == 0, err
    assert set(re.findall(r"lists = [^\n]*\[\d+ x \[(\d+) x i16\]\]", text)) == {str(limit)}


@pytest.mark.parametrize("limit", [1000, 65536 + 64])
def test_a_limit_that_the_lists_cannot_hold_does_not_compile(limit, tmp_path):
    code, err, _ = compiled(limit, tmp_path)
    assert code != 0 and "static assertion failed" in err
