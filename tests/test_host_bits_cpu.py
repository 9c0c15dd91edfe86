"""The host side's integer helpers over the whole range of a cache's page size (up to
2^31 - 1 slots in one page), compiled on their own and ended if they do not return."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "post_weight_quantization_22_amd", "csrc")

PROGRAM = r"""
#include "bits.hpp"
#include <cstdio>
int main() {
  const long long some[] = {1, 2, 3, 16, 17, 64, 4095, 4096, 1 << 29, (1 << 30) - 1, 1 << 30,
                            (1LL << 30) + 1, (1LL << 31) - 1};
  for (long long v : some) std::printf("%lld %d %d\n", v, gptq::log2_at_least(v), gptq::log2_exact(v));
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_logarithms_end_and_are_right(tmp_path):
    (tmp_path / "t.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "t")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(tmp_path / "t.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=10).stdout
    lines = [tuple(map(int, l.split())) for l in out.splitlines()]
    assert len(lines) == 13
    for v, at_least, exact in lines:
        assert at_least == (v - 1).bit_length()
        assert exact == (v.bit_length() - 1 if v & (v - 1) == 0 else -1)
