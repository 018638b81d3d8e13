"""A launch that the runtime refuses: the operators report it and leave no error
behind for the library's next launch to find.  The runtime refuses the block of 2000
threads on the host: nothing reaches the GPU."""
import os
import subprocess

import pytest

from block_scaled_grouped_gb300 import build as bsgg_build

pytestmark = pytest.mark.gpu

SOURCE = """
#include <cstdio>
#include "bsgg_ops.cuh"
__global__ void nothing(int) {}
int main() {
  const bsgg::LaunchConfig c(dim3(1), 2000, 0, nullptr);
  const bsgg_status st = bsgg::launch_kernel(c, nothing, 1);
  std::printf("%d %d", static_cast<int>(st), static_cast<int>(cudaGetLastError()));
}
"""


def test_refused_launch_leaves_no_error(tmp_path):
    src, exe = tmp_path / "launch.cu", tmp_path / "launch"
    src.write_text(SOURCE)
    subprocess.run([bsgg_build._nvcc(), *bsgg_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", bsgg_build.INCLUDE,
                    "-I", bsgg_build.CSRC, "-cudart", "static", "-o", os.fspath(exe), os.fspath(src)], check=True,
                   capture_output=True)
    out = subprocess.run([os.fspath(exe)], check=True, capture_output=True, text=True).stdout
    assert out == "3 0"                                 # BSGG_ERR_CUDA; no error left
