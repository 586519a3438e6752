"""Rows of a contiguous tensor cut at 16-byte boundaries (csrc/norm.cuh): which vectors end past the tensor.

The norm's kernels take such a vector element by element and load every other one whole.  The rule is compiled for the
host from the kernels' own header, and replayed over every row and vector of small tensors.
"""
import os
import shutil
import subprocess

import pytest

from chunked_gated_delta_prepare_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "norm.cuh"

// Rows of D elements, `per` of them in 16 bytes: prints the first vector that the rule takes wrongly, and their number.
int main() {
    long wrong = 0, past = 0;
    for (int per = 4; per <= 8; per += 4)
        for (int D = 1; D <= 70; ++D)
            for (int64_t rows = 1; rows <= 40; ++rows)
                for (int64_t row = 0; row < rows; ++row) {
                    const int shift = (int)(row * D % per);
                    for (int c = -shift; c < D; c += 8) {
                        const bool ends = row * D + c + 8 > rows * D;
                        past += ends;
                        if (gdr::layer::ends_past(row, rows, c, D) != ends && wrong++ == 0)
                            std::printf("16 / %d bytes, row %ld of %ld, D %d, column %d\n", per, (long)row, (long)rows, D, c);
                    }
                }
    // a tensor near the limits: no overflow, and only its last rows count
    const int64_t rows = (1 << 30) - 1;
    for (int64_t row : {int64_t{0}, rows / 2, rows - 9, rows - 8, rows - 2, rows - 1})
        for (int D : {1, 5, 32767})
            for (int c : {0, D - 1})
                wrong += gdr::layer::ends_past(row, rows, c, D) != (row * D + c + 8 > rows * D);
    std::printf("%ld wrong of %ld\n", wrong, past);
    return wrong != 0 || past == 0;
}
"""


@pytest.mark.skipif(not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"), reason="needs nvcc")
def test_vectors_that_end_past_the_tensor(tmp_path):
    source, program = tmp_path / "replay.cu", tmp_path / "replay"
    source.write_text(PROGRAM)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", str(program),
                    str(source)], check=True, capture_output=True, text=True)
    ran = subprocess.run([str(program)], capture_output=True, text=True)
    assert ran.returncode == 0, ran.stdout
