"""The copies of rows that begin inside a 16-byte vector: none takes a byte behind the tensor's end, all live elements come
along.  The kernels' own arithmetic, compiled for the host; needs no GPU."""

import subprocess

from gated_delta_rule_38_gb300 import build as gbuild

SOURCE = r"""
#include "rowclip.h"
#include <cstdio>
#include <initializer_list>
// A row's vectors of `per` elements are those of the tensor: the first holds the row's first element, (row D) mod 8 elements
// (whole 16-bit vectors, for both types) before it in memory.
int main() {
    for (int elem : {2, 4})
        for (int D = 1; D < 16; ++D)
            for (int rows = 1; rows < 24; ++rows) {
                if (D % 8 == 0) continue;
                const int per = 16 / elem;
                for (int row = 0; row < rows; ++row) {
                    const int shift = row * D % 8;
                    for (int c = -shift; c < D; c += per) {
                        if (c + per <= 0) continue;
                        const long long first = (long long)row * D + c, left = ((long long)rows * D - first) * elem;
                        const int n = gdr::rownorm::bytes_to_copy(row, rows, left);
                        const int live = (D - c < per ? D - c : per) * elem;  // up to the row's last element
                        if (n < 0 || n > left || n < live || n > 16) {
                            std::printf("elem %d D %d rows %d row %d column %d: %d bytes of %lld\n", elem, D, rows, row, c, n, left);
                            return 1;
                        }
                    }
                }
            }
    return 0;
}
"""


def test_copies_end_with_the_tensor(tmp_path):
    src, exe = tmp_path / "clip.cpp", tmp_path / "clip"
    src.write_text(SOURCE)
    r = subprocess.run(["g++", "-std=c++17", "-I" + gbuild.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
