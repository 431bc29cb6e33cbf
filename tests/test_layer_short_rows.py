"""What the norm reads whole lies inside its tensors: the kernel's own condition (csrc/gdr_piece.h), compiled for the
host, over every piece of small tensors."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_chunked_delta_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "gdr_piece.h"
int main() {
    long long whole = 0, cut = 0, outside = 0, lost = 0;
    const long long gaps[] = {0, 1, 8, 64, -1};  // elements between rows; -1: one row read M times
    for (long long gap : gaps)
        for (int D = 1; D <= 40; ++D)
            for (long long M = 1; M <= 12; ++M) {
                const long long stride = gap < 0 ? 0 : D + gap, last = (M - 1) * stride + D;  // elements [0, last) exist
                for (long long r = 0; r < M; ++r)
                    for (int c = -(int)((r * D) & 7); c < D; c += 8) {
                        const bool exact = c >= 0 && c + 8 <= D;  // lies in the row itself
                        const bool in = gdr::piece_inside(r, c, M, D, stride);
                        const long long at = r * stride + c;
                        if (in && (at < 0 || at + 8 > last)) ++outside;
                        if (exact && gap >= 0 && !in) ++lost;
                        ++(in ? whole : cut);
                    }
            }
    printf("%lld %lld %lld %lld\n", whole, cut, outside, lost);
}
"""


def test_pieces_read_whole_lie_inside_the_tensor(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "pieces.cc", tmp_path / "pieces"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)], check=True, timeout=120)
    whole, cut, outside, lost = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split())
    assert whole > 0 and cut > 0
    assert outside == 0  # read past the tensor's first or last element
    assert lost == 0     # a piece of the row's own eight elements is always read whole


def test_the_kernel_asks_that_condition():
    text = open(os.path.join(CSRC, "gdr_norm.cu")).read()
    assert "gdr::piece_inside(" in text
