"""Numbers that the layer operators ask a device for once (csrc/gdr_once.h): each device has its own."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_chunked_delta_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "gdr_once.h"
gdr::OncePerDevice known;
int main() {
    int asked = 0, bad = 0;
    auto say = [&](int n) { return [&asked, n] { ++asked; return n; }; };
    if (known.get(0, 7, say(76)) != 76 || known.get(1, 7, say(66)) != 66) ++bad;  // another device, another number
    if (known.get(0, 7, say(5)) != 76 || known.get(1, 7, say(5)) != 66 || asked != 2) ++bad;
    if (known.get(2, 7, say(0)) != 7 || known.get(2, 7, say(3)) != 3) ++bad;  // no answer is not kept
    if (known.get(-1, 7, say(3)) != 7 || known.get(64, 7, say(3)) != 7) ++bad;
    std::vector<std::thread> all;
    std::vector<int> got(16);
    for (int i = 0; i < 16; ++i) all.emplace_back([&got, i] { got[i] = known.get(9, 1, [] { return 42; }); });
    for (auto &t : all) t.join();
    for (int v : got) bad += v != 42;
    printf("%d\n", bad);
}
"""


def test_each_device_has_its_number(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "once.cc", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-pthread", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)], check=True, timeout=120)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout == "0\n"


@pytest.mark.parametrize("file", ["gdr_layer.h", "gdr_fp8.cu"])
def test_no_plain_static_number_is_kept(file):
    text = open(os.path.join(CSRC, file)).read()
    assert "static int " not in text and "gdr::OncePerDevice" in text
