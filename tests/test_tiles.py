"""The tiles that workgroups take (csrc/tiles.h, compiled for the host): each tile of a product goes to one workgroup of its
grid, and each die gets a contiguous run of them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r'''
#include "lossless_entropy_coded_amd/csrc/tiles.h"
#include <cstdio>
#include <vector>
using namespace wc;
int main() {
    unsigned checked = 0;
    for (uint32_t ms = 1; ms <= 40; ++ms)
        for (uint32_t ns = 1; ns <= 40; ++ns) {
            std::vector<int> taken(ms * ns, 0);
            const uint32_t grid = tile_grid(ms, ns);
            if (grid < ms * ns || grid % kDies != 0 || grid >= ms * ns + kDies) return 1;
            for (uint32_t id = 0; id < grid; ++id) {
                uint32_t m = 0, n = 0;
                if (!tile_of(id, ms, ns, m, n)) continue;
                if (m >= ms || n >= ns || taken[m * ns + n]++) return 2;
                ++checked;
            }
            for (int t : taken)
                if (t != 1) return 3;
            // a die's workgroups in a band of 4 x ns tiles take whole columns of it, one behind the other
            for (uint32_t die = 0; die < kDies; ++die)
                for (uint32_t id = die; id + kDies < grid; id += kDies) {
                    uint32_t m = 0, n = 0, m1 = 0, n1 = 0;
                    if (!tile_of(id, ms, ns, m, n) || !tile_of(id + kDies, ms, ns, m1, n1)) continue;
                    const bool next = m1 / 4 == m / 4 ? (m1 == m + 1 && n1 == n) || (m1 % 4 == 0 && n1 == n + 1)
                                                      : m1 / 4 == m / 4 + 1 && m1 % 4 == 0 && n1 == 0 && n == ns - 1;
                    if (!next) return 4;
                }
        }
    std::printf("%u\n", checked);
}
'''


def test_each_tile_is_taken_once(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is missing")
    (tmp_path / "tiles.cpp").write_text(SOURCE)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    ROOT, str(tmp_path / "tiles.cpp"), "-o", str(tmp_path / "tiles")], check=True, capture_output=True,
                   timeout=300)
    r = subprocess.run([str(tmp_path / "tiles")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert int(r.stdout) == (40 * 41 // 2) ** 2
