"""Which kernel a product with e4m3 matrices takes (csrc/gemm_fp8_plan.h, compiled for the host): the sizes that the GPU
tests call reach every kernel that any size can reach."""
import os
import shutil
import subprocess

import pytest

from test_gpu_gemm_fp8 import ONCE, SHAPES, TILES
from test_gpu_gemm_fp8_kernels import KERNELS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r'''
#include "lossless_entropy_coded_amd/csrc/gemm_fp8_plan.h"
#include <cmath>
#include <cstdio>
#include <random>
#include <set>
#include <string>
using namespace wc;
std::string name(uint32_t rows, uint32_t cols, uint64_t tokens, bool exact) {
    const GemmPlan g = plan_of(rows, cols, tokens, exact);
    if (g.few) return "few " + std::to_string(g.kind) + (exact ? " f32" : " bf16");
    const Kind& k = exact ? kExactKinds[g.kind] : kCodeKinds[g.kind];
    return std::to_string(k.bm) + "x" + std::to_string(k.bn) + (exact ? " f32" : " bf16") + (g.once ? " once" : "") +
           (g.pair ? " pair" : "") + (g.splits > 1 ? " splits" : "");
}
int main(int argc, char**) {
    if (argc == 1) {   // the plans of the sizes given
        unsigned rows, cols, exact;
        unsigned long tokens;
        while (std::scanf("%u %u %lu %u", &rows, &cols, &tokens, &exact) == 4)
            std::printf("%s\n", name(rows, cols, tokens, exact).c_str());
        return 0;
    }
    std::mt19937_64 r(7);   // those of sizes over the whole range
    std::uniform_real_distribution<double> u(0, 1);
    std::set<std::string> seen;
    for (int i = 0; i < 4000000; ++i) {
        const uint32_t rows = std::exp(u(r) * std::log(4194304.0)), cols = 16 * (uint32_t)std::exp(u(r) * std::log(4096.0));
        const uint64_t tokens = std::exp(u(r) * std::log(i & 1 ? 1048576.0 : 300.0));
        if (tokens * rows > WC_MAX_LOGITS) continue;
        for (bool exact : {false, true}) seen.insert(name(rows, cols, tokens, exact));
    }
    for (const std::string& s : seen) std::printf("%s\n", s.c_str());
}
'''


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is missing")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(SOURCE)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", ROOT, str(at / "plan.cpp"), "-o", str(at / "plan")],
                   check=True, capture_output=True, timeout=300)

    def run(sizes=None):
        text = None if sizes is None else "".join(f"{r} {c} {t} {int(out == 'f32')}\n" for r, c, t, out in sizes)
        return subprocess.run([str(at / "plan")] + (["all"] if sizes is None else []), input=text, text=True, check=True,
                              capture_output=True, timeout=300).stdout.splitlines()
    return run


def test_gpu_tests_reach_every_kernel(plans):
    sizes = [(*s, out) for s in SHAPES + TILES + ONCE for out in ("bf16", "f32")] + [s for s, _ in KERNELS]
    missing = set(plans()) - set(plans(sizes))
    assert not missing, missing


def test_kernels_are_those_that_they_are_here_for(plans):
    assert plans([s for s, _ in KERNELS]) == [name for _, name in KERNELS]


def test_workspaces_follow_the_plan(plans):
    """The library's own plan is the one that is looked at here: its workspace is there where sums are split."""
    import ctypes

    from lossless_entropy_coded_amd import wc

    b, where = ctypes.c_uint64(0), 1 << 24
    sizes = SHAPES + TILES + ONCE
    split = [any("splits" in n for n in plans([(*s, "bf16"), (*s, "f32")])) for s in sizes]
    for (rows, cols, tokens), want in zip(sizes, split):
        W = ctypes.byref(wc._Fp8(where, where, rows, cols))
        assert wc._lib.wc_gemm_fp8_work_bytes(W, tokens, ctypes.byref(b)) == wc.WC_OK
        assert (b.value > 0) == want, (rows, cols, tokens)
