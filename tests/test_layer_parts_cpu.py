"""The host rule that cuts K of moe_layer's second product into parts (csrc/layer_parts.h), compiled as plain C++ and walked over
all sizes the call accepts: no part may be without a stage, because the kernel's unit queue counts on one a unit."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WALK = r"""
#include <cstdio>
#include "layer_parts.h"
using namespace moe;

static long long calls = 0, bad = 0;

static void check(const moe_dims& d, int weights) {
    const int step = weights == MOE_LAYER_BF16 ? 64 : weights == MOE_LAYER_FP8_BLOCK ? 256 : 512;
    const int steps = (d.intermediate + step - 1) / step, parts = layer_parts(d, weights);
    ++calls;
    bool ok = parts >= 1 && parts <= 16;
    // the kernel's bounds of each part
    int at = 0;
    for (int q = 0; ok && q < parts; ++q) {
        const int each = part_steps(steps, parts), st0 = q * each, st1 = std::min(steps, st0 + each);
        ok = st0 == at && st1 > st0;
        at = st1;
    }
    if ((!ok || at != steps) && bad++ < 10)
        std::printf("weights %d H %d I %d T %d K %d E %d S %d: %d stages in %d parts\n", weights, d.hidden, d.intermediate,
                    d.num_tokens, d.topk, d.num_experts, d.num_shared_experts, steps, parts);
}

int main() {
    for (int w = 0; w < 3; ++w)
        for (int H = 128; H <= 1 << 16; H += 128) {
            const int columns = H / (w == MOE_LAYER_BF16 ? 128 : 32);
            // experts with rows: all counts at which the rule can cut at all, and the first one past them
            for (int experts = 1; experts <= 1024; ++experts) {
                for (int I = 128; I <= 1 << 16; I += 128) check({64, H, I, experts, std::min(experts, 32), 0}, w);
                if ((long long)columns * experts > 4096) break;
            }
        }
    // the same count of experts by way of few tokens and of shared experts
    const int hs[] = {128, 512, 1024, 2048, 3584, 4096, 7168, 16384}, es[] = {1, 2, 8, 16, 60, 64, 256, 1000};
    for (int w = 0; w < 3; ++w)
        for (int H : hs)
            for (int I = 128; I <= 1 << 16; I += 128)
                for (int E : es)
                    for (int T : {1, 2, 5, 64})
                        for (int K : {1, 2, 8})
                            for (int S : {0, 1, 4})
                                if (K <= E) check({T, H, I, E, K, S}, w);
    std::printf("%lld calls, %lld bad\n", calls, bad);
    return bad != 0;
}
"""


def test_every_part_of_the_second_product_has_a_stage(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(WALK)
    cc = subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), "-I",
                         os.path.join(ROOT, "moe_expert_ffn_topk_gb300", "csrc"), str(src), "-o", str(exe)],
                        capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
