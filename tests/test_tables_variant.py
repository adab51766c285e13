"""Which of page_tables' kernels a call gets, checked on the host: one CTA only where it has
few pages to move, whatever the number of requests.  The check compiles the kernels'
source file into a host program (nvcc; no GPU needed)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hierarchical_sparse_kv_request_gb300", "csrc")

PROGRAM = r"""
#include "tables.cu"
#include <cstdio>
int main()
{
    using namespace hs;
    int bad = 0;
    const int32_t some = 0;
    auto one = [&](int R, int64_t W, int shared, int tokens) {      // tokens < 0: no slot map
        TablesLaunch a = {};
        a.R = R, a.W = (int32_t)W, a.shared_count = shared, a.bs = 64;
        a.new_tokens = tokens < 0 ? nullptr : &some;
        a.tokens = tokens < 0 ? 0 : tokens;
        return one_cta(a);
    };
    // decode steps of 32 requests of 40,000 tokens in pages of 64, and taking them back
    bad += !one(32, 626, 0, 128) || !one(32, 626, 0, -1);
    // as many tokens in pages of one: far more than one CTA moves in a step's time
    bad += one(25, 81920, 0, -1) || one(25, 81920, 0, 128) || one(1, 81924, 0, -1) || one(8, 5121, 0, 64);
    // the shared prefix's pages do not move
    bad += !one(8, 5121, 5000, 64) || one(8, 5121, 1000, 64);
    // many tokens, or many requests
    bad += one(32, 626, 0, 4097) || one(257, 10, 0, 300) || one(33, 10, 0, -1);
    // sizes at the limits
    bad += one(8192, 1 << 18, 0, -1) || one(1, 1 << 20, 0, 1) || !one(1, 1 << 20, 1 << 20, 1) || !one(1, 1, 0, 0);
    for (int R = 1; R <= 256; R *= 2) bad += !one(R, 32768 / R, 0, 64) || one(R, 32768 / R + 1, 0, 64);
    std::printf("%d wrong\n", bad);
    return bad != 0;
}
"""


def test_one_cta_only_where_few_pages_can_move(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    src = tmp_path / "variant_check.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "variant_check"
    res = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                          "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr
