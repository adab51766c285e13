"""The pieces of attend_prefix's workspace, checked on the host with the kernels' own
constants: each as long as what is written there, one behind the other, none past the
end.  The check compiles the kernels' source file into a host program (nvcc; no GPU
needed)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hierarchical_sparse_kv_request_gb300", "csrc")

PROGRAM = r"""
#include "prefix.cu"
#include <cstdio>
int main()
{
    using namespace hs;
    long bad = 0, n = 0;
    for (int R : {1, 2, 37, 256, 8192})
        for (int H : {1, 16, 40, 128, 1024})
            for (int len : {1, 127, 128, 129, 4256, 4257, 8448, 8449, 40000, 1 << 20}) {
                int64_t bytes;
                const PrefixParts w = lay_out(R, H, len, nullptr, &bytes);
                const int64_t begin[] = {(int64_t)(uintptr_t)w.o, (int64_t)(uintptr_t)w.ml, (int64_t)(uintptr_t)w.there, (int64_t)(uintptr_t)w.image, bytes};
                const int64_t size[] = {(int64_t)w.pairs * 2 * PAIR_HEADS * kLatent * 4, (int64_t)w.pairs * 2 * PAIR_HEADS * (int64_t)sizeof(float2),
                                        // a byte a round of expand_kernel, read 16 at a time
                                        (int64_t)w.tiles * (KEYS / EX_ROWS), (int64_t)w.tiles * TILE_BYTES};
                const int64_t align[] = {16, 8, 16, 128};
                for (int k = 0; k < 4; ++k, ++n) bad += begin[k] < 0 || begin[k] % align[k] || begin[k] + size[k] > begin[k + 1];
                // the rounds that expand_kernel counts are those that prefix_kernel reads, 32 a tile
                bad += KEYS / EX_ROWS != 32 || w.tiles != (len + KEYS - 1) / KEYS;
            }
    std::printf("%ld pieces, %ld wrong\n", n, bad);
    return bad != 0;
}
"""


def test_every_piece_has_its_place(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    src = tmp_path / "workspace_check.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "workspace_check"
    res = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                          "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr
