"""The attention join's places in shared memory, checked on the host for every
number of heads a CTA and of CTAs a cluster: each part of a head's sum, and each
reference and sum, goes to a place of its own inside its array, and lies where
the CTA that joins the head reads it.  A place outside would be a write past the
CTA's shared memory on the GPU; this finds it without one.  The check compiles
the kernel's source file into a host program (nvcc; no GPU needed)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hierarchical_sparse_kv_request_gb300", "csrc")

PROGRAM = r"""
#include "attend.cu"
#include <cstdio>
#include <vector>
int main()
{
    using namespace hs;
    long bad = 0, n = 0;
    for (int splits = 1; splits <= MAX_SPLITS; ++splits) {
        for (int i = 0; i < HEADS + MAX_SPLITS; ++i)
            bad += (int)(i * inverse_of(splits) >> 16) != i / splits;
        if (splits == 1) continue;
        for (int heads = 1; heads <= HEADS; ++heads)
            for (int owner = 0; owner < splits; ++owner) {
                const bool staged = staged_slots(heads, splits) <= SLOTS;
                auto cta = [&](int rank) {
                    return Join{0, 0, 0, nullptr, heads, splits, rank, inverse_of(splits), staged};
                };
                const Join own = cta(owner);
                std::vector<int> slot(SLOTS, 0), ml(HEADS + MAX_SPLITS, 0);
                auto take = [&](std::vector<int> &v, long at) {
                    ++n;
                    if (at < 0 || at >= (long)v.size() || v[at]++) ++bad;
                };
                int mine = 0, sent = 0;
                for (int i = 0; i < heads; ++i) {
                    const int m = i / splits;
                    if (i % splits != owner) {       // staged on its way to another
                        if (staged) take(slot, i);
                        continue;
                    }
                    ++mine;
                    for (int rank = 0; rank < splits; ++rank) {
                        const Join from = cta(rank);
                        const int p = from.ml_at(i, owner) - m * splits;
                        const uint32_t at = from.place(owner, m);
                        // as factors() and finish() go through them
                        bad += at != (p == 0 ? own.own(m) : own.others(owner, m) + (p - 1) * O_STRIDE);
                        bad += (p == 0) != (rank == owner) || p < 0 || p >= splits || at % O_STRIDE != 0;
                        bad += staged && rank == owner && at != i * O_STRIDE;
                        take(slot, at / O_STRIDE);
                        take(ml, from.ml_at(i, owner));
                        sent += rank != owner;
                    }
                }
                bad += own.count(owner) != mine || own.parts() != (uint32_t)sent;
                bad += mine * 16 > AT_NT;             // factors(): 16 threads a head
            }
    }
    std::printf("%ld places, %ld wrong\n", n, bad);
    return bad != 0;
}
"""


def test_every_part_has_a_place_of_its_own(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    src = tmp_path / "join_check.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "join_check"
    res = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                          "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr
    assert " 0 wrong" in run.stdout
