"""How attend_prefix cuts its work up, checked on the host: every tile of every group
of heads belongs to one pair of CTAs, a pair has at most two parts of groups and each
of them a place of its own in the workspace, the join finds those and no others, and
every value of a part has a place inside it.  A place outside would be a write past the
workspace on the GPU; this finds it without one.  The check compiles the kernel's source
file into a host program (nvcc; no GPU needed)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hierarchical_sparse_kv_request_gb300", "csrc")

PROGRAM = r"""
#include "prefix.cu"
#include <cstdio>
#include <vector>
int main()
{
    using namespace hs;
    long bad = 0, n = 0;
    const int heads[] = {1, 64, 127, 128, 129, 512, 1480, 4096, 9728, 9729, 25600, 1 << 20};
    for (int h : heads)
        for (int len = 1; len <= 1 << 20; len = len < 700 ? len + 61 : len * 3) {
            if ((int64_t)h * len > 40000000) continue;
            int64_t bytes;
            PrefixParts w = lay_out(h > 1024 ? h / 1024 : 1, h > 1024 ? 1024 : h, len, nullptr, &bytes);
            const int groups = ((h > 1024 ? h / 1024 * 1024 : h) + 127) / 128, most = w.pairs;
            bad += w.tiles != (len + 127) / 128 || w.groups != groups;
            bad += most < 1 || most > MAX_PAIRS;
            // the workspace's pieces, one behind the other
            const int64_t o = (int64_t)(uintptr_t)w.o, ml = (int64_t)(uintptr_t)w.ml, there = (int64_t)(uintptr_t)w.there,
                          image = (int64_t)(uintptr_t)w.image;
            bad += o < 0 || o % 16 || ml < o + (int64_t)most * 2 * 128 * 512 * 4 || ml % 8;
            bad += there < ml + (int64_t)most * 2 * 128 * 8 || there % 16 || image < there + (int64_t)w.tiles * 16 || image % 16;
            bad += bytes < image + (int64_t)w.tiles * TILE_BYTES;
            cut_evenly(w);
            bad += w.pairs < 1 || w.pairs > most;
            bad += w.start[0].group != 0 || w.start[0].tile != 0 || w.start[w.pairs].group != groups || w.start[w.pairs].tile != 0;
            std::vector<std::vector<int64_t>> parts(groups);    // of a group: places
            std::vector<int> used(most * 2, 0);
            int64_t all = 0;
            for (int p = 0; p < w.pairs; ++p) {
                const auto begin = w.start[p], end = w.start[p + 1];
                bad += begin.group >= groups || begin.tile >= w.tiles || begin.tile < 0;
                const int64_t count = (int64_t)(end.group - begin.group) * w.tiles + end.tile - begin.tile;
                bad += count < 1 || count > INT32_MAX;      // no pair without work
                all += count;
                int64_t n1 = 0;
                int group = begin.group, t0 = begin.tile;
                const int last_group = end.tile > 0 ? end.group : end.group - 1;
                for (; group <= last_group; ++group, t0 = 0) {        // as prefix_kernel goes through them
                    const int t1 = group == end.group ? end.tile : w.tiles;
                    ++n;
                    n1 += t1 - t0;
                    bad += t1 <= t0 || group >= groups;
                    const bool whole = t0 == 0 && t1 == w.tiles;
                    const int64_t place = (int64_t)p * 2 + (t0 == 0);
                    if (!whole && used[place]++) ++bad;
                    parts[group].push_back(whole ? -1 : place);
                }
                bad += n1 != count;
            }
            bad += all != (int64_t)w.tiles * groups;
            int joins = 0;
            for (int g = 0; g < groups; ++g) {                  // as join_kernel does
                bad += (parts[g].size() == 1) != (parts[g][0] < 0);
                if (parts[g].size() == 1) continue;
                if (joins >= w.joins || joins >= MAX_PAIRS) {
                    ++bad;
                    break;
                }
                const auto join = w.join[joins++];
                bad += join.group != g || join.parts != (int)parts[g].size();
                for (int k = 0; k < (int)parts[g].size(); ++k) bad += parts[g][k] != (int64_t)(join.first + k) * 2 + (k == 0);
            }
            bad += joins != w.joins;
        }
    // a part's values: heads by fours of values
    std::vector<int> at(128 * 512 / 4, 0);
    for (int i = 0; i < 128; ++i)
        for (int v = 0; v < 128; ++v) {
            const int x = part_at(i, v);
            if (x % 16 || x < 0 || x / 16 >= (int)at.size() || at[x / 16]++) ++bad;
            // as the softmax warps write them: warp (half of the values, heads' half), image of 32
            // columns, lane, unit
            const int rank = i / 64, lane = i % 32, warp = (v / 64) * 2 + i / 32 % 2, c = v / 8 % 8, unit = v % 8;
            bad += x != ((rank * 4 + warp) * 8 + c) * PART_IMAGE + lane * 128 + ((unit ^ (lane & 7)) << 4);
        }
    // the blocks of a half tile: each once, the rope part last, X and Y of 128 values in turn
    int seen = 0;
    for (int k = 0; k < 9; ++k) seen |= 1 << block_at(k);
    bad += seen != 511 || block_at(8) != 8;
    for (int k = 0; k < 8; ++k) {
        const int h = k / 4, y = k / 2 % 2;
        bad += block_at(k) != y * 4 + h * 2 + k % 2;
    }
    for (int u = 0; u < 64; ++u)      // where expand_kernel puts unit u
        bad += block_at((u % 32 / 16) * 4 + (u % 32 / 8 & 1) + (u >= 32 ? 2 : 0)) != u / 8;
    bad += MISC_AT % 1024 != 0 || sizeof(PrefixSmem) + MISC_AT > 232448 || ROPE_AT != SLOTS * SLOT || SLOT != 4 * BLOCK;
    bad += Q_SMEM * BLOCK < 8 * PART_IMAGE || P_AT + 4 * PART_IMAGE > MISC_AT || T_Q + Q_TMEM * 32 > 512 || T_S + 128 > T_Q;
    // the heads of both CTAs of every group: each once, 64 of a CTA at most
    for (int heads = 1; heads < 400; ++heads) {
        std::vector<int> had(heads, 0);
        for (int g = 0; g * 128 < heads; ++g) {
            const int share = heads_of_cta(heads, g);
            bad += share < 1 || share > 64;
            for (int rank = 0; rank < 2; ++rank)
                for (int i = 0; i < share; ++i) {
                    const int head = g * 128 + rank * share + i;      // as prefix_kernel
                    if (head >= heads) continue;
                    bad += head >= (g + 1) * 128 || had[head]++;
                    const int h = head % 128;                         // as join_kernel
                    bad += (h < share ? h : h - share + 64) != rank * 64 + i;
                }
        }
        for (int n : had) bad += n != 1;
    }
    // the rounds of expand_kernel: none left out, whatever the length
    for (int tiles = 1; tiles <= 8192; ++tiles) {
        const int rounds = tiles * (KEYS / EX_ROWS), n = expand_rounds(tiles), warps = expand_ctas(tiles) * (EX_NT / 32);
        bad += n < 1 || n > 2 || (int64_t)warps * n < rounds;
    }
    std::printf("%ld parts, %ld wrong\n", n, bad);
    return bad != 0;
}
"""


def test_every_tile_and_part_has_one_place(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    src = tmp_path / "parts_check.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "parts_check"
    res = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                          "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr
    assert " 0 wrong" in run.stdout
