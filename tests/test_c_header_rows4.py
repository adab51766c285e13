"""include/hisparse_rows4.h is plain C: a C99 program (and the same file as
C++17) that includes it alone compiles without warnings, links against
libhisparse.so and runs its host-only checks (no GPU is needed for these)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "hierarchical_sparse_kv_request_gb300")

PROGRAM = r"""
#include <stdio.h>
#include <string.h>
#include "hisparse_rows4.h"

int main(void)
{
    hisparse_attend_args args;
    int64_t bytes = 0;
    memset(&args, 0, sizeof args);
    if (hisparse_pack_rows(NULL, 576, HISPARSE_BF16, 1, NULL, 416, NULL) != HISPARSE_ERR_INVALID_ARG) return 1;
    if (hisparse_unpack_rows(NULL, 416, 0, NULL, 576, HISPARSE_F16, NULL) != HISPARSE_OK) return 2;
    if (hisparse_attend(&args, NULL) != HISPARSE_ERR_INVALID_ARG) return 3;
    if (hisparse_attend_workspace(2, HISPARSE_MAX_HEADS, HISPARSE_MAX_TOP_K, 1, &bytes) != HISPARSE_OK) return 4;
    if (bytes <= 0) return 5;
    if (hisparse_evict_select(1, 1, NULL, 0, 0, NULL, NULL, 0, 1, NULL, NULL, NULL, NULL) != HISPARSE_ERR_INVALID_ARG)
        return 6;
    if (hisparse_evict(NULL, 0, NULL, 0, 0, NULL, 0, 1, NULL, NULL, NULL, NULL) != HISPARSE_ERR_INVALID_ARG) return 7;
    if (HISPARSE_MAX_PACKED_ROWS <= 0 || HISPARSE_STATUS_BIT(HISPARSE_STATUS_ATTEND_TIMEOUT) != 512) return 8;
    printf("ok %d %d\n", (int)sizeof args, HISPARSE_ROW4_LATENT + HISPARSE_ROW4_ROPE - HISPARSE_ROW4_VALUES);
    return 0;
}
"""


@pytest.fixture(scope="module")
def lib_built():
    import __graft_entry__
    __graft_entry__.build()
    return os.path.join(PKG, "libhisparse.so")


@pytest.mark.parametrize("compiler,flags", [("gcc", ["-x", "c", "-std=c99", "-pedantic"]),
                                            ("g++", ["-x", "c++", "-std=c++17"])])
def test_header_compiles_links_and_runs(tmp_path, lib_built, compiler, flags):
    if shutil.which(compiler) is None:
        pytest.skip(f"{compiler} not found")
    import ctypes

    from hierarchical_sparse_kv_request_gb300 import hisparse as H
    src = tmp_path / "use_rows4.c"
    src.write_text(PROGRAM)
    exe = tmp_path / "use_rows4"
    cmd = [compiler, *flags, "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
           str(src), "-x", "none", lib_built, "-o", str(exe), f"-Wl,-rpath,{PKG}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, (run.returncode, run.stderr)
    assert run.stdout.strip() == f"ok {ctypes.sizeof(H.AttendArgs)} 0"
