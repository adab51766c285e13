"""include/hisparse_pages.h is plain C: a C99 program (and the same file as C++17)
that includes it alone compiles without warnings, links against libhisparse.so and
runs its host-only checks (no GPU is needed for these)."""

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "hierarchical_sparse_kv_request_gb300")

PROGRAM = r"""
#include <stddef.h>
#include <stdio.h>
#include <string.h>
#include "hisparse_pages.h"

int main(void)
{
    hisparse_page_tables_args tables;
    hisparse_attend_prefix_args prefix;
    int64_t bytes = 0;
    memset(&tables, 0, sizeof tables);
    memset(&prefix, 0, sizeof prefix);
    if (hisparse_page_tables(&tables, NULL) != HISPARSE_ERR_INVALID_ARG) return 1;
    if (hisparse_attend_prefix(&prefix, NULL) != HISPARSE_ERR_INVALID_ARG) return 2;
    if (hisparse_attend_prefix_workspace(2, HISPARSE_MAX_HEADS, HISPARSE_MAX_PREFIX, &bytes) != HISPARSE_OK) return 3;
    if (bytes <= (int64_t)HISPARSE_MAX_PREFIX * HISPARSE_ROW16_BYTES) return 4;
    if (hisparse_norm_rows(NULL, 576, HISPARSE_F16, 0, NULL, 1e-6f, NULL, HISPARSE_ROW8_BYTES, HISPARSE_ROW8_BYTES, 0,
                           NULL, NULL) != HISPARSE_OK)
        return 5;
    if (hisparse_gather_rows(NULL, HISPARSE_ROW16_BYTES, HISPARSE_ROW16_BYTES, 0, NULL, 1, NULL, 576, HISPARSE_BF16,
                             NULL) != HISPARSE_ERR_INVALID_ARG)
        return 6;
    if (HISPARSE_MAX_TABLE_BLOCKS <= 0) return 7;
    printf("ok %d %d %d %d\n", (int)sizeof tables, (int)offsetof(hisparse_page_tables_args, num_tokens),
           (int)sizeof prefix, (int)offsetof(hisparse_attend_prefix_args, part));
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
    from hierarchical_sparse_kv_request_gb300 import hisparse as H
    src = tmp_path / "use_pages.c"
    src.write_text(PROGRAM)
    exe = tmp_path / "use_pages"
    cmd = [compiler, *flags, "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
           str(src), "-x", "none", lib_built, "-o", str(exe), f"-Wl,-rpath,{PKG}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, (run.returncode, run.stderr)
    assert run.stdout.split() == ["ok", str(ctypes.sizeof(H.PageTablesArgs)), str(H.PageTablesArgs.num_tokens.offset),
                                  str(ctypes.sizeof(H.AttendPrefixArgs)), str(H.AttendPrefixArgs.part.offset)]
