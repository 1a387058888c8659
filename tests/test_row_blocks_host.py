"""How the bias gradient's kernel deals rows over its blocks, on the CPU: every row in one block, up to the most rows the entry
accepts, without an integer that wraps (undefined behaviour is trapped)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mlp_latency_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "row_blocks.h"
using namespace mlpl;
static long bad(int64_t N, int64_t rows)
{
    const int32_t block = grad_block_rows(N, 152, rows), blocks = static_cast<int32_t>((rows + block - 1) / block);
    int64_t next = 0;
    for (int32_t b = 0; b < blocks; ++b) {
        const int32_t lo = b * block, hi = block_end(lo, block, static_cast<int32_t>(rows));
        if (lo != next || hi <= lo)
            return 1;
        next = hi;
    }
    return next != rows;
}
int main()
{
    long n = 0;
    for (int64_t N : {8, 264, 4096, 40000}) {
        for (int64_t rows = 1; rows < 3000; ++rows)
            n += bad(N, rows);
        for (int64_t rows = (int64_t{1} << 31) - 1024; rows > (int64_t{1} << 31) - 5000; --rows)
            n += bad(N, rows);
    }
    std::printf("%ld\n", n);
    return n != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_blocks_of_rows_cover_them_once(tmp_path):
    src, exe = tmp_path / "blocks.cpp", str(tmp_path / "blocks")
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-I", CSRC, "-o", exe, str(src)],
                   check=True)
    run = subprocess.run([exe], capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout.strip() == "0", (run.returncode, run.stdout)
