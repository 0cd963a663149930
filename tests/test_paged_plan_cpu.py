"""What the planner of paged_attention takes for granted: the CTAs that an SM holds of each kernel. Parts are joined in
clusters only where all of them run at once, which a number too large would belie."""
import os
import re
import subprocess

import pytest

SRC = r"""
#include <cstdio>
#include "paged_attn.h"
using namespace kvevict;
int main()
{
    for (int q4 = 0; q4 < 2; ++q4)
        for (int d = 64; d <= 128; d += 64)
            for (int r = 1; r <= 8; r *= 2) std::printf("simt %d %d %d %d\n", q4, d, r, paged_simt_ctas(q4, d, r));
    for (int q4 = 0; q4 < 2; ++q4)
        for (int r = 8; r <= 16; r += 8) std::printf("mma %d %d %d\n", q4, r, paged_mma_ctas(q4, r));
}
"""


def registers(build, name, tmp_path):
    """{template arguments: registers a thread} of a source's kernels."""
    out = subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-Xptxas", "-v", "-c", os.path.join(build.CSRC, name), "-o", str(tmp_path / "o")],
                         check=True, capture_output=True, text=True).stderr
    found, args = {}, None
    for line in out.split("\n"):
        if "Compiling entry function" in line:
            m = re.search(r"paged_(?:simt|mma)_kernelI((?:L[bi]\d+E)+)E", line)
            args = tuple(int(x) for x in re.findall(r"L[bi](\d+)E", m.group(1))) if m else None
        m = re.search(r"Used (\d+) registers", line)
        if m and args:
            found[args] = int(m.group(1))
    return found


@pytest.fixture(scope="module")
def planned(tmp_path_factory):
    from kv_cache_eviction_decode_gb300 import build
    d = tmp_path_factory.mktemp("plan")
    (d / "s.cu").write_text(SRC)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, str(d / "s.cu"), "-o", str(d / "s")], check=True)
    lines = subprocess.run([str(d / "s")], capture_output=True, text=True, check=True).stdout.split("\n")
    return [line.split()[:1] + [int(x) for x in line.split()[1:]] for line in lines if line]


@pytest.mark.parametrize("kind,name", [("simt", "paged_attn.cu"), ("mma", "paged_attn_mma.cu")])
def test_an_sm_holds_the_planned_ctas(planned, kind, name, tmp_path):
    from kv_cache_eviction_decode_gb300 import build
    found = registers(build, name, tmp_path)
    seen = 0
    for p in planned:
        if p[0] != kind:
            continue
        for args, regs in found.items():
            if args == tuple(p[1:4]) if kind == "simt" else (args[1], 8 * args[2]) == tuple(p[1:3]):
                seen += 1
                assert 65536 // ((regs + 7) // 8 * 8 * 128) >= p[-1], (args, regs, p[-1])
    assert seen == len(found) and seen > 0
