"""The choice of the kernel that writes N channels of D beside a product (adapter_beside.cuh),
on the CPU: never for a gated D, which has half of them. And the largest sizes that both calls take."""
import itertools
import os
import re
import shutil
import subprocess

import dense_gemm_persistent_gb300 as dg
from dense_gemm_persistent_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_persistent_gb300", "csrc_adapters")

PROGRAM = r"""
#include <cstdio>
#include "adapter_forms.h"
int main() {
    for (int bits = 0; bits < 32; ++bits)
        for (int N = 2; N <= 16; N += 2)
            std::printf("%d %d %d\n", bits, N, dg::adapters::beside_form(bits & 1, bits & 2, bits & 4, bits & 8, bits & 16, N));
}
"""


def test_no_gated_result_is_written_as_n_channels(tmp_path):
    (tmp_path / "main.cpp").write_text(PROGRAM)
    compiler = shutil.which("g++") or shutil.which("c++")
    subprocess.run([compiler, "-std=c++17", "-I", CSRC, "-o", str(tmp_path / "main"), str(tmp_path / "main.cpp")], check=True)
    out = subprocess.run([str(tmp_path / "main")], check=True, capture_output=True, text=True).stdout
    rows = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert [r[:2] for r in rows] == list(itertools.product(range(32), range(2, 17, 2)))
    for bits, N, beside in rows:
        prompt, product, gated, d_f32, c_f32 = (bool(bits >> i & 1) for i in range(5))
        assert beside == (prompt and not (product or gated or d_f32 or c_f32) and N % 8 == 0), (bits, N)


def test_the_launches_follow_the_rule():
    text = open(os.path.join(CSRC, "adapters.cu")).read()
    assert re.findall(r"const bool beside = (.*);", text) == [
        "dg::adapters::beside_form(p.prompt, c.W != nullptr, p.gated, p.d_f32, c.C && p.c_f32, p.N)"]
    assert len(re.findall(r"launch_beside<\w+>\(c, p, dev\)", text)) == text.count("if (beside) return") * 2 == 2


def test_the_limits_that_the_header_states():
    build.build()
    size = dg.dgemm_adapter_workspace_size
    assert size(1 << 24, 8, 8, 8, 1) > 0 and size((1 << 24) + 1, 8, 8, 8, 1) == 0
    assert size(1, (1 << 30) - 1, 8, 8, 1) > 0 and size(1, 1 << 30, 8, 8, 1) == 0
    assert size(1, 8, (1 << 30) - 8, 8, 1) > 0 and size(1, 8, 1 << 30, 8, 1) == 0
