"""The host's choice between single CTAs and CTA pairs, at sizes where both were measured
(152 SMs); the type of the operands plays no part."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_persistent_gb300", "csrc_experts")

PROGRAM = r"""
#include <cstdio>
#include "experts_plan.h"
int main() {
    long long R, E, wide, step;
    while (std::scanf("%lld %lld %lld %lld", &R, &E, &wide, &step) == 4)
        std::printf("%d\n", dg::experts::takes_pairs(R, E, wide, step, 152));
}
"""

# R, E, channels of D, channels of a single CTA's tile; the faster variant
CASES = [
    ((64 * 32, 64, 2048, 128), "single"), ((64 * 40, 64, 2048, 128), "single"), ((64 * 48, 64, 2048, 128), "single"),
    ((64 * 64, 64, 2048, 128), "pairs"), ((64 * 192, 64, 2048, 128), "pairs"), ((64 * 40, 64, 1024, 64), "single"),
    ((64 * 64, 64, 1024, 64), "pairs"),
    ((32 * 40, 32, 4096, 128), "single"), ((32 * 48, 32, 4096, 128), "single"), ((32 * 64, 32, 4096, 128), "pairs"),
    ((8 * 40, 8, 4096, 128), "single"), ((8 * 64, 8, 4096, 128), "pairs"),
    ((32 * 48, 32, 2048, 64), "single"), ((32 * 80, 32, 2048, 64), "pairs"),
    ((512, 1, 1024, 128), "single"), ((64, 1, 18432, 128), "single"), ((96, 1, 18432, 128), "pairs"),
    ((256, 1, 4096, 128), "single"), ((512, 1, 4096, 128), "pairs"),
    ((1, 1, 1, 128), "single"), ((2 ** 30 - 1, 1024, 2 ** 30 - 1, 64), "pairs"),
]


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "main.cpp").write_text(PROGRAM)
    compiler = shutil.which("g++") or shutil.which("c++")
    subprocess.run([compiler, "-std=c++17", "-I", CSRC, "-o", str(d / "main"), str(d / "main.cpp")], check=True)
    return str(d / "main")


def test_the_faster_variant_is_taken(program):
    text = "\n".join(" ".join(map(str, sizes)) for sizes, _ in CASES)
    out = subprocess.run([program], input=text, check=True, capture_output=True, text=True).stdout.split()
    assert [("single", "pairs")[int(x)] for x in out] == [want for _, want in CASES]
