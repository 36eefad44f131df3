"""Shared memory of the routing kernel that places pairs: for every number of experts the
arrays lie inside the bytes that its launch requests, apart from one another and aligned."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_persistent_gb300", "csrc_experts")

PROGRAM = r"""
#include <cstdio>
#include "route_layout.h"
int main() {
    for (int E = 1; E <= 1024; ++E) {
        const dg::route::PlaceLayout l(E);
        std::printf("%d %d %d %zu %zu %zu\n", E, l.pitch, l.parts, l.before, l.base, l.bytes);
    }
}
"""


@pytest.fixture(scope="module")
def layouts(tmp_path_factory):
    d = tmp_path_factory.mktemp("layout")
    (d / "main.cpp").write_text(PROGRAM)
    compiler = shutil.which("g++") or shutil.which("c++")
    subprocess.run([compiler, "-std=c++17", "-I", CSRC, "-o", str(d / "main"), str(d / "main.cpp")], check=True)
    out = subprocess.run([str(d / "main")], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_every_array_is_inside_the_request(layouts):
    assert [row[0] for row in layouts] == list(range(1, 1025))
    for E, pitch, parts, before, base, size in layouts:
        assert pitch % 4 == 0 and E <= pitch < E + 4 and 1 <= parts and parts * (pitch // 4) <= 1024
        assert before >= 8 * E                                # the masks, one 64-bit word an expert
        assert before % 16 == 0 and base % 16 == 0            # quads are stored 16 bytes at a time
        last = 4 * ((parts - 1) * pitch + 4 * (pitch // 4))   # end of the last part's last quad
        assert base >= before + last and size >= base + last
        assert size <= 48 * 1024                              # what a launch has without an attribute


def test_the_launch_requests_the_layout():
    text = open(os.path.join(CSRC, "route.cu")).read()
    launches = re.findall(r"PLACE_THREADS, (.*), s\);\n", text)
    assert launches == ["dg::route::PlaceLayout(p.E).bytes"]
    kernel = text[text.index("route_place(const RouteParams p)"):]
    assert "PlaceLayout layout(p.E)" in kernel and "smem + layout.before" in kernel and "smem + layout.base" in kernel
