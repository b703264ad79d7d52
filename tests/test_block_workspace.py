"""The workspace that selective_scan_bwd takes stays within what include/ttt.h promises."""
import os
import re
import subprocess

import pytest

from linear_attention_ttt_b200 import build as B

PROGRAM = r"""
#include <stdio.h>
#include "block.cuh"
int main() {
  const int ns[] = {1, 15, 16, 17, 32, 33, 48, 49, 64}, bs[] = {1, 3, 64}, hs[] = {1, 5};
  const int ts[] = {1, 2, 31, 32, 33, 63, 64, 65, 127, 200, 1000, 4096, 33333, 300000};
  const int ds[] = {1, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 203, 4096};
  for (int N : ns) for (int T : ts) for (int d : ds) for (int b : bs) for (int h : hs) {
    ttt::ScanBwdArgs a{};
    a.f.B = b, a.f.H = h, a.f.T = T, a.f.d = d, a.f.N = N, a.f.G = 1;
    printf("%d %d %d %d %d %zu\n", b, h, T, d, N, ttt::selective_scan_bwd_workspace(a));
  }
}
"""


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    """(B, H, T, d, N, bytes): the library's own answer, asked by a small program."""
    B.build()
    at = tmp_path_factory.mktemp("workspace")
    (at / "ask.cu").write_text(PROGRAM)
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", f"-I{B.CSRC}", str(at / "ask.cu"),
                    "-o", str(at / "ask"), B.LIB, "-Xlinker", "-rpath", "-Xlinker", B.PKG], check=True)
    out = subprocess.run([str(at / "ask")], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_scan_backward_workspace(sizes):
    text = open(os.path.join(B.ROOT, "include", "ttt.h")).read()
    per = int(re.search(r"Workspace: at most (\d+) bytes x B\*H x \(T rounded up to 32\) x ceil\(N/16\) x", text).group(1))
    up = lambda n, k: -(-n // k) * k
    assert len(sizes) > 1000
    for b, h, T, d, N, got in sizes:
        assert 0 < got <= per * b * h * up(T, 32) * -(-N // 16) * up(d, 64), (b, h, T, d, N)
