"""The ranks that the product of t and B reads beyond 16 tokens
(csrc/wc12_ranks.cuh), on the host: no lane reads past a row's end, not even
in the last row of B or of t, and each rank is taken once."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp32_weight_compression_b200", "csrc")
PROGRAM = """
#include <cstdio>
#include "wc12_ranks.cuh"
int main() {
  for (uint32_t r = 8; r <= 256; r += 8)
    for (uint32_t j = 0; j < r; j += 16)
      for (uint32_t t = 0; t < 4; t++)
        std::printf("%u %u %u %d %u\\n", r, j, t, int(wc12a::has_ranks(j, t, r)), wc12a::ranks_from(j, t, r));
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    d = tmp_path_factory.mktemp("ranks")
    (d / "ranks.cpp").write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-D__host__=", "-D__device__=", "-I", CSRC, str(d / "ranks.cpp"), "-o", str(d / "ranks")])
    return [tuple(map(int, l.split())) for l in subprocess.check_output([str(d / "ranks")], text=True).splitlines()]


def test_no_lane_reads_past_a_row(lines):
    for r, j, t, has, at in lines:
        assert at % 4 == 0 and at + 4 <= r, (r, j, t)  # 8 aligned bytes within the row


def test_each_rank_once(lines):
    for r in range(8, 257, 8):
        taken = sorted(at + i for q, _j, _t, has, at in lines if q == r and has for i in range(4))
        assert taken == list(range(r))
