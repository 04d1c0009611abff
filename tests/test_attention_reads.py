"""Where attention's lanes read in a key's and a value's row (paged_rows.h, which the kernel
uses), gone through on the CPU for every head size, element size and lane."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# prints "D es row highest missing once": the bytes of a row, the byte after the last that any lane asks
# for, how many elements the lane that owns them does not get, and the byte after the last with one test a
# lane for all of its elements
PROGRAM = r"""
#include <stdio.h>
#include "paged_rows.h"
int main(void) {
    for (int es = 1; es <= 2; ++es)
        for (int D = 16 / es; D <= 256; D += 16 / es) {
            const int dp = tcm::head_instance(D), row = D * es;
            int high = 0, missing = 0, once = 0;
            if (D > dp) return 1;
            for (int c = 0; c < dp * es / 16; ++c)
                if (tcm::key_piece_in(c, D, es)) high = high > 16 * c + 16 ? high : 16 * c + 16;
            const int vb = tcm::value_bytes(dp, es), b = tcm::value_load(dp, es);
            if (vb % b || b > 16) return 1;
            for (int c = 0; c < 16; ++c) {
                for (int i = 0; i < vb / b; ++i) {
                    const int at = tcm::value_at(c, i, D, dp, es), own = c * vb + i * b;
                    if (at < 0) return 1;
                    high = high > at + b ? high : at + b;
                    for (int x = 0; x < b; x += es)
                        if (own + x < row && at != own) ++missing;
                }
                const int at = c * vb < row ? c * vb : 0;
                once = once > at + vb ? once : at + vb;
            }
            printf("%d %d %d %d %d %d\n", D, es, row, high, missing, once);
        }
    return 0;
}
"""


@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    d = tmp_path_factory.mktemp("reads")
    (d / "r.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "tensor_core_matrix_amd", "csrc"), str(d / "r.cpp"), "-o", str(d / "r")],
                   check=True)
    out = subprocess.run([str(d / "r")], check=True, capture_output=True, text=True).stdout
    return [tuple(int(x) for x in line.split()) for line in out.splitlines()]


def test_no_lane_reads_past_a_row(rows):
    assert len(rows) == 32 + 16
    for D, es, row, high, missing, _ in rows:
        assert high <= row and missing == 0, (D, es, row, high, missing)


def test_one_test_a_lane_would_not_do(rows):
    """The sizes whose last elements share a lane with what lies past the row: the check above sees
    them."""
    assert [D for D, es, row, _, _, once in rows if es == 2 and once > row] == list(range(136, 256, 16))
    assert not [D for D, es, row, _, _, once in rows if es == 1 and once > row]
