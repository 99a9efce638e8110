"""How moe_tree_attention's launches are cut (csrc/ops/attention_plan.h, host
code alone)."""
import subprocess

import pytest

from tests.conftest import ROOT

PROGRAM = r"""
#include <stdio.h>
#include "mxfp4_moe_expert_02_amd/csrc/ops/attention_plan.h"
int main() {
    long long T, heads;
    while (scanf("%lld %lld", &T, &heads) == 2) {
        const moe::AttentionJoin j = moe::attention_join(T, heads);
        printf("%d %u %u %d %lld\n", j.heads, j.x, j.y, moe::kJoinWaves, (long long)moe::kJoinRow);
    }
}
"""


@pytest.fixture(scope="module")
def joins(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", ROOT,
                    str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def joins(sizes):  # (tokens, heads)
        r = subprocess.run([str(d / "plan")], input="".join("%d %d\n" % s for s in sizes), capture_output=True,
                           text=True, check=True)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return joins


def test_join_covers_every_row_within_a_grid(joins):
    """Every head of every token has a wave, the grid is one that can be
    launched (less than 2^32 threads a dimension, 2^16 rows), and a wave's
    number is a 32-bit one."""
    sizes = [(T, heads) for T in (1, 9, 288, 4095, 4096, 65535, 1 << 18, (1 << 18) + 1, (1 << 20) - 1, 1 << 20)
             for heads in (1, 3, 7, 56, 64, 255, 256, 257, 1023, 1024)]
    for (T, heads), (of_wave, x, y, waves, row) in zip(sizes, joins(sizes)):
        need = T * -(-heads // of_wave)
        assert of_wave == (4 if T * heads >= 4096 else 1)
        assert 1 <= x * waves * 64 < 1 << 32 and 1 <= y < 1 << 16, (T, heads)
        assert x == row or y == 1
        assert need <= x * y * waves < need + (row if y > 1 else 1) * waves, (T, heads)
        assert x * y * waves < 1 << 31
