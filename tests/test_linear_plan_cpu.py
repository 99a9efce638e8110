"""How moe_mxfp8_linear cuts its calls (csrc/ops/linear_plan.h, host code alone):
every size is covered once and fits the workspace, and each size of the GPU
tests reaches the form that it is there for."""
import subprocess

import pytest

from tests.conftest import ROOT

PROGRAM = r"""
#include <stdio.h>
#include "mxfp4_moe_expert_02_amd/csrc/ops/linear_plan.h"
int main() {
    long long T, rows, inner;
    int act, mx;
    while (scanf("%lld %lld %lld %d %d", &T, &rows, &inner, &act, &mx) == 5) {
        const moe::LinearPlan p = moe::linear_plan(T, rows, inner, act, mx != 0);
        printf("%d %d %d %d %d %d %d %d %d %d\n", p.rows, p.wide, p.splits, p.grid.split_chunks, p.G, p.NT,
               p.grid.units, p.grid.groups, p.tile.row_blocks, p.tile.tok_blocks);
    }
}
"""
FIELDS = ("rows", "wide", "splits", "chunks", "G", "NT", "units", "groups", "row_blocks", "tok_blocks")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", ROOT,
                    str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def plans(sizes):  # (tokens, rows, inner, activation, MXFP8 output)
        text = "".join("%d %d %d %d %d\n" % s for s in sizes)
        r = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True)
        return [dict(zip(FIELDS, map(int, line.split()))) for line in r.stdout.splitlines()]
    return plans


def _form(p):
    name = "rows" if p["rows"] else "wide" if p["wide"] else "narrow"
    return name + (" split" if p["splits"] > 1 else "")


def test_every_size_is_covered(plans):
    sizes = [(T, rows, K, act, mx) for T in (1, 9, 16, 17, 100, 128, 129, 200, 511, 1001, 1024, 1025, 4096, 33333, 1 << 20)
             for rows in (64, 128, 192, 448, 2048, 4160, 7168, 1 << 20) for K in (128, 384, 2048, 7168, 65536)
             for act in (0, 3) for mx in (0, 1)]
    for s, p in zip(sizes, plans(sizes)):
        T, rows, K, act, mx = s
        chunks = K // 128
        # the parts of the inner axis cover it, and none is empty
        assert 1 <= p["splits"] <= 8 and (p["splits"] - 1) * p["chunks"] < chunks <= p["splits"] * p["chunks"], (s, p)
        assert p["splits"] == 1 or p["splits"] * T <= 8192, (s, p)
        if p["rows"]:
            assert p["units"] * 16 * p["G"] == rows and (p["groups"] - 1) * 16 * p["NT"] < T <= p["groups"] * 16 * p["NT"]
            # the shapes that are instantiated; whole blocks of 32 columns for MXFP8
            assert p["G"] in (1, 2, 4) and 1 <= p["NT"] <= 4 and (p["G"], p["NT"]) != (1, 4), (s, p)
            assert not mx or p["G"] * (1 if act == 3 else 2) >= 4, (s, p)
            assert act != 3 or p["G"] >= 2, (s, p)
        else:
            n = 256 if p["wide"] else 128
            assert (p["row_blocks"] - 1) * n < rows <= p["row_blocks"] * n
            assert (p["tok_blocks"] - 1) * n < T <= p["tok_blocks"] * n
    # the workspace is that of MXFP8 output: the other needs no more
    for a, b in zip(plans([s[:4] + (0,) for s in sizes]), plans([s[:4] + (1,) for s in sizes])):
        assert a["splits"] in (1, b["splits"])


def test_gpu_tests_reach_their_forms(plans):
    from tests.test_gpu_linear_sums import FORMS
    sizes = [s + (act, mx) for _, s in FORMS.values() for act, mx in ((0, 0), (0, 1), (3, 1))]
    want = [form for form, _ in FORMS.values() for _ in range(3)]
    for s, f, p in zip(sizes, want, plans(sizes)):
        assert _form(p) == f, (s, p)
        if not p["rows"]:  # past what is staged, twice over
            assert p["chunks"] >= 5, (s, p)
    assert {f for f, _ in FORMS.values()} == {"rows", "narrow", "narrow split", "wide"}
    narrow = [p for s, p in zip(sizes, plans(sizes)) if _form(p) == "narrow"]
    tiles = [p["row_blocks"] * p["tok_blocks"] for p in narrow]
    assert min(tiles) <= 256 < max(tiles)  # one workgroup per CU, and two
