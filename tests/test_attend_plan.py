"""The rule that spreads a row of the paged attention over CTAs (csrc/attend_plan.h), compiled for the host, on devices that
hold different numbers of clusters."""
import os
import subprocess

import pytest

import test_gpu_paged_attend as T
from conftest import ROOT

PROGRAM = r"""
#include <stdio.h>
#include "attend_plan.h"
int main() {
    int fit[17], rows, tiles;
    for (int i = 0; i < 17; ++i)
        if (scanf("%d", &fit[i]) != 1) return 1;
    while (scanf("%d %d", &rows, &tiles) == 2)
        printf("%d\n", csa2::paged_attend_split(rows, tiles, [&](int size) { return fit[size]; }));
}
"""
# clusters of each size at once (index: CTAs of a cluster), as cudaOccupancyMaxActiveClusters gives them
WHOLE = [0, 148, 74, 45, 33, 26, 22, 15, 15, 15, 11, 7, 7, 7, 7, 7, 7]
PART = [0, 18, 9, 5, 4, 3, 2, 2, 2] + [0] * 8  # one GPC: no cluster above 8
NONE = [0, 148] + [0] * 15


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, exe = str(d / "p.cpp"), str(d / "p")
    open(src, "w").write(PROGRAM)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "compressed_sparse_attention_append_b200", "csrc"),
                           src, "-o", exe])

    def call(fit, cases):
        text = " ".join(map(str, fit)) + "\n" + "\n".join(f"{r} {t}" for r, t in cases)
        return list(map(int, subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60)
                        .stdout.split()))

    return call


@pytest.mark.parametrize("fit", [WHOLE, PART, NONE])
def test_no_cluster_is_larger_than_the_device_takes(split, fit):
    cases = [(rows, tiles) for rows in (*range(1, 80), 1000) for tiles in range(0, 18)]
    for (rows, tiles), s in zip(cases, split(fit, cases)):
        assert 1 <= s <= max(tiles, 1)
        if s > 1:
            # a size that the device takes (one that it holds all of, or a smaller one with as few tiles a CTA)
            assert any(rows <= fit[size] for size in range(s, 17)), (rows, tiles, s)
            each = -(-tiles // s)
            assert s == 1 or -(-tiles // (s - 1)) > each


def test_few_rows_are_spread_as_wide_as_they_fit(split):
    cases = [(1, 16), (7, 16), (8, 16), (15, 17), (16, 12), (22, 6), (23, 5), (26, 5), (27, 5), (74, 5), (75, 5), (1, 17), (1, 1)]
    assert split(WHOLE, cases) == [16, 16, 8, 6, 6, 6, 5, 5, 3, 2, 1, 9, 1]
    # (nine clusters of 2 hold 7 and 8 rows)
    assert split(PART, cases) == [8, 2, 2, 1, 1, 1, 1, 1, 1, 1, 1, 6, 1]


def test_the_gpu_tests_reach_every_cluster(split):
    cases = [(B, -(-k // 128) + (win > 0)) for B, k, win in T.CLUSTERS]
    assert set(split(WHOLE, cases)) >= set(range(1, 17))
