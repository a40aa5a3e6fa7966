"""The rule that chooses the kernel of an FP8 product (csrc/fp8_plan.h), compiled for the host: the sizes of the GPU tests
reach what they are there for, whatever the rule becomes."""
import os
import subprocess

import pytest

import test_gpu_fp8_tiles as T
from conftest import ROOT

PROGRAM = r"""
#include <stdio.h>
#include "fp8_plan.h"
int main() {
    long long m, n;
    int k;
    while (scanf("%lld %lld %d", &m, &n, &k) == 3)
        printf("%d %d\n", (int)csa2::fp8_by_columns(m, n, k), csa2::fp8_cols_split((n + 127) / 128 * ((m + 63) / 64), (k + 127) / 128));
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, exe = str(d / "p.cpp"), str(d / "p")
    open(src, "w").write(PROGRAM)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "compressed_sparse_attention_append_b200", "csrc"),
                           src, "-o", exe])

    def call(m, n, k):
        by_columns, split = subprocess.run([exe], input=f"{m} {n} {k}", capture_output=True, text=True, check=True,
                                           timeout=60).stdout.split()
        return bool(int(by_columns)), int(split)

    return call


def test_the_sizes_of_the_persistent_kernels_tests(plan):
    odd = even = 0
    for m, n, k in T.MANY:
        assert not plan(m, n, k)[0], (m, n, k)
        tiles = -(-m // 128) * -(-n // 256)
        assert tiles > 148  # a CTA takes a second tile
        blocks = -(-k // 128)
        odd, even = odd + blocks % 2, even + 1 - blocks % 2
    assert odd and even
    assert any(-(-m // 128) * -(-n // 256) > 2 * 148 for m, n, k in T.MANY)  # and a third
    assert not plan(*T.FRAME)[0] and not plan(*T.NOT_FINITE)[0] and not plan(*T.STREAMS)[0]


def test_the_sizes_of_the_joins_tests(plan):
    splits = [plan(m, n, k) for m, n, k in T.JOINS]
    assert all(by_columns for by_columns, _ in splits) and {s for _, s in splits} == {2, 4, 8}


def test_the_split_leaves_every_cta_a_block(plan):
    for m in (1, 16, 64, 65, 300):
        for n in (1, 128, 4099):
            for k in (16, 128, 144, 512, 1024, 8192):
                split = plan(m, n, k)[1]
                assert split in (1, 2, 4, 8) and (split == 1 or -(-k // 128) >= 2 * split)
