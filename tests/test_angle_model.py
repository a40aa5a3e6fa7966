"""The rotation's angle (csrc/angle.cuh) compiled for the host, against whole-number arithmetic."""
import os
import random
import subprocess

import pytest

import _angles
from conftest import ROOT

PROGRAM = r"""
#include <stdio.h>
#include "angle.cuh"
int main() {
    long long pos;
    double f;
    while (scanf("%lld %la", &pos, &f) == 2) printf("%a\n", csa2::half_turns(pos, f));
}
"""


@pytest.fixture(scope="module")
def half_turns(tmp_path_factory):
    d = tmp_path_factory.mktemp("angle")
    src, exe = str(d / "a.cpp"), str(d / "a")
    open(src, "w").write(PROGRAM)
    subprocess.check_call(["g++", "-O2", "-ffp-contract=off", "-std=c++17", "-I",
                           os.path.join(ROOT, "compressed_sparse_attention_append_b200", "csrc"), src, "-o", exe])

    def call(cases):
        text = "".join(f"{p} {f.hex()}\n" for p, f in cases)
        return [float.fromhex(x) for x in subprocess.run([exe], input=text, capture_output=True, text=True, check=True,
                                                         timeout=60).stdout.split()]

    return call


def test_angles_hold_at_any_position_below_2_31(half_turns):
    """The last addition rounds a sum of at most 1 (2^-53); what is left out is below 2^-74: 2^-52 bounds both."""
    rng = random.Random(5)
    freqs = [10000.0 ** (-2 * j / 64) for j in range(32)] + [1.0, 1e-9, 0.7390851332151607, 3.0, 2.0 - 2.0 ** -52]
    cases = [(p, f) for f in freqs for p in (0, 1, 2, 4096, 131071, (1 << 20) + 1, (1 << 30) - 1, (1 << 31) - 2, (1 << 31) - 1)
             if p * f < 2.0 ** 32]
    cases += [(rng.randrange(1 << rng.randrange(1, 32)), rng.choice(freqs[:34]) * rng.uniform(0.1, 1.0)) for _ in range(20000)]
    got = half_turns(cases)
    assert len(got) == len(cases)
    for (p, f), h in zip(cases, got):
        d = abs(h - _angles.turns(p, f))
        assert min(d, abs(d - 2.0)) <= 2.0 ** -52, (p, f, h)
        assert abs(h) <= 1.0 + 2.0 ** -20


def test_the_whole_number_angles():
    import math

    for p, f in ((0, 1.0), (3, 0.5), (100, 0.25), (355, 1.0)):
        assert abs(_angles.angle(p, f) - math.remainder(p * f, 2 * math.pi)) < 1e-13
        assert abs(_angles.turns(p, f) - math.remainder(p * f, 2 * math.pi) / math.pi) < 1e-13
