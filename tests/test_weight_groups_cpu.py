"""Sums of words' weights by groups of neighbouring values (csrc/weight.h), compiled for the
CPU, against long double."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("groups") / "check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-I", os.path.join(ROOT, "int4_weight_quantized_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "weight_groups_check.cpp"), "-o", exe], check=True)
    return lambda *a: [float(x) for x in subprocess.run([exe, *map(str, a)], check=True, capture_output=True, text=True).stdout.split()]


# A weight is off by 2^-46 y ln 2 of itself, y its logarithm to base 2 (0 for 1), and by
# 2^-44.4 for Taylor terms and low words: 2^-41 from 2^-43 on.  A group's is the product of two of them: the first
# value's and, relative to that, the others'.  Cutting a step to 2^-63 takes 2^-41 of it where it
# is 2^-22 or more: 2^-39.4 in all.  Where it is less, what is cut is 2^-74 a word, which the
# program takes off.
@pytest.mark.parametrize("most", [1, 30, 16000])
@pytest.mark.parametrize("top", ["0x4d1f", "0x4d00", "0x3c00", "0x0400", "0x7bff"])
@pytest.mark.parametrize("T", ["1", "0.3", "1.7", "100", "0.05", "0.01", "9e-4", "6e-4", "1e-5", "1e4", "1e-30", "inf"])
def test_group_sums(check, T, top, most):
    for seed in range(4):
        worst, total = check(T, top, seed, most)
        assert worst <= 2.0 ** -39
        assert total <= 2.0 ** -39
