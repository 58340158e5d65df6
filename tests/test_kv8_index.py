"""The index arithmetic of the paged 8-bit cache and of packed sequences
(csrc/kv8_index.h), compiled for the CPU: offsets past 32 bits, item numbers
that reach every row and block of every sequence once, and work ranges that
cover all units."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def X(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("kv8") / "kv8_index.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-static-libubsan", "-I", os.path.join(ROOT, "int4_weight_quantized_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "kv8_index_check.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    ll = ctypes.c_longlong
    for f in ("code_offset", "scale_offset"):
        getattr(L, f).restype = ctypes.c_size_t
    L.first_unit.argtypes, L.first_unit.restype = [ll, ll, ll], ll
    L.worker_of_unit.argtypes = [ll, ll, ll]
    return L


def test_offsets_pass_32_bits(X):
    assert X.code_offset(3, 8, 5, 64, 17, 128) == ((3 * 8 + 5) * 64 + 17) * 128
    assert X.code_offset(2000000, 8, 7, 128, 127, 256) == ((2000000 * 8 + 7) * 128 + 127) * 256
    assert X.scale_offset(5, 4, 3, 64, 33) == (5 * 4 + 3) * 4 + 2
    assert X.scale_offset(300000000, 8, 7, 128, 127) == (300000000 * 8 + 7) * 8 + 7


def test_bad_pages_are_none(X):
    lo, hi = -2 ** 31, 2 ** 31 - 1
    row = (ctypes.c_int32 * 6)(0, 9, 10, -1, lo, hi)
    assert [X.page_of_row(row, 6, i, 10) for i in range(6)] == [0, 9, -1, -1, -1, -1]
    assert X.page_of_row(row, 6, 5, hi) == -1 and X.page_of_row(row, 6, 2, hi) == 10
    # behind the row's end nothing is read
    assert [X.page_of_row(row, n, i, 10) for n, i in ((0, 0), (1, 1), (6, 6), (6, hi), (6, -1), (6, lo))] == [-1] * 6


def test_held_entries(X):
    for T in (16, 32, 64, 128):
        assert [X.held_entries(n, T, 5) for n in (-2 ** 31, -1, 0, 1, T, T + 1, 4 * T, 5 * T, 5 * T + 1, 2 ** 31 - 1)] == \
            [0, 0, 0, 1, 1, 2, 4, 5, 5, 5]


@pytest.mark.parametrize("unit,slack", [(16, 1), (16, 2), (1, 1), (8, 1), (42, 1), (256, 1)])
def test_items_reach_every_row_once(X, unit, slack):
    rng = random.Random(unit * 10 + slack)
    for _ in range(200):
        lens = [rng.choice([0, 1, unit - 1, unit, unit + 1, rng.randrange(5 * unit + 2)]) for _ in range(rng.randint(1, 40))]
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + max(0, n))
        B = len(lens)
        bases = [X.item_base(cu[b], unit, slack, b) for b in range(B)]
        total = X.item_count(cu[-1], unit, slack, B)
        assert all(x < y for x, y in zip(bases, bases[1:]))         # the search needs them to ascend
        for b in range(B):
            room = (bases[b + 1] if b + 1 < B else total) - bases[b]
            n = cu[b + 1] - cu[b]
            assert room * unit >= n
            if slack == 2 and n:
                for r in range(16):                                  # blocks touched from any place
                    assert X.touched_blocks(r, n) == (r + n - 1) // 16 - r // 16 + 1
                    assert X.touched_blocks(r, n) <= room


def test_work_ranges_cover_all_units(X):
    rng = random.Random(3)
    for _ in range(300):
        C = rng.choice([1, 2, 7, 152, 304])
        U = rng.choice([C, C + 1, 3 * C - 1, rng.randrange(C, 10 ** rng.randint(3, 12) + C)])
        cuts = [X.first_unit(c, U, C) for c in range(C + 1)]
        assert cuts[0] == 0 and cuts[-1] == U
        sizes = [y - x for x, y in zip(cuts, cuts[1:])]
        assert min(sizes) >= 1 and max(sizes) - min(sizes) <= 1
        for u in {0, U - 1, *(rng.randrange(U) for _ in range(50)), *(x for x in cuts[:-1]), *(x - 1 for x in cuts[1:])}:
            c = X.worker_of_unit(u, U, C)
            assert cuts[c] <= u < cuts[c + 1]


@pytest.mark.parametrize("W", [0, 8])
def test_pair_parts_take_every_worker_once(X, W):
    rng = random.Random(17 + W)
    out, seen = (ctypes.c_int * 3)(), set()
    for _ in range(400):
        C = 8 * rng.choice([1, 2, 3, 19, 152, 304])
        sizes = [rng.choice([1, 7, 8, 9, rng.randrange(1, 3000), rng.randrange(1, 10 ** 6)]) for _ in range(rng.randint(1, 6))]
        sizes[0] += max(0, C - sum(sizes))
        U, us = sum(sizes), 0
        cuts = [X.first_unit(c, U, C) for c in range(C + 1)]
        for nt in sizes:
            first, last = X.worker_of_unit(us, U, C), X.worker_of_unit(us + nt - 1, U, C)
            X.pair_parts(first, cuts[first] < us, us + nt, U, C, W, out)
            head, ctas, tail = out
            got = []
            for i in range(head + ctas + tail):
                c = X.part_worker(first, head, ctas, tail, W, i)
                whole = head <= i < head + ctas
                # a group's part is its first worker's; the whole group is inside the pair
                assert not whole or (c % W == 0 and cuts[c] >= us and cuts[c + W] <= us + nt)
                got += range(c, c + W) if whole else [c]
            assert got == list(range(first, last + 1))
            # and every group that is inside the pair has one part
            inside = [k for k in range(C // 8) if W and cuts[8 * k] >= us and cuts[8 * k + 8] <= us + nt]
            assert len(inside) == ctas
            seen.add((head > 0, ctas > 0, tail > 0))
            us += nt
    # without groups every part is a worker's of the head; with them any of the five forms that there are
    assert len(seen) == (1 if W == 0 else 5)
