"""The prompt kernel's ring of K and V tiles (csrc/prompt_ring.h), compiled for the
CPU: the items' order, and that nobody waits by parity for an item of a slot
whose item before may still be on its way."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# by head dimension: row tiles per CTA, slots to a tile, next S ahead, P beside S
FORMS = {64: (1, 1, True, True), 128: (2, 1, False, False), 256: (1, 2, True, False)}


@pytest.fixture(scope="module")
def X(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("ring") / "prompt_ring.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-static-libubsan", "-I", os.path.join(ROOT, "int4_weight_quantized_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "prompt_ring_check.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def _loads(steps, k_first):
    """The tiles in the order in which the copying thread loads them."""
    order = [("K", 0)]
    for j in range(steps):
        nxt = [("K", j + 1)] if j + 1 < steps else []
        order += nxt + [("V", j)] if k_first else [("V", j)] + nxt
    return order


def _products(n, ns_ahead):
    """The products in the order of issue: (S or O, row tile, step); n: steps of each row tile."""
    if len(n) == 1:
        out = [("S", 0, 0)]
        for j in range(n[0]):
            out += [("S", 0, j + 1)] if j + 1 < n[0] else []
            out += [("O", 0, j)]
        return out
    out = [("S", i, 0) for i in range(2) if n[i]]
    for j in range(max(n)):
        for i in range(2):
            if j < n[i]:
                out += [("O", i, j)] + ([("S", i, j + 1)] if j + 1 < n[i] else [])
    return out


def _steps(nq):
    for m in range(1, 24):
        if nq == 1:
            yield [m]
        else:
            # the second tile's tokens come behind the first one's, or there are none
            yield from ([m, 0], [m, m], [m, m + 1], [max(m - 2, 0), m])


def test_items_are_loaded_in_order(X):
    for nq, spt, k_first, _ in FORMS.values():
        for steps in range(1, 40):
            for t, (what, j) in enumerate(_loads(steps, k_first)):
                assert t == (X.k_tile(j, k_first) if what == "K" else X.v_tile(j, steps, k_first))
    for i in range(200):
        assert X.slot_of(i) == i % X.slots() and X.parity_of(i) == i // X.slots() % 2


def _late(X, D, after):
    """Waits of the softmax warps for V(j) that may find their slot's barrier a phase behind: (wait, steps, row tile, j)."""
    nq, spt, k_first, beside = FORMS[D]
    bad = set()
    for n in _steps(nq):
        steps = max(n)
        order, issued = _loads(steps, k_first), _products(n, k_first)

        def landed(*products):
            # a product's completion comes behind those of all that were issued before
            done = issued[:max((issued.index(p) + 1 for p in products if p in issued), default=0)]
            return {("K" if what == "S" else "V", j) for what, _, j in done}
        for i in range(nq):
            for j in range(n[i]):
                before = [("S", i, j - 1)] + ([("O", i, j - 2)] if beside else [])       # waited for in the step before
                scores = before + [("S", i, j)]
                know = {"screen": landed(*(scores + [("O", i, j - 1)] if after else before)),
                        "zero": landed(*(scores + ([("O", i, j - 1)] if beside else [])))}
                for h in range(spt):
                    item = X.v_tile(j, steps, k_first) * spt + h
                    assert order[item // spt] == ("V", j)
                    prev = item - X.slots()
                    if prev < 0:
                        continue
                    for wait in know:
                        # the rows past the keys' end are zeroed in the last tile only
                        if order[prev // spt] not in know[wait] and (wait == "screen" or j == steps - 1):
                            bad.add((wait, tuple(n), i, j))
    return bad


@pytest.mark.parametrize("D", [64, 128, 256])
def test_no_wait_is_a_phase_behind(X, D):
    assert not _late(X, D, bool(X.screen_after_products(FORMS[D][1])))


def test_the_model_sees_a_wait_that_is_missing(X):
    # two slots to a tile, V looked through before S of the same step
    late = _late(X, 256, False)
    assert ("screen", (4,), 0, 2) in late and ("screen", (4,), 0, 3) in late
    assert all(w == "screen" for w, *_ in late)


def test_a_slot_is_not_loaded_again_before_its_users_are_done(X):
    # V(j)'s slots are given back by the last product that reads them, which
    # needs the weights of step j: no warp that still has to look at V(j) finds a later item
    for nq, spt, k_first, _ in FORMS.values():
        for n in _steps(nq):
            issued = _products(n, k_first)
            for i in range(nq):
                for j in range(n[i]):
                    last = max(x for x, (w, _, s) in enumerate(issued) if w == "O" and s == j)
                    assert last >= issued.index(("O", i, j))
