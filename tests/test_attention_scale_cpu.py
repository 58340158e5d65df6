"""The softmax scale that prompt attention and the 8-bit decode attention take:
scale log2(e), which the kernels work with, has to be a finite fp32 number."""
import ctypes

import pytest

from .test_kv8_cpu import GOOD, INVALID, WORKSPACE, _cache, _prompt, w4  # noqa: F401 (w4 is a fixture)


@pytest.mark.parametrize("scale,refused", [(2.3e38, False), (2.35e38, False), (2.36e38, True), (2.9e38, True), (3.0e38, True),
                                           (3.3e38, True), (1e-38, False), (1e-45, False), (0.0, True)])
def test_scale(w4, scale, refused):  # noqa: F811
    # calls that run nothing whatever the scale: no query, no workspace
    assert (_prompt(w4, scale=scale, Tq=0) == INVALID) == refused
    c = ctypes.byref(_cache(w4))
    got = w4.lib().w4a8_decode_attention_kv8(GOOD, c, GOOD, GOOD, 1, 8, 200, scale, GOOD, GOOD, 0, None)
    assert got == (INVALID if refused else WORKSPACE)
