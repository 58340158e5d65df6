"""The serving example on the GPU: prompt, decode, fork, prefix, compaction."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_serve_kv8():
    from int4_weight_quantized_gb300.build import build
    build()
    spec = importlib.util.spec_from_file_location("serve_kv8", os.path.join(ROOT, "examples", "serve_kv8.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    lines = []
    got = m.main(layers=2, steps=4, say=lines.append)
    assert got["forked_equal"] and got["forked_other"] and got["compacted_equal"] and got["front"]
    assert got["status"] == 0
    assert len(lines) == 5
    # 8-bit rounding of keys and values moves the logits by its noise only
    assert float(got["near"].min()) > 0.98
