"""What the build does where the Python module of the newer operators cannot be
built: the C library, which needs neither Python nor torch, is built all the same."""
import json
import os

import pytest

from int4_weight_quantized_gb300 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A small source tree of its own; compiled with the real compilers."""
    src, out = tmp_path / "csrc", tmp_path / "_build"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (src / "binding.cpp").write_text("#error no headers here\n")
    for name, value in (("CSRC", str(src)), ("OUT_DIR", str(out)), ("LIB", str(out / "libw4a8.so")), ("EXT", str(out / "_w4a8.so")),
                        ("STAMP", str(out / "_w4a8.json"))):
        monkeypatch.setattr(B, name, value)
    return tmp_path


def _counted(monkeypatch, name, value=None):
    calls, was = [], getattr(B, name)
    monkeypatch.setattr(B, name, lambda *a: (calls.append(a), value if value is not None else was(*a))[1])
    return calls


def _module(obj):
    with open(B.EXT, "w") as f:
        f.write("module")


def test_the_library_is_built_where_the_module_does_not_compile(tree, monkeypatch):
    cu, cpp = _counted(monkeypatch, "_compile"), _counted(monkeypatch, "_compile_binding")
    with pytest.warns(UserWarning, match="was not built"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.EXT)
    assert "no headers here" in B.binding_error()
    assert (len(cu), len(cpp)) == (1, 1)
    assert B.build() == B.LIB and (len(cu), len(cpp)) == (1, 1)       # nothing is tried again
    (tree / "csrc" / "binding.cpp").write_text("int two() { return 2; }\n")
    os.utime(tree / "csrc" / "binding.cpp", (os.path.getmtime(B.STAMP) + 5,) * 2)
    monkeypatch.setattr(B, "_link_binding", _module)
    B.build()
    assert os.path.exists(B.EXT) and B.binding_error() == "" and len(cpp) == 2


def test_the_library_stays_where_the_module_does_not_link(tree, monkeypatch):
    _counted(monkeypatch, "_compile_binding", "binding.o")
    monkeypatch.setattr(B, "_link_binding", _module)
    B.build()
    assert os.path.exists(B.EXT)

    def fails(obj):
        raise RuntimeError("link failed: cannot find -lc10_cuda")
    monkeypatch.setattr(B, "_link_binding", fails)
    with pytest.warns(UserWarning, match="c10_cuda"):
        assert B.build(force=True) == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.EXT)        # no module of an older build stays
    assert "c10_cuda" in B.binding_error()


def test_another_torch_gets_a_module_of_its_own(tree, monkeypatch):
    cu = _counted(monkeypatch, "_compile")
    cpp = _counted(monkeypatch, "_compile_binding", "binding.o")
    monkeypatch.setattr(B, "_link_binding", _module)
    B.build()
    assert B.build() == B.LIB and (len(cu), len(cpp)) == (1, 1)
    monkeypatch.setattr(B, "_torch_id", lambda: "another torch")
    B.build()
    assert (len(cu), len(cpp)) == (1, 2)                              # the library is not touched
    assert json.load(open(B.STAMP)) == {"torch": "another torch", "error": ""}
    os.remove(B.EXT)
    B.build()
    assert len(cpp) == 3 and os.path.exists(B.EXT)


def test_builds_side_by_side_note_their_module(tree, monkeypatch):
    # as parallel test workers do: nobody takes the file that another is writing
    from concurrent.futures import Future, ThreadPoolExecutor
    os.makedirs(B.OUT_DIR)
    done = Future()
    done.set_result("binding.o")
    monkeypatch.setattr(B, "_link_binding", _module)
    with ThreadPoolExecutor(8) as ex:
        for f in [ex.submit(B._finish_binding, done) for _ in range(200)]:
            f.result()
    assert json.load(open(B.STAMP))["error"] == "" and os.listdir(B.OUT_DIR) in (["_w4a8.so", "_w4a8.json"], ["_w4a8.json", "_w4a8.so"])


def test_a_library_that_does_not_compile_is_an_error(tree, monkeypatch):
    (tree / "csrc" / "one.cu").write_text("#error broken\n")
    with pytest.raises(RuntimeError, match="broken"):
        B.build()
    assert not os.path.exists(B.LIB)


def test_a_call_says_why_the_module_is_missing(monkeypatch, tmp_path):
    import int4_weight_quantized_gb300 as w4
    monkeypatch.setattr(w4, "_native", None)
    monkeypatch.setattr(w4, "lib", lambda: None)
    monkeypatch.setattr(w4, "_HERE", str(tmp_path))
    monkeypatch.setattr(B, "binding_error", lambda: "no c10_cuda")
    with pytest.raises(RuntimeError, match="no c10_cuda"):
        w4._ext()
