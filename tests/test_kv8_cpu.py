"""Prompt attention and the 8-bit cache without a GPU: refusals of bad shapes,
strides and pointers before any device work, workspace sizes, and the
binding's own checks."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def w4():
    from int4_weight_quantized_gb300.build import build
    build()
    import int4_weight_quantized_gb300 as w4
    _declare(w4.lib())
    return w4


INVALID, MISALIGNED, WORKSPACE, UNSUPPORTED = 1, 2, 7, 6
P = ctypes.c_void_p
GOOD, ODD, NULL = 4096, 4097, 0


class _CKv8(ctypes.Structure):
    _fields_ = [(n, P) for n in ("k_codes", "k_scale", "v_codes", "v_scale")] + [
        (n, ctypes.c_int) for n in ("pages", "heads", "page_tokens", "dim")]


def _declare(L):
    """The C signatures of include/w4a8.h that the tests call with plain numbers for pointers."""
    i, sz, ll, f, C = ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_float, ctypes.POINTER(_CKv8)
    for name, args in (("prompt_attention", [P, P, P, ll, ll, ll, P, P, i, i, i, i, i, i, i, f, P, P]),
                       ("kv8_append", [C, P, P, ll, ll, P, P, P, i, i, i, P]), ("kv8_read", [C, P, P, i, i, i, P, P, P]),
                       ("decode_attention_kv8", [P, C, P, P, i, i, i, f, P, P, sz, P]),
                       ("kv8_free_pages", [P, P, i, i, i, i, P, P, P]), ("kv8_fork", [C, P, P, P, P, P, i, i, i, P]),
                       ("kv8_compact", [C, P, P, i, i, P, P, P, sz, P])):
        getattr(L, "w4a8_" + name).argtypes = args


def _prompt(w4, q=GOOD, k=GOOD, v=GOOD, ld_q=2048, ld_k=256, ld_v=256, cu_q=GOOD, cu_k=GOOD, B=1, Tq=8, Tk=8, Hq=8, Hkv=1,
            D=256, causal=1, scale=0.0625, out=GOOD):
    return w4.lib().w4a8_prompt_attention(q, k, v, ld_q, ld_k, ld_v, cu_q, cu_k, B, Tq, Tk, Hq, Hkv, D, causal, scale, out, None)


@pytest.mark.parametrize("bad", [dict(D=96), dict(Hkv=3), dict(Hkv=0), dict(Hq=0), dict(B=0), dict(B=65536), dict(Tq=-1),
                                 dict(Tk=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                 dict(scale=float("inf")), dict(ld_q=2047), dict(ld_q=2044), dict(ld_q=1024), dict(ld_k=128),
                                 dict(ld_v=260), dict(ld_k=1 << 39), dict(Hq=129, ld_q=129 * 256),
                                 dict(Tq=2 ** 31 - 1, Hkv=8, Hq=8, ld_k=2048, ld_v=2048)])
def test_prompt_attention_refuses_shapes(w4, bad):
    assert _prompt(w4, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(q=GOOD + 8), dict(k=NULL), dict(v=ODD), dict(out=GOOD + 2), dict(cu_q=GOOD + 2),
                                 dict(cu_k=NULL)])
def test_prompt_attention_refuses_pointers(w4, bad):
    assert _prompt(w4, **bad) == MISALIGNED


def _cache(w4, **kw):
    f = dict(k_codes=GOOD, k_scale=GOOD, v_codes=GOOD, v_scale=GOOD, pages=10, heads=2, page_tokens=32, dim=128)
    f.update(kw)
    return _CKv8(*(f[n] for n, _ in _CKv8._fields_))


BAD_CACHES = [(dict(pages=0), INVALID), (dict(heads=0), INVALID), (dict(page_tokens=8), INVALID), (dict(page_tokens=48), INVALID),
              (dict(page_tokens=256), INVALID), (dict(dim=96), INVALID), (dict(k_codes=NULL), MISALIGNED),
              (dict(v_codes=GOOD + 8), MISALIGNED), (dict(k_scale=GOOD + 4), MISALIGNED), (dict(v_scale=NULL), MISALIGNED)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_cache_call_refuses_a_bad_cache(w4, bad, status):
    L, c = w4.lib(), ctypes.byref(_cache(w4, **bad))
    big = 1 << 40
    assert L.w4a8_kv8_append(c, GOOD, GOOD, 256, 256, GOOD, GOOD, GOOD, 1, 4, 8, None) == status
    assert L.w4a8_kv8_read(c, GOOD, GOOD, 1, 4, 8, GOOD, GOOD, None) == status
    assert L.w4a8_decode_attention_kv8(GOOD, c, GOOD, GOOD, 1, 8, 4, 0.1, GOOD, GOOD, big, None) == status
    assert L.w4a8_kv8_fork(c, GOOD, GOOD, GOOD, GOOD, GOOD, 1, 4, 4, None) == status
    assert L.w4a8_kv8_compact(c, GOOD, GOOD, 4, 4, GOOD + 4096, GOOD, GOOD, big, None) == status
    assert L.w4a8_kv8_append(None, GOOD, GOOD, 256, 256, GOOD, GOOD, GOOD, 1, 4, 8, None) == INVALID


def test_cache_calls_refuse_arguments(w4):
    L, c, big = w4.lib(), ctypes.byref(_cache(w4)), 1 << 40

    def append(k=GOOD, v=GOOD, ld_k=256, ld_v=256, table=GOOD, start=GOOD, cu=GOOD, B=1, maxp=4, n=8):
        return L.w4a8_kv8_append(c, k, v, ld_k, ld_v, table, start, cu, B, maxp, n, None)
    for bad in (dict(ld_k=255), dict(ld_v=128), dict(B=0), dict(B=65536), dict(maxp=0), dict(maxp=1 << 27), dict(n=-1)):
        assert append(**bad) == INVALID, bad
    for bad in (dict(k=GOOD + 8), dict(v=NULL), dict(table=ODD), dict(start=NULL), dict(cu=GOOD + 1)):
        assert append(**bad) == MISALIGNED, bad

    def decode(q=GOOD, table=GOOD, lens=GOOD, B=1, Hq=8, maxp=4, scale=0.1, out=GOOD, ws=GOOD, n=big):
        return L.w4a8_decode_attention_kv8(q, c, table, lens, B, Hq, maxp, scale, out, ws, n, None)
    for bad in (dict(Hq=7), dict(Hq=34), dict(Hq=0), dict(scale=0.0), dict(scale=float("nan")), dict(B=0), dict(maxp=0)):
        assert decode(**bad) == INVALID, bad
    for bad in (dict(q=GOOD + 8), dict(out=NULL), dict(table=ODD), dict(lens=NULL)):
        assert decode(**bad) == MISALIGNED, bad
    need = L.w4a8_decode_attention_kv8_workspace_bytes(1, 8, 2, 128, 32, 200)
    assert decode(maxp=200, n=need - 1) == WORKSPACE and decode(maxp=200, ws=NULL) == WORKSPACE and decode(maxp=200, ws=GOOD + 4) == WORKSPACE

    assert L.w4a8_kv8_read(c, GOOD, GOOD, 1, 4, -1, GOOD, GOOD, None) == INVALID
    assert L.w4a8_kv8_read(c, GOOD, GOOD, 1, 4, 8, GOOD + 8, GOOD, None) == MISALIGNED
    assert L.w4a8_kv8_free_pages(GOOD, GOOD, 4, 4, 24, 10, GOOD, GOOD, None) == INVALID
    assert L.w4a8_kv8_free_pages(GOOD, GOOD, 4, 4, 32, 0, GOOD, GOOD, None) == INVALID
    assert L.w4a8_kv8_free_pages(GOOD, GOOD, 4, 4, 32, 10, ODD, GOOD, None) == MISALIGNED
    assert L.w4a8_kv8_free_pages(GOOD, GOOD, 4, 4, 32, 12582913, GOOD, GOOD, None) == UNSUPPORTED
    assert L.w4a8_kv8_fork(c, GOOD, GOOD, GOOD, GOOD, GOOD, 65536, 4, 4, None) == INVALID
    assert L.w4a8_kv8_fork(c, GOOD, GOOD, GOOD, NULL, GOOD, 1, 4, 4, None) == MISALIGNED
    assert L.w4a8_kv8_compact(c, GOOD, GOOD, 4, 4, GOOD, GOOD, GOOD, big, None) == INVALID          # in place
    assert L.w4a8_kv8_compact(c, GOOD, GOOD, 4, 4, GOOD + 4096, GOOD, GOOD, 16, None) == WORKSPACE
    huge = ctypes.byref(_cache(w4, pages=12582913))
    assert L.w4a8_kv8_compact(huge, GOOD, GOOD, 4, 4, GOOD + 4096, GOOD, GOOD, big, None) == UNSUPPORTED


def test_workspace_sizes(w4):
    L = w4.lib()
    ws = L.w4a8_decode_attention_kv8_workspace_bytes
    assert ws(1, 8, 1, 96, 32, 4) == 0 and ws(1, 8, 3, 128, 32, 4) == 0 and ws(1, 32, 1, 128, 32, 4) == 0
    assert ws(0, 8, 1, 128, 32, 4) == 0 and ws(1, 8, 1, 128, 20, 4) == 0
    assert ws(1, 8, 1, 128, 16, 256) == 0 and ws(500, 8, 1, 128, 64, 64) == 0      # one cluster a pair: no parts
    assert ws(1, 8, 1, 128, 16, 257) > 0 and ws(500, 8, 1, 128, 64, 65) > 0
    assert ws(64, 32, 8, 128, 32, 4096) == ws(64, 32, 8, 128, 32, 512)        # independent of the length
    assert L.w4a8_kv8_compact_workspace_bytes(0) == 0 and L.w4a8_kv8_compact_workspace_bytes(12582913) == 0
    assert L.w4a8_kv8_compact_workspace_bytes(100) >= 4 * (100 + 2 * 51 + 1)


def test_status_string(w4):
    assert w4.lib().w4a8_status_string(8) not in (b"unknown status", b"")
    assert w4.STATUS[8] == "W4A8_ERR_PAGE"


def test_binding_refuses_tensors(w4):
    cpu = torch.zeros((4, 8, 64), dtype=torch.float16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        w4.prompt_attention(cpu, cpu, cpu, cu)
    with pytest.raises(TypeError):
        w4.decode_attention_kv8(cpu, w4.kv8_cache(2, 1, 16, 64, device="cpu"), cu[None], cu)
    with pytest.raises(TypeError):
        w4.kv8_append(w4.kv8_cache(2, 1, 16, 64, device="cpu"), cpu, cpu, cu[None], cu, cu)
