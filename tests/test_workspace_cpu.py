"""A caller's workspace that counts more bytes than it has (an expanded tensor) is
refused before anything else is looked at or launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def w4():
    from int4_weight_quantized_gb300.build import build
    build()
    import int4_weight_quantized_gb300 as w4
    return w4


BAD = [torch.empty(1, dtype=torch.uint8).expand(1 << 30), torch.empty((64, 64), dtype=torch.uint8)[:, :32]]


@pytest.mark.parametrize("ws", BAD, ids=["expanded", "strided"])
def test_newer_operators(w4, ws):
    cache, table, lens = w4.kv8_cache(2, 1, 16, 64, device="cpu"), torch.zeros((1, 300), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((1, 8, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="workspace"):
        w4.decode_attention_kv8(q, cache, table, lens, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        w4.kv8_compact(cache, table, lens, workspace=ws)


@pytest.mark.parametrize("ws", BAD, ids=["expanded", "strided"])
def test_older_operators(w4, ws, monkeypatch):
    # (their other checks would refuse tensors of the CPU first)
    monkeypatch.setattr(w4, "_need", lambda *a: None)
    monkeypatch.setattr(w4, "_stream", lambda: None)
    M, N, K = 512, 256, 64
    x, packed, scales = torch.zeros((M, K), dtype=torch.float16), torch.zeros((N, K // 2), dtype=torch.uint8), torch.zeros((N, K // 32), dtype=torch.float16)
    codes, sx = torch.zeros((M, K), dtype=torch.int8), torch.zeros((M, K // 32))
    kc = torch.zeros((1, 1, 64, 64), dtype=torch.float16)
    for call in (lambda: w4.linear(x, packed, scales, workspace=ws),
                 lambda: w4.linear_gated(x, packed, scales, workspace=ws),
                 lambda: w4.linear_q8(codes, sx, packed, scales, workspace=ws),
                 lambda: w4.decode_attention(torch.zeros((1, 8, 64), dtype=torch.float16), kc, kc, torch.zeros(1, dtype=torch.int32), workspace=ws),
                 lambda: w4.debug_block_dots(x, packed, scales, workspace=ws)):
        with pytest.raises(ValueError, match="workspace"):
            call()


def test_a_workspace_counts_its_bytes(w4):
    p, n = w4._workspace(None)
    assert not p.value and n == 0
    t = torch.empty(512, dtype=torch.uint8)
    p, n = w4._workspace(t[16:])
    assert p.value == t.data_ptr() + 16 and n == 496
