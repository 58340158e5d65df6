"""Decode attention on long tables of the 8-bit cache (the split kernel and its merge,
the only ones that use a workspace) on another stream, captured in a graph, and with one
workspace kept for calls of other shapes."""
import numpy as np
import pytest
import torch

from .test_kv8_gpu import _cu, _i32, _random_cache, _table, _verify_decode

pytestmark = pytest.mark.gpu
GUARD = 8192


@pytest.fixture(scope="module")
def w4():
    from int4_weight_quantized_gb300.build import build
    build()
    import int4_weight_quantized_gb300 as w4
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return w4


def _case(w4, D, Hq, H, T, lens, seed):
    P = sum(-(-n // T) for n in lens) + 2
    table = _table(lens, T, P, seed, extra=4096 // T + 1)
    q = torch.randn((len(lens), Hq, D), generator=torch.Generator().manual_seed(seed)).half()
    return q, _random_cache(w4, P, H, T, D, seed), table


def _bytes(w4, q, cache, table):
    P, H, T, D = cache.k_codes.shape
    return w4.lib().w4a8_decode_attention_kv8_workspace_bytes(q.shape[0], q.shape[1], H, D, T, table.shape[1])


@pytest.mark.parametrize("lens", [[5000, 70], [30000], [12000, 0, 9000, 1]])
def test_another_stream_and_a_graph(w4, lens):
    T, D = 32, 128
    q, cache, table = _case(w4, D, 8, 1, T, lens, seed=1)
    qd, td, ld = q.cuda(), _i32(table), _i32(lens)
    want = w4.decode_attention_kv8(qd, cache, td, ld)
    _verify_decode(want, q, cache, table, lens, T)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [w4.decode_attention_kv8(qd, cache, td, ld) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(x, want) for x in got)
    ws = torch.empty(_bytes(w4, q, cache, td), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    new = torch.randn((len(lens), 1, D), generator=torch.Generator().manual_seed(2)).half().cuda()
    free = sorted(set(range(cache.k_codes.shape[0])) - {int(p) for row, n in zip(table, lens) for p in row[:-(-n // T)]})
    for b, n in enumerate(lens):                      # a page for the token that comes
        if n % T == 0:
            td[b, n // T] = free.pop()
    one, out, more = _cu([1] * len(lens)), torch.empty_like(want), ld.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.kv8_append(cache, new, new, td, ld, one)
        torch.add(ld, 1, out=more)
        w4.decode_attention_kv8(qd, cache, td, more, out=out, workspace=ws)
    copy = w4.KV8Cache(*(t.clone() for t in cache))
    for fill in (0, 255):
        ws.fill_(fill)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        if fill == 0:
            w4.kv8_append(copy, new, new, td, ld, one)
        for a, b in zip(cache, copy):                 # the same token again changes nothing
            assert torch.equal(a, b)
        assert torch.equal(out, w4.decode_attention_kv8(qd, copy, td, ld + 1))
    assert w4.get_device_status() == 0


SHAPES = [(128, 16, 2, 128, [60000]), (64, 16, 1, 16, [0, 0, 0]), (64, 8, 8, 32, [300, 4097, 0, 1]), (256, 32, 2, 64, [9000, 1, 20000]),
          (128, 8, 8, 32, [int(x) for x in np.random.RandomState(1).randint(0, 6000, 40)]), (128, 4, 4, 16, [5000] * 3),
          (64, 3, 1, 64, [100000, 0]), (256, 8, 1, 128, [4097]), (128, 16, 2, 128, [60001])]


@pytest.mark.parametrize("fill", [0, 255])
def test_one_workspace_for_calls_of_other_shapes(w4, fill):
    # what an earlier call left there (parts, lists of parts) and what was there before any
    # call (255: every word a NaN) do not matter, and nothing behind its bytes is written
    cases = [_case(w4, *s, seed=i) for i, s in enumerate(SHAPES)]
    need = [_bytes(w4, q, c, t) for q, c, t in cases]
    assert min(need) > 0
    buf = torch.full((max(need) + GUARD,), fill, dtype=torch.uint8, device="cuda")
    fresh = [w4.decode_attention_kv8(q.cuda(), c, _i32(t), _i32(s[4])) for (q, c, t), s in zip(cases, SHAPES)]
    for (q, c, t), s, out in zip(cases, SHAPES, fresh):
        _verify_decode(out, q, c, t, s[4], s[3])
        assert all(bool((out[b] == 0).all()) for b, n in enumerate(s[4]) if n == 0)
    for turn in (range(len(cases)), reversed(range(len(cases)))):
        for i in turn:
            (q, c, t), s = cases[i], SHAPES[i]
            buf[need[i]:].fill_(0xA5)
            got = w4.decode_attention_kv8(q.cuda(), c, _i32(t), _i32(s[4]), workspace=buf[:need[i]])
            assert torch.equal(got, fresh[i])
            assert bool((buf[need[i]:] == 0xA5).all())
            if fill:
                buf.fill_(fill)
    assert w4.get_device_status() == 0
