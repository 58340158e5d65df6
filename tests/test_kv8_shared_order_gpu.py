"""Decode attention over shared pages right behind the kernels that write what it reads:
lengths, table, keys and queries of every step are new, step after step without a pause, and
the kernel of own tokens runs beside the kernel of the shared ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    from int4_weight_quantized_gb300.build import build
    build()
    import int4_weight_quantized_gb300 as w4
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return w4


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows,H,D", [(3, 1, 64), (40, 2, 128), (7, 1, 256)])
def test_steps_in_a_row(w4, rows, H, D):
    """Growth, writing and attention of 24 steps in one graph, each step's output kept, against the same steps one by one."""
    T, steps, prompt, maxp = 16, 24, 400, 700      # (tables too long for the kernel of short caches)
    g = torch.Generator().manual_seed(rows)
    k, v = (torch.randn((prompt, H, D), generator=g).half().cuda() for _ in range(2))
    new = torch.randn((2, steps, rows, H, D), generator=g).half().cuda()
    q = torch.randn((steps, rows, 4 * H, D), generator=g).half().cuda()
    cu, shared, one = _i32([0, rows]), _i32([prompt // T] * rows), _i32([1] * rows)
    P = prompt // T + rows * (steps // T + 2)

    def begin():
        cache = w4.kv8_cache(P, H, T, D)
        table = torch.full((rows, maxp), -1, dtype=torch.int32, device="cuda")
        table[:, :prompt // T] = _i32(list(range(prompt // T)))
        w4.kv8_append(cache, k, v, table[:1].contiguous(), _i32([0]), _i32([0, prompt]))
        return cache, table, _i32([prompt] * rows)

    def step(i, cache, table, lens, sync):
        start, at, _, _ = w4.kv8_extend(cache, table, lens, one, rows)
        w4.kv8_append(cache, new[0, i], new[1, i], table, start, at)
        if sync:
            torch.cuda.synchronize()
        out = w4.decode_attention_kv8_shared(q[i], cache, table, lens, cu, shared)
        if sync:
            torch.cuda.synchronize()
        return out

    state = begin()
    want = [step(i, *state, True) for i in range(steps)]
    whole = w4.decode_attention_kv8(q[-1], *state)
    assert float((whole.float() - want[-1].float()).abs().max()) <= float(max(v.abs().max(), new[1].abs().max())) * 2.0 ** -9
    kept = begin()
    state = begin()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [step(i, *state, False) for i in range(steps)]
    for _ in range(4):
        for x, y in zip((*state[0], *state[1:]), (*kept[0], *kept[1:])):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert w4.get_device_status() == 0


def test_a_workspace_is_left_for_the_next_call(w4):
    """Whatever its first word is before a call, and 0 behind it."""
    T, D = 16, 128
    cache = w4.kv8_cache(200, 1, T, D)
    for x in cache:
        x.copy_(torch.rand(x.shape, device="cuda") * 100 if x.dtype == torch.int8 else torch.rand(x.shape, device="cuda"))
    table, lens = torch.arange(200, dtype=torch.int32, device="cuda").repeat(2, 3), _i32([3000, 2500])
    q = torch.randn((2, 8, D), device="cuda").half()
    need = w4.lib().w4a8_decode_attention_kv8_shared_workspace_bytes(2, 1, 8, 1, D, T, 600)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = w4.decode_attention_kv8_shared(q, cache, table, lens, _i32([0, 2]), _i32([100, 90]), workspace=ws)
    for word in (-1, 0x6b76385f62656775, 0):
        ws.view(torch.int64)[0] = word
        assert torch.equal(w4.decode_attention_kv8_shared(q, cache, table, lens, _i32([0, 2]), _i32([100, 90]), workspace=ws), want)
        assert int(ws.view(torch.int64)[0]) == 0
    assert w4.get_device_status() == 0
