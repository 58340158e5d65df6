"""Decode attention over shared pages where a few rows have long parts of their own: there
the warps of a CTA join their parts on chip, and a pair's parts are those of warps, of
whole CTAs and of warps again.  Against attention over each sequence's own keys in 64 bits
with the derived bound."""
import pytest
import torch

from .test_kv8_shared_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    from int4_weight_quantized_gb300.build import build
    build()
    import int4_weight_quantized_gb300 as w4
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return w4


@pytest.fixture(autouse=True)
def wide():
    Case.wide = 5000


def _joined(c, Hq, H, D):
    """How many parts of whole CTAs there are, by the kernel's rule: ranges of U units of 32 tokens, 8 to a CTA."""
    grid = 152 if D == 256 or Hq // H > 8 else 304
    own = [-(-max(n - s * c.T, 0) // 32) for n, s in zip(c.lens, c.shared)]
    U = sum(own) * H
    C = min(grid * 8, U) // 8 * 8
    if C < 16 * len(own) * H:
        return 0
    ends, at = [], 0
    for n in own:
        for _ in range(H):
            ends.append((at, at + n))
            at += n
    return sum(any(lo <= k * U // C and (k + 8) * U // C <= hi for lo, hi in ends) for k in range(0, C, 8))


# (own lengths of the rows of one group, of rows in none)
ROWS = [([40000], []), ([3000, 9000], []), ([20011, 0, 7777], [5000]), ([1, 33000, 31, 12345], []), ([], [17001]), ([700, 700, 30000], [1, 64])]


@pytest.mark.parametrize("shared", [0, 300])
@pytest.mark.parametrize("own,alone", ROWS)
@pytest.mark.parametrize("D,Hq,H,T", [(64, 8, 1, 16), (64, 16, 1, 64), (128, 6, 2, 32), (128, 11, 1, 128), (256, 8, 1, 64), (256, 16, 1, 128)])
def test_long_own_parts(w4, D, Hq, H, T, own, alone, shared):
    pages = -(-shared // T)
    c = Case(w4, D, Hq, H, T, [[(pages, pages * T + n) for n in own]], alone=alone, seed=D + T)
    assert _joined(c, Hq, H, D) > 0
    out = c.check(w4)
    assert torch.equal(out, c.run(w4))
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("D,Hq,H", [(64, 32, 4), (128, 4, 4), (256, 6, 3)])
def test_many_heads(w4, D, Hq, H):
    c = Case(w4, D, Hq, H, 64, [[(10, 640 + n) for n in (9000, 4001)], [(3, 192 + 6000)]], alone=[5000], seed=D)
    assert _joined(c, Hq, H, D) > 0
    c.check(w4)
    assert w4.get_device_status() == 0


def test_in_a_graph(w4):
    """Lengths are read on the device: one graph with parts of whole CTAs and without."""
    c = Case(w4, 128, 8, 1, 32, [[(20, 640 + n) for n in (30000, 8000)]], seed=1)
    args = [c.q.cuda(), c.cache, torch.from_numpy(c.table).cuda(), *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (c.lens, c.cu, c.shared))]
    out = torch.empty_like(args[0])
    need = w4.lib().w4a8_decode_attention_kv8_shared_workspace_bytes(2, 1, 8, 1, 128, 32, c.table.shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.decode_attention_kv8_shared(*args, out=out, workspace=ws)
    whole = c.lens
    for lens in (whole, [700, 640 + 17], whole, [640 + 30000, 3]):
        args[3].copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        c.lens = lens
        c.check(w4, out)
    assert w4.get_device_status() == 0
