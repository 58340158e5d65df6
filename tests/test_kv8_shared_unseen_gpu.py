"""Decode attention over shared pages where a group's rows see different parts of them:
what a row does not see changes nothing for it, whatever the others see there (a token
whose values were infinite has an infinite scale)."""
import pytest
import torch

from .test_kv8_gpu import _verify_decode
from .test_kv8_shared_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    from int4_weight_quantized_gb300.build import build
    build()
    import int4_weight_quantized_gb300 as w4
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return w4


@pytest.fixture(params=[0, 5000], ids=["narrow", "wide"], autouse=True)
def wide(request):
    """Tables with so many more tokens' entries: short ones may take another kernel."""
    Case.wide = request.param


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("D,Hq,H,T", [(64, 8, 1, 16), (64, 4, 2, 128), (128, 16, 1, 32), (128, 8, 2, 64), (256, 8, 1, 64), (256, 3, 3, 128)])
def test_a_block_that_others_see(w4, D, Hq, H, T, value):
    # rows 1, 3, 5 and 6 end, or leave the others' way, before the block (row 3 two blocks before it); the others see it
    tok, pages = 304, 512 // T
    page, blk = tok // T, tok % T // 16
    c = Case(w4, D, Hq, H, T, [[(pages, 512 + 9), (page, page * T + 20 if T < 64 else page * T), (pages, 512), (pages, tok - 20), (pages, tok + 1)], [(2, 2 * T + 3)]],
             alone=[70], seed=D + T)
    sees, others = [0, 2, 4], [1, 3, 5, 6]
    want = c.check(w4)
    page = int(c.whole[0, page])
    for scale in (c.cache.v_scale, c.cache.k_scale):
        kept = scale.clone()
        scale[page, :, blk] = value
        out = c.run(w4)
        assert torch.equal(out[others], want[others])
        _verify_decode(out[others], c.q[others], c.cache, c.whole[others], [c.lens[b] for b in others], T)
        scale.copy_(kept)
    # (what sees an infinite value has none of its own: nothing finite is claimed of it)
    assert torch.equal(c.run(w4)[sees], want[sees])
    assert w4.get_device_status() == 0


def test_a_written_infinity(w4):
    """The same by the writer: a prompt's token whose V is infinite, behind a shorter row's end."""
    T, H, D = 16, 1, 128
    cache = w4.kv8_cache(64, H, T, D)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((400, H, D), generator=g).half().cuda() for _ in range(2))
    v[300, 0, 5] = float("inf")
    width = 25 + Case.wide // T
    table = torch.full((2, width), -1, dtype=torch.int32)
    table[0, :25] = torch.arange(25)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")      # noqa: E731
    table = table.cuda()
    w4.kv8_append(cache, k, v, table, i32([0, 0]), i32([0, 400, 400]))
    q = torch.randn((2, 4, D), generator=g).half().cuda()
    lens, both, own = i32([400, 250]), i32([0, 2]), table.clone()
    own[1] = table[0]
    got = w4.decode_attention_kv8_shared(q, cache, table, lens, both, i32([25, 25]))
    want = w4.decode_attention_kv8(q, cache, own, lens)
    assert bool(torch.isfinite(want[1]).all()) and bool(torch.isfinite(got[1]).all())
    # both are attention of the same codes, each output rounded to fp16 and its weights before that
    assert float((got[1].float() - want[1].float()).abs().max()) <= float(v[:250].abs().max()) * 2.0 ** -9
    assert w4.get_device_status() == 0
