"""Prompt attention on the GPU against 64-bit attention of each sequence and head."""
import numpy as np
import pytest
import torch

from .attention_ref import attention, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    from int4_weight_quantized_gb300.build import build
    build()
    import int4_weight_quantized_gb300 as w4
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return w4


def _cu(lens):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()


def _inputs(nq, nk, Hq, Hkv, D, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((nq, Hq, D), generator=g) * spread).half()
    k, v = (torch.randn((nk, Hkv, D), generator=g).half() for _ in range(2))
    return q, k, v


def _verify(out, q, k, v, lq, lk, causal, scale=None, what=""):
    Hq, D = q.shape[1], q.shape[2]
    Hkv = k.shape[1]
    aq = ak = 0
    for b, (n, m) in enumerate(zip(lq, lk)):
        see = None
        if causal:
            see = torch.arange(m)[None] <= (torch.arange(n) + m - n)[:, None]
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            ref, bound = attention(q[aq:aq + n, h], k[ak:ak + m, kv], v[ak:ak + m, kv], scale or D ** -0.5, see)
            check(out[aq:aq + n, h], ref, bound, f"{what} sequence {b} ({n} on {m}) head {h}")
        aq, ak = aq + n, ak + m


RAGGED = [1, 2, 17, 0, 128, 129, 33, 300]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (6, 2), (4, 4), (10, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_ragged(w4, D, Hq, Hkv, causal):
    n = sum(RAGGED)
    q, k, v = _inputs(n, n, Hq, Hkv, D, seed=D + Hq)
    out = w4.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _cu(RAGGED), causal=causal)
    _verify(out, q, k, v, RAGGED, RAGGED, causal)
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("L", [1, 15, 16, 127, 128, 255, 256, 257, 640])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_sequence(w4, D, L):
    q, k, v = _inputs(L, L, 3, 1, D, seed=L)
    out = w4.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _cu([L]))
    _verify(out, q, k, v, [L], [L], True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_and_keys_of_other_lengths(w4, D, causal):
    # a prefix before the queries, fewer keys than queries (early rows see
    # nothing where causal), no keys at all, no queries
    lq = [1, 5, 40, 300, 7, 0, 130, 2]
    lk = [200, 5, 700, 100, 0, 50, 131, 1]
    q, k, v = _inputs(sum(lq), sum(lk), 4, 2, D, seed=5)
    out = w4.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _cu(lq), _cu(lk), causal=causal)
    _verify(out, q, k, v, lq, lk, causal)


@pytest.mark.parametrize("G", [2, 3, 5, 7, 12, 16, 40, 64, 100, 128])
def test_group_sizes(w4, G):
    lens = [3, 90, 20]
    q, k, v = _inputs(sum(lens), sum(lens), G, 1, 64, seed=G)
    out = w4.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _cu(lens))
    _verify(out, q, k, v, lens, lens, True)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long(w4, D):
    lens = [2100, 900]
    q, k, v = _inputs(sum(lens), sum(lens), 2, 1, D, seed=9)
    out = w4.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _cu(lens))
    _verify(out, q, k, v, lens, lens, True)


def test_scores_that_grow_and_shrink(w4):
    # the running maximum moves late, early, and by more than the lazy margin
    # in either direction; large scores that overflow exp without it
    L, D = 700, 128
    q, k, v = _inputs(L, L, 2, 1, D, seed=21)
    ramp = torch.linspace(-4, 4, L)[:, None, None]
    for f in (ramp, -ramp, ramp.abs()):
        kk = (k.float() * 0.2 + f * torch.sign(q[L // 2, :1].float())[None]).half()
        qq = (torch.sign(q[L // 2, :1].float()).expand(L, 2, D) + 0.1 * q.float()).half()
        out = w4.prompt_attention(qq.cuda(), kk.cuda(), v.cuda(), _cu([L]), causal=False)
        _verify(out, qq, kk, v, [L], [L], False)


def test_scale_argument(w4):
    q, k, v = _inputs(150, 150, 4, 2, 64, seed=2)
    out = w4.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _cu([150]), scale=0.3)
    _verify(out, q, k, v, [150], [150], True, scale=0.3)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_parts_of_a_fused_projection(w4, D):
    Hq, Hkv, lens = 6, 2, [100, 37]
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn((sum(lens), Hq + 2 * Hkv, D), generator=g).half()
    dev = qkv.cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    out = w4.prompt_attention(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], _cu(lens))
    _verify(out, q, k, v, lens, lens, True)
    dense = w4.prompt_attention(q.cuda(), k.cuda().contiguous(), v.cuda().contiguous(), _cu(lens))
    assert torch.equal(out, dense)


def test_strides_past_32_bits(w4):
    # 300 tokens 8 Mi elements apart: offsets of 2.5 G elements
    L, D, ld = 300, 64, 8 << 20
    q, k, v = _inputs(L, L, 2, 1, D, seed=6)
    big = torch.empty((L, ld), dtype=torch.float16, device="cuda")
    kd = big[:, :D].view(L, 1, D)
    vd = big[:, 1024:1024 + D].view(L, 1, D)
    kd.copy_(k)
    vd.copy_(v)
    out = w4.prompt_attention(q.cuda(), kd, vd, _cu([L]))
    _verify(out, q, k, v, [L], [L], True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -65504.0])
def test_neighbours_do_not_reach(w4, D, bad):
    # the sequences between hold anything; theirs are the only rows it reaches
    lens = [77, 50, 130, 3, 200]
    n = sum(lens)
    q, k, v = _inputs(n, n, 4, 1, D, seed=8)
    cu = np.concatenate([[0], np.cumsum(lens)])
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    clean = w4.prompt_attention(qd, kd, vd, _cu(lens))
    for t in (qd, kd, vd):
        t[cu[1]:cu[2]] = bad
        t[cu[3]:cu[4]] = bad
    out = w4.prompt_attention(qd, kd, vd, _cu(lens))
    for b in (0, 2, 4):
        assert torch.equal(out[cu[b]:cu[b + 1]], clean[cu[b]:cu[b + 1]])
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 1), (128, 1, 1), (128, 8, 1), (256, 4, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_keys_that_a_row_does_not_see_hold_anything(w4, D, Hq, Hkv, bad):
    # rows before the spoilt keys are as without them, and so are the dimensions
    # of V that are not spoilt; a row that sees a spoilt value gets it
    L, at = 400, [70, 131, 250, 399]
    q, k, v = _inputs(L, L, Hq, Hkv, D, seed=15)
    qd, kd, vd, cu = q.cuda(), k.cuda(), v.cuda(), _cu([L])
    clean = w4.prompt_attention(qd, kd, vd, cu)
    for t in at:
        kk, vv = kd.clone(), vd.clone()
        kk[t] = bad
        vv[t] = bad
        out = w4.prompt_attention(qd, kk, vv, cu)
        assert torch.equal(out[:t], clean[:t])
        assert not bool(torch.isfinite(out[t:]).any())
        vv = vd.clone()
        vv[t, :, 5] = bad
        out = w4.prompt_attention(qd, kd, vv, cu)
        assert torch.equal(out[:t], clean[:t])
        rest = torch.ones(D, dtype=torch.bool)
        rest[5] = False
        assert torch.equal(out[t:, :, rest.cuda()], clean[t:, :, rest.cuda()])
        assert not bool(torch.isfinite(out[t:, :, 5]).any())
        if bad != bad:
            assert bool(torch.isnan(out[t:, :, 5]).all())
        else:
            assert bool((out[t:, :, 5] == bad).all())
    assert w4.get_device_status() == 0


def test_rows_of_no_sequence_stay(w4):
    q, k, v = _inputs(100, 100, 2, 1, 64, seed=3)
    out = torch.full((100, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    cu = torch.tensor([0, 30, 60], dtype=torch.int32, device="cuda")
    w4.prompt_attention(q.cuda(), k.cuda(), v.cuda(), cu, out=out)
    assert bool((out[60:] == 7.0).all())
    _verify(out[:60], q[:60], k[:60], v[:60], [30, 30], [30, 30], True)


def test_nothing_to_do(w4):
    e = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    assert w4.prompt_attention(e, e[:, :1], e[:, :1], _cu([0, 0])).shape == (0, 2, 64)
    q = torch.ones((5, 2, 64), dtype=torch.float16, device="cuda")
    out = w4.prompt_attention(q, e[:, :1], e[:, :1], _cu([5]), _cu([0]))
    assert bool((out == 0).all())


def test_many_sequences(w4):
    rs = np.random.RandomState(1)
    lens = [int(x) for x in rs.randint(0, 12, 1500)]
    n = sum(lens)
    q, k, v = _inputs(n, n, 2, 1, 64, seed=13)
    out = w4.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _cu(lens))
    _verify(out, q, k, v, lens, lens, True)


def test_another_stream_and_a_graph(w4):
    lens = [200, 90]
    q, k, v = _inputs(290, 290, 8, 1, 128, seed=14)
    qd, kd, vd, cu = q.cuda(), k.cuda(), v.cuda(), _cu(lens)
    want = w4.prompt_attention(qd, kd, vd, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = w4.prompt_attention(qd, kd, vd, cu)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.prompt_attention(qd, kd, vd, cu, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals(w4):
    q = torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda")
    cu = _cu([4])
    with pytest.raises(TypeError):
        w4.prompt_attention(q.float(), q, q, cu)
    with pytest.raises(ValueError):
        w4.prompt_attention(q, q, q[:3], cu)
    with pytest.raises(ValueError):
        w4.prompt_attention(q, q[:, :, :32], q, cu)
    with pytest.raises(ValueError):
        w4.prompt_attention(q.transpose(1, 2).contiguous().transpose(1, 2), q, q, cu)
    with pytest.raises(TypeError):
        w4.prompt_attention(q, q, q, cu.long())
    with pytest.raises(w4.W4A8Error):
        w4.prompt_attention(q, q, q, cu, scale=-1.0)
    with pytest.raises(w4.W4A8Error):
        w4.prompt_attention(q, q[:, :1].expand(4, 1, 64)[:, :, :], q[:, :1], cu, scale=float("nan"))
