"""Prompt attention on the GPU: what a row does not see changes nothing of it, bit for bit."""
import numpy as np
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


def _cu(lens):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()


def _inputs(nq, nk, Hq, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((nq, Hq, D), generator=g) * 1.5).half()
    k, v = (torch.randn((nk, Hkv, D), generator=g).half() for _ in range(2))
    return q.cuda(), k.cuda(), v.cuda()


@pytest.mark.parametrize("D,G,prefix", [(256, 1, 0), (256, 3, 37), (256, 7, 100), (256, 2, 191), (256, 8, 515), (128, 3, 37),
                                        (128, 7, 191), (64, 3, 100), (64, 7, 515)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_spoilt_values_on_the_diagonal(w4, D, G, prefix, bad):
    # the diagonal crosses tiles of 128 keys anywhere, in first, middle and last tiles
    n = 600
    q, k, v = _inputs(n, n + prefix, G, 1, D, seed=D + G)
    cu, ck = _cu([n]), _cu([n + prefix])
    clean = w4.prompt_attention(q, k, v, cu, ck)
    for at in (1, 84, 126, 127, 128, 129, 200, 255, 256, 383, 384, 450, 512, 598, 599):
        vv = v.clone()
        vv[prefix + at] = bad
        out = w4.prompt_attention(q, k, vv, cu, ck)
        assert torch.equal(out[:at], clean[:at])
        assert not bool(torch.isfinite(out[at:]).any())
    vv = v.clone()                                     # all of them from some key on
    vv[prefix + 64:] = bad
    out = w4.prompt_attention(q, k, vv, cu, ck)
    assert torch.equal(out[:64], clean[:64]) and not bool(torch.isfinite(out[64:]).any())
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("D,G,prefix", [(64, 1, 0), (64, 3, 40), (128, 1, 0), (128, 5, 130), (128, 8, 0), (256, 3, 100), (256, 8, 0)])
def test_large_keys_behind_a_row_change_no_bit_of_it(w4, D, G, prefix):
    # finite values: a later token's scores may be as large as they like
    n = 500
    q, k, v = _inputs(n, n + prefix, G, 1, D, seed=D + G)
    cu, ck = _cu([n]), _cu([n + prefix])
    clean = w4.prompt_attention(q, k, v, cu, ck)
    for at in (1, 60, 130, 250, 257, 400, 499):
        kk, vv, qq = k.clone(), v.clone(), q.clone()
        # growing scores of the later tokens, on keys that the earlier rows see too
        qq[at:] = 40.0 * qq[at:].sign() * torch.linspace(1, 8, n - at, device="cuda")[:, None, None].half()
        kk[prefix + at:] *= 30.0
        vv[prefix + at:] = 65504.0
        out = w4.prompt_attention(qq, kk, vv, cu, ck)
        assert torch.equal(out[:at], clean[:at])
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("D,G", [(64, 1), (64, 3), (128, 2), (128, 7), (256, 1), (256, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_large_neighbours_change_no_bit(w4, D, G, causal):
    # neighbours in the packing of several key tiles, with queries and keys whose
    # scores on a sequence's own keys grow from tile to tile
    lq, lk = [77, 300, 130, 5, 200], [400, 300, 655, 517, 900]
    q, k, v = _inputs(sum(lq), sum(lk), G, 1, D, seed=D + G)
    aq, ak = np.concatenate([[0], np.cumsum(lq)]), np.concatenate([[0], np.cumsum(lk)])
    for b in (0, 2, 4):                                  # keys that grow along the sequence
        k[ak[b]:ak[b + 1]] *= torch.linspace(0.1, 3, lk[b], device="cuda")[:, None, None].half()
    clean = w4.prompt_attention(q, k, v, _cu(lq), _cu(lk), causal=causal)
    for f in (60.0, -60.0):
        qq, kk, vv = q.clone(), k.clone(), v.clone()
        for b in (1, 3):
            qq[aq[b]:aq[b + 1]] *= f
            kk[ak[b]:ak[b + 1]] *= f
            vv[ak[b]:ak[b + 1]] = f * 1000
        out = w4.prompt_attention(qq, kk, vv, _cu(lq), _cu(lk), causal=causal)
        for b in (0, 2, 4):
            assert torch.equal(out[aq[b]:aq[b + 1]], clean[aq[b]:aq[b + 1]])
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("D,G", [(64, 3), (128, 5), (128, 3), (256, 7), (256, 3)])
def test_rows_that_a_group_leaves_over_change_no_bit(w4, D, G):
    # 128 / G tokens to a tile: its last rows belong to no token, and their queries
    # are whatever shared memory held
    n = 700
    q, k, v = _inputs(n, n, G, 1, D, seed=D + G)
    k *= torch.linspace(0.1, 3, n, device="cuda")[:, None, None].half()
    first = w4.prompt_attention(q, k, v, _cu([n]))
    for f in (1.0, 100.0, -100.0, 3000.0):
        # another group size fills every row of the tiles
        x = torch.full((152 * 128, 1, D), f, dtype=torch.float16, device="cuda") * q[:1, :1].sign()
        w4.prompt_attention(x, x, x, _cu([152 * 128]), causal=False) if D == 64 else w4.prompt_attention(x[:8192], x[:8192], x[:8192], _cu([8192]))
        assert torch.equal(w4.prompt_attention(q, k, v, _cu([n])), first)
