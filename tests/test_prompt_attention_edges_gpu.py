"""Prompt attention on the GPU: what a row does not see changes nothing of it, bit
for bit, and weights far below the largest still count."""
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
