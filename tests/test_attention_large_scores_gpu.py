"""Scores so large that neighbouring fp32 values are 16 apart, of prompt attention and of
decode attention on the 8-bit cache: weights stay finite."""
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


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def _cu(lens):
    return _i32(np.concatenate([[0], np.cumsum(lens)]))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("odd", [0, 1])
def test_prompt(w4, D, odd):
    # neighbouring fp32 scores are 16 apart there; they grow by one such step with every
    # tile of 128 keys (exact sums: 2048 (1.5 2^16 / D) (D - 1) + 16 t, c = scale log2 e near 1).
    # A maximum that stays behind by a step must not take a weight past fp16's range.
    n = 700
    g = torch.Generator().manual_seed(D)
    v = torch.randn((n, 1, D), generator=g).half()
    q = torch.full((n, 2, D), 2048.0, dtype=torch.float16)
    k = torch.full((n, 1, D), 1.5 * 65536 / D, dtype=torch.float16)
    t = torch.arange(n) // 128 + odd
    q[..., -1] = 16.0
    k[:, 0, -1] = t.half()
    out = w4.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _cu([n]), scale=float(np.float32(1 / np.log2(np.e)))).double().cpu()
    see = torch.arange(n)[None] <= torch.arange(n)[:, None]
    x = torch.where(see, 16.0 * t[None].double(), -torch.inf)
    p = torch.exp2(x - x.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    want, A = (p @ v[:, 0].double())[:, None], (p @ v[:, 0].double().abs())[:, None]
    # weights 2^-11, their exponents 2^-18, sums n / 16 times 2^-22; the output 2^-11
    tol = A * (2.0 ** -11 + 2.0 ** -18 + n / 16 * 2.0 ** -22) + 2.0 ** -11 * want.abs() + 2.0 ** -25
    assert bool(((out - want).abs() <= tol).all()), float(((out - want).abs() / tol).max())


@pytest.mark.parametrize("D,T", [(64, 16), (128, 32), (256, 64)])
@pytest.mark.parametrize("n,every", [(4096, 64), (700, 8), (150000, 2)])
@pytest.mark.parametrize("odd", [0, 1])
def test_decode(w4, D, T, n, every, odd):
    # neighbouring fp32 scores are 16 apart there; they grow by one such step every few
    # blocks, so that a warp meets several: q 2048 times code 64 times a scale of 1536 + t 2^-13 (exact; c = scale log2 e = 1)
    scale = next(x for x in (np.nextafter(np.float32(0.6931472), np.float32(i)) for i in (0, 0.6931472, 1))
                 if x * np.float32(1.4426950408889634) == 1)
    P = -(-n // T)
    g = torch.Generator().manual_seed(D)
    t = torch.arange(P * T // 16) // every + odd
    kc = torch.zeros((P, 1, T, D), dtype=torch.int8)
    kc[..., 0] = 64
    ks = (1536.0 + t.float() * 2.0 ** -13).view(P, 1, T // 16)
    vc = torch.randint(-127, 128, (P, 1, T, D), generator=g).to(torch.int8)
    vs = torch.full((P, 1, T // 16), 1.0 / 64)
    q = torch.zeros((1, 8, D), dtype=torch.float16)
    q[..., 0] = 2048.0
    x = (16.0 * t.double()).repeat_interleave(16)[:n]
    v = vc.double().view(-1, D)[:n] / 64
    p = torch.exp2(x - x.max())
    want, A = p @ v / p.sum(), p @ v.abs() / p.sum()
    # weights 2^-11, sums n / 16 times 2^-22, the output 2^-11; log2 of V's scale is far
    # below a step of the scores: weights times 2^-6, as they all are
    tol = A * (2.0 ** -11 + 2.0 ** -18 + n / 16 * 2.0 ** -22) + 2.0 ** -11 * want.abs() + 2.0 ** -25
    cache = w4.KV8Cache(kc.cuda(), ks.cuda(), vc.cuda(), vs.cuda())
    for extra in (0, 4096 // T + 1):
        table = _i32(np.concatenate([np.arange(P), np.full(extra, -1)])[None])
        out = w4.decode_attention_kv8(q.cuda(), cache, table, _i32([n]), scale=float(scale)).double().cpu()
        assert bool(((out[0] - want).abs() <= tol).all()), float(((out[0] - want).abs() / tol).max())
