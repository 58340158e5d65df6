"""Many tokens of small weight beside one that takes almost all of it, in prompt
attention and in decode attention on the 8-bit cache."""
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
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("gap", [12, 18.05, 20.05, 22.5, 25.2])
def test_prompt(w4, D, causal, gap):
    # one key takes almost the whole weight and has v = 0, n - 1 others have 2^-gap of it
    # each and v = 1: out = (n - 1) 2^-gap / (1 + (n - 1) 2^-gap).  The scores are
    # multiples of one value times c = scale log2 e, so x is off by 2^-22 of 26 at most
    # (2^-17 of the weight); a weight is rounded to fp16 at 2^7 times itself or more:
    # 2^-11 of it or 2^-25 2^-7; sums: n / 16 accumulations of 2^-23 each; the output 2^-11.
    n = 16384
    scale = gap * np.log(2.0) / (D * 1.0)
    q = torch.ones((256, 2, D), dtype=torch.float16, device="cuda")
    k = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda")
    v = torch.ones((n, 1, D), dtype=torch.float16, device="cuda")
    for first in (0, n // 2, n - 300):
        k.zero_()
        v.fill_(1.0)
        k[first] = 1.0                                # score gap, the others 0
        v[first] = 0.0
        out = w4.prompt_attention(q, k, v, _cu([256]), _cu([n]), causal=causal, scale=float(np.float32(scale))).double().cpu()
        seen = torch.arange(n - 256, n) + 1 if causal else torch.full((256,), n)
        w = (seen - 1) * 2.0 ** -gap
        want = (w / (1 + w))[:, None, None]
        tol = want * (2.0 ** -17 + 2.0 ** -11 + n / 16 * 2.0 ** -22 + 2.0 ** -11) + n * 2.0 ** -32 + 2.0 ** -25
        assert bool(((out - want).abs() <= tol).all()), float(((out - want).abs() / tol).max())


@pytest.mark.parametrize("n,Hq,D", [(131072, 8, 64), (131072, 8, 128), (65536, 16, 128), (4096, 8, 256), (3000, 16, 64), (40000, 8, 256)])
@pytest.mark.parametrize("gap", [12, 18.05, 20.05, 22.5, 25.2])
def test_decode(w4, n, Hq, D, gap):
    # one token with score gap (in powers of two) and v = 0, the others with score 0 and v =
    # 1 (code 127 of scale 1/127, off by 2^-23): out = (n - 1) 2^-gap / (1 + (n - 1) 2^-gap).
    # Scores: 2^-17 of a weight; a weight 2^-11 of it or 2^-32 of the largest one; sums:
    # a worker's tokens and the parts, n / 16 accumulations of 2^-23 at most; the output 2^-11.
    T = 64
    P = -(-n // T)
    codes, scale = (P, 1, T, D), (P, 1, T // 16)
    kc = torch.zeros(codes, dtype=torch.int8, device="cuda")
    ks = torch.full(scale, 1.0, device="cuda")
    vc = torch.full(codes, 127, dtype=torch.int8, device="cuda")
    vs = torch.full(scale, 1.0 / 127, device="cuda")
    table = _i32(np.arange(P)[None])
    q = torch.ones((1, Hq, D), dtype=torch.float16, device="cuda")
    s = float(np.float32(gap * np.log(2.0) / D))
    for first in (0, n // 2, n - 1):
        kc.zero_()
        vc.fill_(127)
        kc[first // T, 0, first % T] = 1
        vc[first // T, 0, first % T] = 0
        out = w4.decode_attention_kv8(q, w4.KV8Cache(kc, ks, vc, vs), table, _i32([n]), scale=s).double().cpu()
        w = (n - 1) * 2.0 ** -gap
        want = w / (1 + w)
        tol = want * (2.0 ** -23 + 2.0 ** -17 + 2.0 ** -11 + n / 16 * 2.0 ** -22 + 2.0 ** -11) + n * 2.0 ** -32 + 2.0 ** -25
        assert bool(((out - want).abs() <= tol).all()), float(((out - want).abs() / tol).max())
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("n", [600, 5000])
def test_a_worker_at_its_margin_stays_in_range(w4, n):
    # scores that grow by less than the margin of the running maximum, block by block,
    # and V's scale beside them: no weight passes fp16's range, no sum is lost
    D, T = 64, 16
    P = -(-n // T)
    g = torch.Generator().manual_seed(n)
    blk = torch.arange(P, device="cuda")
    for step in (14.9, 15.0, 15.1, 7.9, 8.1):
        kc = torch.zeros((P, 1, T, D), dtype=torch.int8, device="cuda")
        kc[..., 0] = 1
        ks = (step * (blk % 9)).float()[:, None, None].contiguous()
        vc = torch.randint(-127, 128, (P, 1, T, D), generator=g).to(torch.int8).cuda()
        vs = (2.0 ** (blk % 5 - 2).float())[:, None, None].contiguous()
        q = torch.zeros((1, 8, D), dtype=torch.float16, device="cuda")
        q[..., 0] = 1.0
        scale = float(np.float32(np.log(2.0)))
        wide = np.concatenate([np.arange(P), np.full(4096 // T + 1, -1)])[None]
        x = (ks.double() * np.log2(np.e) * scale).expand(P, 1, T).reshape(-1)[:n].cpu()
        v = (vc.double() * vs[:, :, :, None].double()).reshape(-1, D)[:n].cpu()
        p = torch.exp2(x - x.max())
        want = p @ v / p.sum()
        # 2^-16: scores up to 120; weights 2^-11 or 2^-32 of the largest times V's scale (its
        # codes up to 127 times 2^2); sums n / 16 accumulations; the output 2^-11
        A = p @ v.abs() / p.sum()
        tol = A * (2.0 ** -16 + 2.0 ** -11 + n / 16 * 2.0 ** -22) + n * 2.0 ** -32 * 508 + 2.0 ** -11 * want.abs() + 2.0 ** -25
        for table in (np.arange(P)[None], wide):
            out = w4.decode_attention_kv8(q, w4.KV8Cache(kc, ks, vc, vs), _i32(table), _i32([n]), scale=scale).double().cpu()
            assert bool(((out[0] - want).abs() <= tol).all()), float(((out[0] - want).abs() / tol).max())
