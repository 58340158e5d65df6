"""Decode attention of long sequences on the 8-bit cache, with inputs in which a part
that is lost or counted twice cannot hide.

Scores are whole powers of two apart (c = scale log2 e = 1, q = e_0, K's code of
dimension 0 from 0 to 3 with scale 1), so every weight is a power of two and its rounding
to fp16 exact; V has random codes and one scale.  What is left are the fp32 sums: a worker
has at most 4096 tokens here, or 256 accumulations of 16 tokens, then up to 8 warps and
304 parts are added, each step off by 2^-24 of the sum of magnitudes (2^-23 where a matrix
product truncates), the exponential and the merges' factors 2^-22 each, the division and
the product 2^-23, the output 2^-11:
  |err| <= A (256 2^-23 + 312 2^-24 + 8 2^-22) + 2^-11 |o| + 2^-25,  A = sum p|v| / sum p."""
import numpy as np
import pytest
import torch

SCALE = float(np.float32(0.6931472))


@pytest.fixture(scope="module")
def w4():
    from int4_weight_quantized_gb300.build import build
    build()
    import int4_weight_quantized_gb300 as w4
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return w4


def _tokens(lens, H, D, seed):
    """K's codes of dimension 0 and V's codes of every token: [H][n], [H][n][D]."""
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    return torch.randint(0, 4, (H, n), generator=g), torch.randint(-127, 128, (H, n, D), generator=g)


def _want(k, v, vs, skip=slice(0, 0)):
    """Formula and bound of one sequence and KV head; `skip`: tokens left out."""
    p = torch.exp2(k.double())
    p[skip] = 0.0
    o, A = p @ v.double() * vs / p.sum(), p @ v.abs().double() * vs / p.sum()
    return o, A * (256 * 2.0 ** -23 + 312 * 2.0 ** -24 + 8 * 2.0 ** -22) + 2.0 ** -11 * o.abs() + 2.0 ** -25, p.sum()


def _cache(w4, k, v, lens, T, D, vs, seed):
    """Pages in random order for sequences whose tokens lie one behind another in k and v."""
    need = [-(-n // T) for n in lens]
    H, P = k.shape[0], sum(need) + 2
    order = np.random.RandomState(seed).permutation(P)
    table = np.full((len(lens), max(need)), -1, np.int32)
    kc, vc = torch.zeros((P, H, T, D), dtype=torch.int8), torch.full((P, H, T, D), 99, dtype=torch.int8)
    at = used = 0
    for b, n in enumerate(lens):
        pages = order[used:used + need[b]]
        table[b, :need[b]] = pages
        kk, vv = torch.zeros((H, need[b] * T, D), dtype=torch.int8), torch.full((H, need[b] * T, D), 99, dtype=torch.int8)
        kk[:, :n, 0], vv[:, :n] = k[:, at:at + n].to(torch.int8), v[:, at:at + n].to(torch.int8)
        kc[pages] = kk.view(H, need[b], T, D).transpose(0, 1)
        vc[pages] = vv.view(H, need[b], T, D).transpose(0, 1)
        at, used = at + n, used + need[b]
    cache = w4.KV8Cache(kc.cuda(), torch.ones((P, H, T // 16)).cuda(), vc.cuda(), torch.full((P, H, T // 16), vs).cuda())
    return cache, torch.from_numpy(table).cuda()


def _q(B, Hq, D):
    q = torch.zeros((B, Hq, D), dtype=torch.float16)
    q[..., 0] = 1.0
    return q.cuda()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


LONG = [(64, 4, 1, 128, [131067]), (64, 16, 1, 16, [30000]), (64, 24, 3, 128, [70001, 5000]), (128, 32, 2, 32, [20000, 0, 9000]),
        (128, 10, 2, 64, [8192] * 4), (128, 16, 2, 128, [131072]), (256, 16, 1, 64, [4097, 33333]), (256, 5, 1, 128, [100000]),
        (128, 8, 8, 32, [16000, 3, 700, 12345, 1, 0, 5000, 4096]), (64, 2, 1, 16, [int(x) for x in np.random.RandomState(3).randint(0, 5200, 60)])]


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hq,H,T,lens", LONG)
def test_every_token_counts_once(w4, D, Hq, H, T, lens):
    k, v = _tokens(lens, H, D, seed=D + T)
    cache, table = _cache(w4, k, v, lens, T, D, 0.5, seed=1)
    wide = torch.nn.functional.pad(table, (0, max(0, 4096 // T + 1 - table.shape[1])), value=-1).contiguous()
    out = w4.decode_attention_kv8(_q(len(lens), Hq, D), cache, wide, _i32(lens), scale=SCALE).double().cpu()
    at = 0
    for b, n in enumerate(lens):
        for h in range(H):
            rows = out[b, h * (Hq // H):(h + 1) * (Hq // H)]
            if n == 0:
                assert bool((rows == 0).all())
                continue
            o, tol, _ = _want(k[h, at:at + n], v[h, at:at + n], 0.5)
            assert bool(((rows - o).abs() <= tol).all()), (b, h, float(((rows - o).abs() / tol).max()))
        at += n
    assert w4.get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("D,T,n,pieces", [(64, 128, 131067, 40), (128, 32, 50000, 9), (256, 64, 20011, 5)])
def test_one_long_sequence_equals_its_parts(w4, D, T, n, pieces):
    # the same tokens as one sequence and as several: out = sum L_i out_i / sum L_i, where
    # L_i are the parts' sums of weights (whole numbers); each out_i is off by its own bound
    k, v = _tokens([n], 1, D, seed=D)
    cuts = [0] + sorted(int(x) for x in np.random.RandomState(D).choice(np.arange(1, n), pieces - 1, replace=False)) + [n]
    lens = [y - x for x, y in zip(cuts, cuts[1:])]
    c1, t1 = _cache(w4, k, v, [n], T, D, 0.5, seed=2)
    c2, t2 = _cache(w4, k, v, lens, T, D, 0.5, seed=3)
    one = w4.decode_attention_kv8(_q(1, 8, D), c1, t1, _i32([n]), scale=SCALE).double().cpu()[0]
    many = w4.decode_attention_kv8(_q(pieces, 8, D), c2, t2, _i32(lens), scale=SCALE).double().cpu()
    parts = [_want(k[0, x:y], v[0, x:y], 0.5) for x, y in zip(cuts, cuts[1:])]
    L = torch.stack([p[2] for p in parts])
    merged = (L[:, None, None] * many).sum(0) / L.sum()
    tol = sum(w * p[1] for w, p in zip(L / L.sum(), parts)) + _want(k[0], v[0], 0.5)[1]
    assert bool(((one - merged).abs() <= tol).all()), float(((one - merged).abs() / tol).max())


@pytest.fixture
def one_thread():
    """Tests that fork may follow: no threads of torch are left behind."""
    n = torch.get_num_threads()
    torch.set_num_threads(1)
    yield
    torch.set_num_threads(n)


@pytest.mark.parametrize("D,Hq,H,T,lens", LONG)
def test_the_bound_shows_a_lost_tile(one_thread, D, Hq, H, T, lens):
    # on the CPU: leaving any 32 consecutive tokens out, or counting them twice, passes the bound several times
    k, v = _tokens(lens, H, D, seed=D + T)
    at = 0
    for n in lens:
        if n >= 64:
            o, tol, L = _want(k[0, at:at + n], v[0, at:at + n], 0.5)
            for lo in (0, n // 3 // 32 * 32, (n - 32) // 32 * 32):
                less = _want(k[0, at:at + n], v[0, at:at + n], 0.5, slice(lo, lo + 32))
                assert float(((less[0] - o).abs() / tol).max()) > 2.0
                p = torch.exp2(k[0, at + lo:at + lo + 32].double())
                twice = (o * L + p @ v[0, at + lo:at + lo + 32].double() * 0.5) / (L + p.sum())
                assert float(((twice - o).abs() / tol).max()) > 2.0
        at += n
