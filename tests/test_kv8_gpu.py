"""The 8-bit paged KV cache on the GPU: writing, reading, decode attention and
the page operations, against plain implementations on the CPU."""
import numpy as np
import pytest
import torch

from .attention_ref import attention, check

pytestmark = pytest.mark.gpu
ERR_PAGE = 8


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


def _table(lens, T, P, seed, extra=0):
    """Pages in random order; entries behind a row's end name no page at all."""
    need = [-(-n // T) for n in lens]
    order = np.random.RandomState(seed).permutation(P)[:sum(need)]
    t = np.full((len(lens), max(max(need), 1) + extra), -5, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def _random_cache(w4, P, H, T, D, seed):
    g = torch.Generator().manual_seed(seed)

    def one():
        return (torch.randint(-127, 128, (P, H, T, D), generator=g).to(torch.int8).cuda(),
                (torch.rand((P, H, T // 16), generator=g) * 0.02 + 0.005).cuda())
    kc, ks = one()
    vc, vs = one()
    return w4.KV8Cache(kc, ks, vc, vs)


def _f32(x):
    return np.float32(x)


def _ref_append(codes, scale, x, table, start, lens, T):
    """One of the two tensors on the CPU, token by token and block by block, in fp32."""
    codes, scale = codes.copy(), scale.copy()
    P, H, _, D = codes.shape
    at = 0
    for b, n in enumerate(lens):
        new = {start[b] + i: x[at + i].astype(np.float32) for i in range(n)}
        at += n
        for blk in sorted({p // 16 for p in new}):
            page = table[b, blk * 16 // T] if blk * 16 // T < table.shape[1] else -1
            if not 0 <= page < P:
                continue
            for h in range(H):
                toks = [p for p in range(blk * 16, blk * 16 + 16)]
                old = [p for p in toks if p < start[b]]
                s_old = scale[page, h, blk * 16 % T // 16] if old else _f32(0)
                amax = max(np.abs(new[p][h]).max() for p in toks if p in new)
                s = max(s_old, _f32(amax) / _f32(127))
                for p in toks:
                    if p in new:
                        codes[page, h, p % T] = np.clip(np.rint(new[p][h] / s), -127, 127) if s > 0 else 0
                    elif p in old and s > s_old:
                        codes[page, h, p % T] = np.rint(codes[page, h, p % T].astype(np.float32) * (s_old / s))
                scale[page, h, blk * 16 % T // 16] = s
    return codes, scale


def _np(c):
    return [t.cpu().numpy() for t in c]


@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("D,H", [(64, 1), (64, 3), (128, 2), (256, 1)])
def test_append_and_read(w4, D, H, T):
    start = np.array([0, 3, 16, 31, 130, 5, 0, 200], np.int64)
    new = [1, 20, 1, 1, 90, 0, 75, 16]
    P = 60
    cache = _random_cache(w4, P, H, T, D, seed=T + D)
    table = _table([s + n for s, n in zip(start, new)], T, P, seed=3, extra=1)
    rs = np.random.RandomState(D)
    x = [(rs.standard_normal((sum(new), H, D)) * rs.choice([0.1, 1.0, 6.0], (sum(new), 1, 1))).astype(np.float16) for _ in range(2)]
    x[0][5] = 0                                   # a token of zeros
    x[1][22:27] = 0
    before = _np(cache)
    w4.kv8_append(cache, torch.from_numpy(x[0]).cuda(), torch.from_numpy(x[1]).cuda(), _i32(table), _i32(start), _cu(new))
    after = _np(cache)
    for i in range(2):
        c, s = _ref_append(before[2 * i], before[2 * i + 1], x[i], table, start, new, T)
        assert np.array_equal(after[2 * i + 1], s)
        assert np.array_equal(after[2 * i], c)
    total = [int(s + n) for s, n in zip(start, new)]
    got = w4.kv8_read(cache, _i32(table), _cu(total), sum(total))
    at = 0
    for b, n in enumerate(total):
        for p in range(n):
            page = table[b, p // T]
            for i in range(2):
                want = (after[2 * i][page, :, p % T].astype(np.float32) * after[2 * i + 1][page, :, p % T // 16][:, None]).astype(np.float16)
                assert np.array_equal(got[i][at + p].cpu().numpy(), want)
        at += n
    assert w4.get_device_status() == 0


def test_append_token_by_token_stays_near(w4):
    # 70 tokens one at a time: each growth of a block's scale may move an
    # earlier code by half a step of the new scale, and 16 tokens grow it at
    # most 15 times: a value is off by at most (1 + 15) / 2 steps
    T, D, H = 32, 64, 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn((70, H, D), generator=g).half()
    cache = w4.kv8_cache(8, H, T, D)
    table = _i32([[4, 1, 6, 0]])
    one = _cu([1])
    for p in range(70):
        w4.kv8_append(cache, x[p:p + 1].cuda(), (2 * x[p:p + 1]).cuda(), table, _i32([p]), one)
    k, v = w4.kv8_read(cache, table, _cu([70]), 70)
    for b in range(0, 70, 16):
        blk = x[b:b + 16].float()
        step = blk.abs().amax((0, 2)) / 127
        assert bool(((k[b:b + 16].cpu().float() - blk).abs() <= 8 * step[None, :, None] + 1e-3).all())
        assert bool(((v[b:b + 16].cpu().float() - 2 * blk).abs() <= 16 * step[None, :, None] + 2e-3).all())
    # the scale is the block's largest value whatever the order
    s = cache.k_scale.cpu()
    for b in range(0, 70, 16):
        page = [4, 1, 6, 0][b // T]
        assert torch.equal(s[page, :, b % T // 16], x[b:b + 16].float().abs().amax((0, 2)) / 127)


def test_append_from_a_fused_projection(w4):
    T, D, H, n = 16, 128, 2, 50
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((n, 8, D), generator=g).half().cuda()
    k, v = qkv[:, 4:6], qkv[:, 6:8]
    table, zero = _i32(_table([n], T, 9, 2)), _i32([0])
    a, b = w4.kv8_cache(9, H, T, D), w4.kv8_cache(9, H, T, D)
    w4.kv8_append(a, k, v, table, zero, _cu([n]))
    w4.kv8_append(b, k.contiguous(), v.contiguous(), table, zero, _cu([n]))
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert int((a.k_scale > 0).sum()) == H * 4


def test_append_to_no_page(w4):
    # tokens whose page is missing are dropped, the others are written
    T, D, H = 16, 64, 1
    cache = w4.kv8_cache(4, H, T, D)
    x = torch.ones((40, H, D), dtype=torch.float16, device="cuda")
    w4.kv8_append(cache, x, x, _i32([[2, 77, 1]]), _i32([0]), _cu([40]))
    assert w4.get_device_status() == ERR_PAGE
    held = cache.k_scale.flatten().cpu() > 0
    assert held.tolist() == [False, True, True, False]
    w4.kv8_append(cache, x, x, _i32([[0]]), _i32([0]), _cu([40]))           # the table ends
    assert w4.get_device_status() == ERR_PAGE
    assert (cache.k_scale.flatten().cpu() > 0).tolist() == [True, True, True, False]
    w4.kv8_append(cache, x[:1], x[:1], _i32([[3]]), _i32([-2]), _cu([1]))   # a negative start
    assert w4.get_device_status() == ERR_PAGE
    assert not bool(cache.k_scale[3].any())
    k, v = w4.kv8_read(cache, _i32([[2, -1, 1]]), _cu([40]), 40)
    assert w4.get_device_status() == ERR_PAGE
    assert bool((k[:16] > 0.99).all()) and bool((k[16:32] == 0).all()) and bool((v[32:] > 0.99).all())
    assert w4.get_device_status() == 0


def _values(cache, table, b, n, T):
    kc, ks, vc, vs = (t.cpu().double() for t in cache)
    pages = torch.tensor(table[b, :-(-n // T)].astype(np.int64))
    H, D = kc.shape[1], kc.shape[3]

    def one(c, s):
        x = c[pages].view(-1, H, T // 16, 16, D) * s[pages][:, :, :, None, None]
        return x.permute(1, 0, 2, 3, 4).reshape(H, -1, D)[:, :n]
    return one(kc, ks), one(vc, vs)


def _verify_decode(out, q, cache, table, lens, T, scale=None):
    B, Hq, D = q.shape
    H = cache.k_codes.shape[1]
    for b, n in enumerate(lens):
        k, v = _values(cache, table, b, n, T)
        for h in range(H):
            rows = slice(h * (Hq // H), (h + 1) * (Hq // H))
            ref, bound = attention(q[b, rows], k[h], v[h], scale or D ** -0.5)
            check(out[b, rows], ref, bound, f"sequence {b} of {n} tokens, KV head {h}")


@pytest.mark.parametrize("extra", [2, 300])         # tables for either kernel
@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 1), (6, 2), (16, 1), (11, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_attention(w4, D, Hq, H, T, extra):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 200, 129, 1000]
    P = 130 if T == 16 else 70
    cache = _random_cache(w4, P, H, T, D, seed=T)
    table = _table(lens, T, P, seed=2, extra=extra)
    q = torch.randn((len(lens), Hq, D), generator=torch.Generator().manual_seed(D)).half()
    out = w4.decode_attention_kv8(q.cuda(), cache, _i32(table), _i32(lens))
    assert bool((out[1] == 0).all())
    _verify_decode(out, q, cache, table, lens, T)
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("B", [1, 5, 20, 75, 150])
@pytest.mark.parametrize("D,Hq,H,T", [(64, 8, 1, 16), (64, 24, 2, 128), (128, 4, 2, 32), (128, 11, 1, 64), (256, 8, 1, 64), (256, 16, 1, 16)])
def test_decode_short_tables(w4, D, Hq, H, T, B):
    # tables of up to 4096 tokens: clusters of 8, 4, 2 and 1 CTAs for each pair,
    # sequences shorter than a cluster's warps and as long as the table
    rs = np.random.RandomState(B + D)
    lens = [[4096, 0, 1, 16, 17, 640, 1009, 127, 128, 129][i] if i < 10 else int(rs.randint(0, 400)) for i in range(B)]
    P = sum(-(-n // T) for n in lens) + 2
    cache = _random_cache(w4, P, H, T, D, seed=T)
    table = _table(lens, T, P, seed=2)
    q = torch.randn((B, Hq, D), generator=torch.Generator().manual_seed(D)).half()
    out = w4.decode_attention_kv8(q.cuda(), cache, _i32(table), _i32(lens))
    _verify_decode(out, q, cache, table, lens, T)
    # the same tables made longer take the other kernels
    wide = np.concatenate([table, np.full((B, 4096 // T + 1), -1, np.int32)], 1)
    other = w4.decode_attention_kv8(q.cuda(), cache, _i32(wide), _i32(lens))
    _verify_decode(other, q, cache, table, lens, T)
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("D,T", [(64, 16), (128, 32), (256, 128)])
def test_decode_long_and_short(w4, D, T):
    # one long sequence over many CTAs, cut at any place, among short ones
    lens = [3, 20000, 1, 4097, 0, 640]
    P = sum(-(-n // T) for n in lens) + 3
    cache = _random_cache(w4, P, 2, T, D, seed=7)
    table = _table(lens, T, P, seed=4)
    q = torch.randn((len(lens), 8, D), generator=torch.Generator().manual_seed(1)).half()
    out = w4.decode_attention_kv8(q.cuda(), cache, _i32(table), _i32(lens))
    _verify_decode(out, q, cache, table, lens, T)


@pytest.mark.parametrize("D,Hq,H,T,lens", [
    (64, 16, 1, 16, [30000]), (64, 24, 3, 128, [70001, 5000]), (128, 32, 2, 32, [20000, 0, 9000]), (128, 10, 2, 64, [8192] * 4),
    (256, 16, 1, 64, [4097, 33333]), (256, 5, 1, 128, [100000])])
def test_decode_parts_joined_on_chip(w4, D, Hq, H, T, lens):
    # few long pairs: CTAs inside one pair join their warps' parts, those over a
    # pair's end do not; one stretch of the last sequence is on no page
    P = sum(-(-n // T) for n in lens) + 1
    cache = _random_cache(w4, P, H, T, D, seed=T + D)
    table = _table(lens, T, P, seed=2)
    n = lens[-1] // T
    table[-1, n // 4:n // 2] = -1
    q = torch.randn((len(lens), Hq, D), generator=torch.Generator().manual_seed(D)).half()
    out = w4.decode_attention_kv8(q.cuda(), cache, _i32(table), _i32(lens))
    assert w4.get_device_status() == ERR_PAGE
    keep = [x for i, x in enumerate(table[-1]) if not n // 4 <= i < n // 2]
    held = np.full_like(table, -1)
    held[:-1] = table[:-1]
    held[-1, :len(keep)] = keep
    _verify_decode(out, q, cache, held, lens[:-1] + [lens[-1] - (n // 2 - n // 4) * T], T)
    again = w4.decode_attention_kv8(q.cuda(), cache, _i32(table), _i32(lens))
    assert torch.equal(out, again) and w4.get_device_status() == ERR_PAGE


@pytest.mark.parametrize("extra", [0, 300])
def test_decode_many_sequences(w4, extra):
    rs = np.random.RandomState(5)
    lens = [int(x) for x in rs.randint(0, 40, 700)]
    T, D = 16, 64
    P = sum(-(-n // T) for n in lens) + 1
    cache = _random_cache(w4, P, 1, T, D, seed=7)
    table = _table(lens, T, P, seed=4, extra=extra)
    q = torch.randn((len(lens), 2, D), generator=torch.Generator().manual_seed(1)).half()
    out = w4.decode_attention_kv8(q.cuda(), cache, _i32(table), _i32(lens))
    _verify_decode(out, q, cache, table, lens, T)


def test_decode_one_long_sequence_equal_to_parts(w4):
    # 131072 tokens: the same tokens in one sequence and its exact reference
    T, D, n = 128, 64, 131072 - 5
    P = n // T + 2
    cache = _random_cache(w4, P, 1, T, D, seed=11)
    table = _table([n], T, P, seed=4)
    q = torch.randn((1, 4, D), generator=torch.Generator().manual_seed(1)).half()
    out = w4.decode_attention_kv8(q.cuda(), cache, _i32(table), _i32([n]))
    _verify_decode(out, q, cache, table, [n], T)


@pytest.mark.parametrize("extra", [0, 300])
def test_decode_scales_of_every_size(w4, extra):
    # blocks whose scales differ by many powers of two, zero scales, equal
    # values everywhere; what is behind a sequence's end holds anything
    T, D, n = 32, 128, 300
    cache = _random_cache(w4, 12, 1, T, D, seed=3)
    table = _table([n], T, 12, seed=1, extra=extra)
    q = torch.randn((1, 8, D), generator=torch.Generator().manual_seed(1)).half()
    rs = np.random.RandomState(2)
    for kmul, vmul in (([1e-4, 1.0], [1e-9, 1e-3, 1.0, 300.0]), ([1.0], [1e-9]), ([0.0, 1.0], [0.0, 1.0]), ([0.5], [0.0])):
        c = w4.KV8Cache(*(t.clone() for t in cache))
        c.k_scale.mul_(torch.from_numpy(rs.choice(kmul, c.k_scale.shape)).float().cuda())
        c.v_scale.mul_(torch.from_numpy(rs.choice(vmul, c.v_scale.shape)).float().cuda())
        page, blk = int(table[0, n // T]), n % T // 16
        ref = w4.KV8Cache(*(t.clone() for t in c))
        c.k_scale[page, :, blk + 1:] = float("nan")
        c.v_scale[page, :, blk + 1:] = float("nan")
        out = w4.decode_attention_kv8(q.cuda(), c, _i32(table), _i32([n]))
        _verify_decode(out, q, ref, table, [n], T)


@pytest.mark.parametrize("extra", [0, 300])
def test_decode_growing_scores(w4, extra):
    T, D, n = 16, 64, 900
    cache = _random_cache(w4, 60, 1, T, D, seed=3)
    table = _table([n], T, 60, seed=1, extra=extra)
    q = torch.randn((1, 8, D), generator=torch.Generator().manual_seed(1)).half()
    for order in (1, -1):
        for i in range(57):
            f = i if order > 0 else 56 - i
            cache.k_scale[int(table[0, i])] = 0.002 * (1 + f)
        out = w4.decode_attention_kv8(q.cuda(), cache, _i32(table), _i32([n]))
        _verify_decode(out, q, cache, table, [n], T)


@pytest.mark.parametrize("extra", [0, 300])
def test_decode_without_a_page(w4, extra):
    # tokens on no page are left out: as if the sequence had the others only
    T, D = 16, 64
    cache = _random_cache(w4, 6, 1, T, D, seed=3)
    q = torch.randn((3, 4, D), generator=torch.Generator().manual_seed(1)).half()
    table = np.array([[0, 1, 2], [0, 99, 2], [-1, 6, -7]], np.int32)
    wide = np.concatenate([table, np.full((3, extra), -9, np.int32)], 1)
    out = w4.decode_attention_kv8(q.cuda(), cache, _i32(wide), _i32([48, 48, 48]))
    assert w4.get_device_status() == ERR_PAGE
    _verify_decode(out[:1], q[:1], cache, table, [48], T)
    _verify_decode(out[1:2], q[1:2], cache, np.array([[0, 2]]), [32], T)
    assert bool((out[2] == 0).all())
    # lengths outside the table are clamped into it
    out = w4.decode_attention_kv8(q.cuda(), cache, _i32([[0, 1, 2]] * 3), _i32([1000, -4, 48]))
    assert torch.equal(out[0], w4.decode_attention_kv8(q.cuda(), cache, _i32([[0, 1, 2]] * 3), _i32([48, 48, 48]))[0])
    assert bool((out[1] == 0).all())
    assert w4.get_device_status() == 0


def test_cache_past_32_bits(w4):
    # 40000 pages of 64 KB: codes past 2^31, both for writing and for reading
    P, H, T, D = 40000, 4, 128, 128
    free = torch.cuda.mem_get_info()[0]
    if free < 8 << 30:
        pytest.skip("needs 6 GB of device memory")
    cache = w4.KV8Cache(*(torch.empty(s, dtype=d, device="cuda") for s, d in
                          (((P, H, T, D), torch.int8), ((P, H, T // 16), torch.float32)) * 2))
    n = 300
    table = np.array([[39999, 3, 36001]], np.int32)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((n, H, D), generator=g).half() for _ in range(2))
    w4.kv8_append(cache, k.cuda(), v.cuda(), _i32(table), _i32([0]), _cu([n]))
    small = w4.KV8Cache(*(t[[39999, 3, 36001]].contiguous() for t in cache))
    want = w4.kv8_cache(3, H, T, D)
    w4.kv8_append(want, k.cuda(), v.cuda(), _i32([[0, 1, 2]]), _i32([0]), _cu([n]))
    for a, b in zip(w4.kv8_read(small, _i32([[0, 1, 2]]), _cu([n]), n), w4.kv8_read(want, _i32([[0, 1, 2]]), _cu([n]), n)):
        assert torch.equal(a, b)
    for a, b in zip(w4.kv8_read(cache, _i32(table), _cu([n]), n), w4.kv8_read(want, _i32([[0, 1, 2]]), _cu([n]), n)):
        assert torch.equal(a, b)
    q = torch.randn((1, 8, D), generator=g).half().cuda()
    assert torch.equal(w4.decode_attention_kv8(q, cache, _i32(table), _i32([n])),
                       w4.decode_attention_kv8(q, want, _i32([[0, 1, 2]]), _i32([n])))
    lens = _i32([n])
    moved, held = w4.kv8_compact(cache, _i32(table), lens)
    assert held.item() == 3 and sorted(moved[0].tolist()) == [0, 1, 2]
    for a, b in zip(w4.kv8_read(cache, moved, _cu([n]), n), w4.kv8_read(want, _i32([[0, 1, 2]]), _cu([n]), n)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ pages

def _held(table, lens, T):
    return sorted({int(p) for row, n in zip(table, lens) for p in row[:-(-n // T)]})


@pytest.mark.parametrize("extra", [0, 5000])
@pytest.mark.parametrize("P", [1, 31, 32, 33, 255, 256, 257, 5000, 300001])
def test_free_pages(w4, P, extra):
    T = 16
    rs = np.random.RandomState(P)
    lens = [int(x) for x in rs.randint(0, 5 * T, 12)] if P > 100 else [min(P, 3) * T - 5, 0]
    table = _table(lens, T, P, seed=P, extra=extra)
    cache = w4.kv8_cache(P, 1, T, 64)
    ids, count = w4.kv8_free_pages(cache, _i32(table), _i32(lens))
    want = sorted(set(range(P)) - set(_held(table, lens, T)))
    assert count.item() == len(want)
    assert ids.tolist() == want + [-1] * (P - len(want))
    assert w4.get_device_status() == 0


@pytest.mark.parametrize("T,H,D", [(16, 1, 64), (64, 3, 128), (128, 1, 256)])
def test_fork(w4, T, H, D):
    lens = [T, T + 1, 3 * T - 1, 5, 0, 40, 0, 0, 0, 0, 0]
    P = 20
    cache = _random_cache(w4, P, H, T, D, seed=1)
    table = _table(lens, T, P, seed=2, extra=1)
    td, ld = _i32(table), _i32(lens)
    free = sorted(set(range(P)) - set(_held(table, lens, T)))
    src, dst = [0, 1, 2, 1, 4], [6, 7, 8, 9, 10]
    before = _np(cache)
    w4.kv8_fork(cache, td, ld, _i32(src), _i32(dst), _i32(free[:5]))
    want = [t.copy() for t in before]
    t2, l2 = table.copy(), list(lens)
    for i, (a, b) in enumerate(zip(src, dst)):
        n = -(-lens[a] // T)
        l2[b] = lens[a]
        t2[b] = list(table[a, :n]) + [-1] * (table.shape[1] - n)
        if lens[a] % T:
            t2[b, n - 1] = free[i]
            for t in want:
                t[free[i]] = t[table[a, n - 1]]
    assert np.array_equal(td.cpu().numpy(), t2) and ld.tolist() == l2
    for a, b in zip(_np(cache), want):
        assert np.array_equal(a, b)
    assert w4.get_device_status() == 0


def test_fork_refuses_bad_places(w4):
    T = 16
    cache = _random_cache(w4, 6, 1, T, 64, seed=1)
    table = np.array([[0, 1], [2, 99], [-1, -1], [-1, -1]], np.int32)
    lens = [20, 20, 0, 0]
    before = _np(cache)
    for src, dst, fresh in (([0], [9], [3]), ([-1], [2], [3]), ([0], [2], [6]), ([0], [2], [-1]), ([1], [2], [3]), ([4], [2], [3])):
        td, ld = _i32(table), _i32(lens)
        w4.kv8_fork(cache, td, ld, _i32(src), _i32(dst), _i32(fresh))
        assert w4.get_device_status() == ERR_PAGE
        assert np.array_equal(td.cpu().numpy(), table) and ld.tolist() == lens
    for a, b in zip(_np(cache), before):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("extra", [2, 5000])       # tables of either kind of marking
@pytest.mark.parametrize("P,T,H,D", [(9, 16, 1, 64), (64, 32, 2, 128), (257, 16, 3, 64), (3000, 16, 1, 64), (40, 128, 2, 256)])
def test_compact(w4, P, T, H, D, extra):
    rs = np.random.RandomState(P)
    lens, left = [], int(P * 0.6)
    while left > 0 and len(lens) < 30:
        n = int(rs.randint(0, min(left, 40) + 1))
        lens.append(max(0, n * T - int(rs.randint(0, T))))
        left -= n
    table = _table(lens, T, P, seed=P, extra=extra)
    if len(lens) > 1 and lens[0] > 0:                 # a shared page
        other = int(np.argmax(lens[1:])) + 1
        if lens[other] >= T and lens[0] >= T:
            table[other, 0] = table[0, 0]
    cache = _random_cache(w4, P, H, T, D, seed=2)
    before = _np(cache)
    td, ld = _i32(table), _i32(lens)
    out, count = w4.kv8_compact(cache, td, ld)
    held = _held(table, lens, T)
    n = len(held)
    to = dict(zip([p for p in held if p >= n], sorted(set(range(n)) - set(held))))
    want = np.full_like(table, -1)
    for b, m in enumerate(lens):
        for i in range(-(-m // T)):
            want[b, i] = to.get(int(table[b, i]), int(table[b, i]))
    assert count.item() == n
    assert np.array_equal(out.cpu().numpy(), want)
    assert np.array_equal(td.cpu().numpy(), table)
    for a, b in zip(_np(cache), before):
        c = b.copy()
        for s, d in to.items():
            c[d] = b[s]
        assert np.array_equal(a, c)
    assert w4.get_device_status() == 0


def test_bad_pages_are_left_out_of_the_lists(w4):
    T = 16
    cache = _random_cache(w4, 8, 1, T, 64, seed=1)
    table, lens = np.array([[7, 200, -3], [5, 5, 1]], np.int32), [48, 20]
    ids, count = w4.kv8_free_pages(cache, _i32(table), _i32(lens))
    assert w4.get_device_status() == ERR_PAGE
    assert count.item() == 6 and ids.tolist()[:6] == [0, 1, 2, 3, 4, 6]
    out, count = w4.kv8_compact(cache, _i32(table), _i32(lens))
    assert w4.get_device_status() == ERR_PAGE
    assert count.item() == 2 and out.tolist() == [[1, -1, -1], [0, 0, -1]]


def test_another_stream_and_a_graph(w4):
    lens, T, D = [300, 70], 32, 128
    cache = _random_cache(w4, 20, 1, T, D, seed=1)
    table, ld = _i32(_table(lens, T, 20, 1)), _i32(lens)
    q = torch.randn((2, 8, D), generator=torch.Generator().manual_seed(1)).half().cuda()
    want = w4.decode_attention_kv8(q, cache, table, ld)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = w4.decode_attention_kv8(q, cache, table, ld)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(w4.lib().w4a8_decode_attention_kv8_workspace_bytes(2, 8, 1, D, T, table.shape[1]), dtype=torch.uint8,
                     device="cuda")
    new = torch.randn((2, 1, D), generator=torch.Generator().manual_seed(2)).half().cuda()
    one, out = _cu([1, 1]), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    more = ld.clone()
    with torch.cuda.graph(graph):
        w4.kv8_append(cache, new, new, table, ld, one)
        more.copy_(ld)
        more.add_(1)
        w4.decode_attention_kv8(q, cache, table, more, out=out, workspace=ws)
    copy = w4.KV8Cache(*(t.clone() for t in cache))
    graph.replay()
    torch.cuda.synchronize()
    w4.kv8_append(copy, new, new, table, ld, one)
    assert torch.equal(out, w4.decode_attention_kv8(q, copy, table, ld + 1))
    for a, b in zip(cache, copy):
        assert torch.equal(a, b)


def test_same_result_every_time(w4):
    lens, T, D = [5000, 70, 900], 16, 128
    P = sum(-(-n // T) for n in lens)
    cache = _random_cache(w4, P, 2, T, D, seed=1)
    table, ld = _i32(_table(lens, T, P, 1)), _i32(lens)
    q = torch.randn((3, 8, D), generator=torch.Generator().manual_seed(1)).half().cuda()
    first = w4.decode_attention_kv8(q, cache, table, ld)
    for _ in range(20):
        assert torch.equal(w4.decode_attention_kv8(q, cache, table, ld), first)


def test_refusals(w4):
    cache = w4.kv8_cache(4, 2, 16, 64)
    table, lens = _i32([[0, 1]]), _i32([20])
    q = torch.zeros((1, 4, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        w4.decode_attention_kv8(q, cache, table, _i32([1, 2]))
    with pytest.raises(ValueError):
        w4.decode_attention_kv8(q, cache._replace(k_scale=cache.k_scale[:, :1]), table, lens)
    with pytest.raises(TypeError):
        w4.decode_attention_kv8(q.float(), cache, table, lens)
    with pytest.raises(w4.W4A8Error):
        w4.decode_attention_kv8(q[:, :3].contiguous(), cache, table, lens)
    with pytest.raises(w4.W4A8Error):
        w4.decode_attention_kv8(q, cache, table.repeat(1, 200), lens, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        w4.kv8_append(cache, q, q, table, lens, _cu([1]))
    with pytest.raises(TypeError):
        w4.kv8_fork(cache, table, lens, lens.long(), lens, lens)
    with pytest.raises(w4.W4A8Error):
        w4.kv8_compact(cache, table, lens, table_out=table)
