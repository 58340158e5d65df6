"""What is measured of the prompt attention and of the 8-bit paged KV cache.

Every case is one pass of one of four operators, either in a plain form
(elementary torch operations in 32 bits, `own` false) or through the library's
entry points (`own` true), on the same inputs:

  prompt  attention of packed sequences of different lengths, grouped heads,
          causal or not, the new tokens at the end of the keys (their prefix
          comes first);
  store   new tokens' keys and values quantised into the pages of an 8-bit
          cache (codes int8, one fp32 scale for each 16 tokens of a head), and
          the sequences read back from it as fp16;
  decode  attention of one new token per sequence over the 8-bit paged cache;
  pages   sequences forked (the page that both would write is copied) and the
          cache compacted (held pages moved to its front).

The sizes are those of the package's decoder layer (8 query heads of 256 on
one KV head, 512 prompt tokens, 640 tokens of context) and generic ones.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16          # tokens that share a scale


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # three chats that go on: a few new tokens each, on a prefix that is in the cache already
        dict(name="prompt_chunk_d256", op="prompt", B=3, L=37, ragged=True, prefix=500, Hq=8, Hkv=1, D=256, causal=True,
             fused=True, lens=11),
        # the decoder layer's own prompt: 512 tokens, 8 query heads on one KV head
        dict(name="prompt_512_d256", op="prompt", B=1, L=512, ragged=False, prefix=0, Hq=8, Hkv=1, D=256, causal=True,
             fused=True, lens=12),
        # a batch of prompts of very different lengths, packed; three query heads to a KV head
        dict(name="prompt_ragged_d64", op="prompt", B=12, L=2500, ragged=True, prefix=0, Hq=24, Hkv=8, D=64, causal=True,
             fused=True, lens=13),
        # one long document
        dict(name="prompt_long_d128", op="prompt", B=1, L=16384, ragged=False, prefix=0, Hq=16, Hkv=2, D=128, causal=True,
             fused=False, lens=14),
        # a decode step's tokens of 32 chats on the decoder layer's one KV head
        dict(name="store_token_d256", op="store", B=32, L=640, new=1, Hkv=1, D=256, T=64, lens=15),
        # a batch of prompts stored at once, some after a prefix
        dict(name="store_prompt_d128", op="store", B=9, L=4096, new=2500, Hkv=8, D=128, T=32, lens=16),
        # one chat's next token: latency
        dict(name="decode_one_d256", op="decode", B=1, L=640, ragged=False, Hq=8, Hkv=1, D=256, T=64, lens=17),
        # 32 chats at the decoder layer's context of 640 tokens
        dict(name="decode_batch_d256", op="decode", B=32, L=640, ragged=False, Hq=8, Hkv=1, D=256, T=64, lens=18),
        # a serving batch: 64 sequences, from a few tokens to 16384
        dict(name="decode_ragged_d128", op="decode", B=64, L=16384, ragged=True, Hq=32, Hkv=8, D=128, T=32, lens=19),
        # one sequence of 131072 tokens
        dict(name="decode_long_d128", op="decode", B=1, L=131072, ragged=False, Hq=16, Hkv=2, D=128, T=128, lens=20),
        # a few chats forked (two answers to one question) in a small cache
        dict(name="pages_small_d256", op="pages", B=16, L=640, forks=4, spare=1.6, Hkv=1, D=256, T=64, lens=21),
        # a large cache compacted after sequences left
        dict(name="pages_large_d128", op="pages", B=96, L=8192, forks=24, spare=1.8, Hkv=4, D=128, T=32, lens=22),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "store", "decode", "decode", "pages"])
    lens = rng.randrange(1 << 20)
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    T = rng.choice([16, 32, 64, 128])
    if op == "prompt":
        while True:
            Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
            c = dict(op=op, B=_log_int(rng, 1, 24), L=_log_int(rng, 1, 12000), ragged=rng.random() < 0.7,
                     prefix=rng.choice([0, 0, _log_int(rng, 1, 4000)]), Hq=Hq, Hkv=Hkv, D=D, causal=rng.random() < 0.8,
                     fused=rng.random() < 0.5, lens=lens)
            if c["B"] * Hq * c["L"] * (c["L"] + c["prefix"]) <= 16 * 16384 * 16384 and work(c)["flops"] <= 1.1e12:
                return c
    if op == "store":
        while True:
            L = _log_int(rng, 1, 8192)
            c = dict(op=op, B=_log_int(rng, 1, 64), L=L, new=rng.choice([1, _log_int(rng, 1, L)]), Hkv=Hkv, D=D, T=T, lens=lens)
            if c["B"] * L * Hkv * D <= 9 * 4096 * 8 * 128:
                return c
    if op == "decode":
        while True:
            Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
            c = dict(op=op, B=_log_int(rng, 1, 96), L=_log_int(rng, 1, 131072), ragged=rng.random() < 0.7, Hq=Hq, Hkv=Hkv,
                     D=D, T=T, lens=lens)
            if c["B"] * c["L"] * max(Hkv * D, Hq * 16) <= 64 * 16384 * 8 * 128 and work(c)["bytes"] <= 1.0e9:
                return c
    while True:
        B = _log_int(rng, 2, 96)
        c = dict(op=op, B=B, L=_log_int(rng, 16, 8192), forks=rng.randint(1, B), spare=rng.uniform(1.3, 2.0), Hkv=Hkv, D=D,
                 T=T, lens=lens)
        if B * c["L"] * Hkv * D <= 64 * 8192 * 4 * 128:
            return c


def _lengths(case):
    """The sequences' lengths: a function of the case alone (the seed changes the values, not the sizes)."""
    rs = np.random.RandomState(case["lens"] % (1 << 31))
    B, L = case["B"], case["L"]
    if case["op"] == "store":
        new = np.minimum(rs.randint(max(1, case["new"] // 2), case["new"] + 1, B), L)
        start = np.array([rs.randint(0, L - n + 1) for n in new])
        return start.astype(np.int64), new.astype(np.int64)
    if case["op"] == "pages" or case["ragged"]:
        lens = np.maximum(1, np.exp(rs.uniform(math.log(max(1.0, L / 30.0)), math.log(L), B))).astype(np.int64)
        lens[rs.randint(B)] = L
    else:
        lens = np.full(B, L, np.int64)
    if case["op"] == "prompt":
        pre = rs.randint(case["prefix"] // 2, case["prefix"] + 1, B) if case["prefix"] else np.zeros(B, np.int64)
        return lens, lens + pre
    return lens, lens


def _layout(case):
    """Pages in scattered order: (number of pages, table [sequences][pages of the longest], -1 where none is held)."""
    T = case["T"]
    a, b = _lengths(case)
    total = a + b if case["op"] == "store" else a
    forks = case.get("forks", 0)
    need = -(-total // T)
    count = int(math.ceil(int(need.sum() + forks) * case.get("spare", 1.1))) + 3
    order = np.random.RandomState((case["lens"] + 77) % (1 << 31)).permutation(count).astype(np.int32)
    table = np.full((len(total) + forks, int(need.max())), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return count, table


def _forks(case):
    """Which sequences are forked, and into which rows of the table."""
    src = np.random.RandomState((case["lens"] + 5) % (1 << 31)).randint(0, case["B"], case["forks"]).astype(np.int32)
    return src, (case["B"] + np.arange(case["forks"])).astype(np.int32)


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    row = D + 4.0 / BLOCK                # a token's codes and its share of the scale, of one head
    a, b = _lengths(case)
    if case["op"] == "prompt":
        lq, lk = a.astype(float), b.astype(float)
        pairs = lq * (lk - lq) + lq * (lq + 1) / 2 if case["causal"] else lq * lk
        return {"bytes": float(2 * D * (2 * case["Hq"] * lq.sum() + 2 * Hkv * lk.sum())), "flops": float(4 * D * case["Hq"] * pairs.sum())}
    if case["op"] == "store":
        new, every = float(b.sum()), float((a + b).sum())
        # in: fp16 keys and values; out: their codes; then every token's codes in and its fp16 values out
        return {"bytes": 2 * Hkv * (new * (2 * D + row) + every * (row + 2 * D)), "flops": 2 * Hkv * D * (2 * new + every)}
    if case["op"] == "decode":
        n = float(a.sum())
        return {"bytes": 2 * Hkv * n * row + 4 * D * case["Hq"] * case["B"], "flops": 4 * D * case["Hq"] * n}
    count, table = _layout(case)
    src, dst = _forks(case)
    T = case["T"]
    part = int((a[src] % T != 0).sum())
    # pages that the forks take come from the free ones, lowest first
    free = np.setdiff1d(np.arange(count), table[table >= 0])
    held = np.union1d(table[table >= 0], free[:len(src)][a[src] % T != 0])
    moved = int((held >= len(held)).sum())
    return {"bytes": (part + moved) * 2.0 * 2 * Hkv * T * row + 8.0 * table.size, "flops": 0.0}


# ------------------------------------------------------------------- the inputs

def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def _cu(lens):
    return _i32(np.concatenate([[0], np.cumsum(lens)]))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)


def _cache(g, case, count):
    shape = (count, case["Hkv"], case["T"], case["D"])

    def one():
        codes = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
        scale = torch.rand((count, case["Hkv"], case["T"] // BLOCK), generator=g, device="cuda") * 0.02 + 0.005
        return codes, scale
    kc, ks = one()
    vc, vs = one()
    return dict(kc=kc, ks=ks, vc=vc, vs=vs)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    Hkv, D = case["Hkv"], case["D"]
    a, b = _lengths(case)
    s = dict(case)
    if case["op"] == "prompt":
        nq, nk, Hq = int(a.sum()), int(b.sum()), case["Hq"]
        if case["fused"] and nq == nk:
            # the fused projection's output: a token's query heads, then its key and its value heads
            qkv = _randn(g, nq, Hq + 2 * Hkv, D)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            q, k, v = _randn(g, nq, Hq, D), _randn(g, nk, Hkv, D), _randn(g, nk, Hkv, D)
        q *= 1.5
        k[..., ::32] *= 2.0
        s.update(q=q, k=k, v=v, cu_q=_cu(a), cu_k=_cu(b), max_q=int(a.max()), max_k=int(b.max()))
        return s
    count, table = _layout(case)
    s.update(_cache(g, case, count), table=_i32(table))
    if case["op"] == "store":
        n = int(b.sum())
        k, v = _randn(g, n, Hkv, D), _randn(g, n, Hkv, D)
        k[..., ::32] *= 4.0
        s.update(k=k, v=v, start=_i32(a), cu_new=_cu(b), cu_all=_cu(a + b), total=int((a + b).sum()))
    elif case["op"] == "decode":
        s.update(q=_randn(g, case["B"], case["Hq"], D), lens=_i32(a))
    else:
        src, dst = _forks(case)
        s.update(lens=_i32(np.concatenate([a, np.zeros(case["forks"], np.int64)])), src=_i32(src), dst=_i32(dst))
    return s


# ------------------------------------------------------- one pass: the calls, or the plain form

def run(s):
    if s["op"] == "prompt":
        return _own_prompt(s) if own else _plain_prompt(s)
    if s["op"] == "store":
        return _own_store(s) if own else _plain_store(s)
    if s["op"] == "decode":
        return _own_decode(s) if own else _plain_decode(s)
    return _own_pages(s) if own else _plain_pages(s)


def _own_cache(s):
    import int4_weight_quantized_gb300 as w4
    return w4, w4.KV8Cache(s["kc"], s["ks"], s["vc"], s["vs"])


def _own_prompt(s):
    import int4_weight_quantized_gb300 as w4
    return w4.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["causal"])


def _own_store(s):
    w4, cache = _own_cache(s)
    w4.kv8_append(cache, s["k"], s["v"], s["table"], s["start"], s["cu_new"])
    return w4.kv8_read(cache, s["table"], s["cu_all"], s["total"])


def _own_decode(s):
    w4, cache = _own_cache(s)
    return w4.decode_attention_kv8(s["q"], cache, s["table"], s["lens"])


def _own_pages(s):
    w4, cache = _own_cache(s)
    table, lens = s["table"].clone(), s["lens"].clone()
    free, _ = w4.kv8_free_pages(cache, table, lens)
    w4.kv8_fork(cache, table, lens, s["src"], s["dst"], free[:s["forks"]])
    table, held = w4.kv8_compact(cache, table, lens)
    return [table, lens, held, s["kc"], s["ks"], s["vc"], s["vs"]]


def _padded(cu, most):
    """Rows of a packed tensor by sequence and place: (index [B][most], which of them there are)."""
    at = torch.arange(most, device=cu.device)
    lens = (cu[1:] - cu[:-1]).long()
    there = at[None] < lens[:, None]
    return torch.where(there, cu[:-1].long()[:, None] + at[None], 0), there, lens


def _plain_prompt(s):
    Hq, Hkv, D, G = s["Hq"], s["Hkv"], s["D"], s["Hq"] // s["Hkv"]
    iq, tq, lq = _padded(s["cu_q"], s["max_q"])
    ik, tk, lk = _padded(s["cu_k"], s["max_k"])
    B = iq.shape[0]
    q = s["q"][iq].float().view(B, -1, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)     # [B][Hkv][G tokens][D]
    k = s["k"][ik].float().permute(0, 2, 3, 1)
    v = torch.where(tk[:, :, None, None], s["v"][ik].float(), 0.0).permute(0, 2, 1, 3)
    x = torch.matmul(q, k).view(B, Hkv, G, s["max_q"], s["max_k"])
    x *= 1.0 / math.sqrt(D)
    mask = tk[:, None, :]
    if s["causal"]:
        row = torch.arange(s["max_q"], device=q.device)[None] + (lk - lq)[:, None]
        mask = mask & (torch.arange(s["max_k"], device=q.device)[None, None] <= row[:, :, None])
    x.masked_fill_(~mask[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x -= torch.where(top == -math.inf, 0.0, top)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, -1, s["max_k"]), v).view(B, Hkv, G, s["max_q"], D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, s["max_q"], Hq, D)
    return o[tq].half()


def _plain_put(codes, scale, x, page, token, start_page, start_token, some):
    """One of the two tensors: x [N][Hkv][D] fp32 at (page, token)[N]; each sequence's block at its start holds
    start_token % 16 earlier tokens (`some`: the sequences that bring new tokens)."""
    P, Hkv, T, D = codes.shape
    nb = T // BLOCK
    at = page * nb + token // BLOCK                                             # block of each token
    first = start_page * nb + start_token // BLOCK                              # and of each start
    first, held = first[some], (start_token % BLOCK)[some]
    flat = scale.transpose(1, 2).reshape(P * nb, Hkv)
    kept = torch.zeros(P * nb, dtype=torch.bool, device=x.device)
    kept[first] = held > 0
    old = torch.where(kept[:, None], flat, 0.0)
    amax = torch.zeros_like(flat).scatter_reduce(0, at[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    new = torch.maximum(old, amax / 127.0)
    blocks = codes.view(P, Hkv, nb, BLOCK, D)
    fp, fb = first // nb, first % nb
    was = blocks[fp, :, fb]                                                     # [B][Hkv][16][D]
    f = torch.where(new[first] > 0, old[first] / new[first], 1.0)[:, :, None, None]
    again = torch.round(was.float() * f).to(torch.int8)
    mine = torch.arange(BLOCK, device=x.device)[None] < held[:, None]
    blocks[fp, :, fb] = torch.where(mine[:, None, :, None], again, was)
    touched = torch.zeros(P * nb, dtype=torch.bool, device=x.device)
    touched[at] = True
    scale.copy_(torch.where(touched[:, None], new, flat).view(P, nb, Hkv).transpose(1, 2))
    sx = new[at][:, :, None]
    q = torch.where(sx > 0, torch.round(x / sx), 0.0).clamp(-127, 127)
    codes[page, :, token] = q.to(torch.int8)


def _plain_store(s):
    T = s["T"]
    cu, start, table = s["cu_new"].long(), s["start"].long(), s["table"].long()
    n = s["k"].shape[0]
    i = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu, i, right=True) - 1
    p = start[b] + i - cu[b]
    page, token = table[b, p // T], p % T
    start_page = table.gather(1, (start // T).clamp(max=table.shape[1] - 1)[:, None])[:, 0].clamp(min=0)
    some = cu[1:] > cu[:-1]
    _plain_put(s["kc"], s["ks"], s["k"].float(), page, token, start_page, start % T, some)
    _plain_put(s["vc"], s["vs"], s["v"].float(), page, token, start_page, start % T, some)
    cu = s["cu_all"].long()
    i = torch.arange(s["total"], device=cu.device)
    b = torch.searchsorted(cu, i, right=True) - 1
    p = i - cu[b]
    page, token = table[b, p // T], p % T
    return [(c[page, :, token].float() * f[page, :, token // BLOCK][:, :, None]).half()
            for c, f in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]


def _plain_values(codes, scale, table):
    """[B][Hkv][tokens][D] fp32 of the pages of `table`."""
    B, n = table.shape
    P, Hkv, T, D = codes.shape
    x = codes[table].float().view(B, n, Hkv, T // BLOCK, BLOCK, D)
    x *= scale[table][:, :, :, :, None, None]
    return x.permute(0, 2, 1, 3, 4, 5).reshape(B, Hkv, n * T, D)


def _plain_decode(s):
    B, Hq, Hkv, D = s["B"], s["Hq"], s["Hkv"], s["D"]
    table = s["table"].long().clamp(min=0)
    k, v = _plain_values(s["kc"], s["ks"], table), _plain_values(s["vc"], s["vs"], table)
    there = torch.arange(k.shape[2], device=k.device)[None] < s["lens"][:, None]
    x = torch.matmul(s["q"].float().view(B, Hkv, Hq // Hkv, D), k.transpose(2, 3)) / math.sqrt(D)
    x = torch.where(there[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v)
    return torch.where(total > 0, o / total, 0.0).reshape(B, Hq, D).half()


def _plain_held(s, table, lens):
    """Which pages are held, as a mask of all, and which entries of the table count."""
    P, T = s["kc"].shape[0], s["T"]
    counts = torch.arange(table.shape[1], device=table.device)[None] < ((lens.long() + T - 1) // T)[:, None]
    held = torch.zeros(P, dtype=torch.bool, device=table.device)
    held[table.long()[counts]] = True
    return held, counts


def _plain_pages(s):
    T = s["T"]
    table, lens = s["table"].clone(), s["lens"].clone()
    src, dst = s["src"].long(), s["dst"].long()
    held, _ = _plain_held(s, table, lens)
    fresh = torch.nonzero(~held)[:s["forks"], 0]
    # the fork: the table's row, and a copy of the page that is not full
    n = lens[src].long()
    part = n % T != 0
    rows = torch.where(torch.arange(table.shape[1], device=table.device)[None] < ((n + T - 1) // T)[:, None], table[src], -1)
    last = (n // T).clamp(max=table.shape[1] - 1)
    old = rows.gather(1, last[:, None])[:, 0].long()
    one, two = old[part], fresh[part]
    tensors = [s[x] for x in ("kc", "ks", "vc", "vs")]
    _ = [t.index_copy_(0, two, t[one]) for t in tensors]
    rows.scatter_(1, last[:, None], torch.where(part, fresh, old).int()[:, None])
    table[dst] = rows
    lens[dst] = n.int()
    # the compaction: held pages behind the front's end into the holes of the front
    held, counts = _plain_held(s, table, lens)
    total = held.sum()
    place = torch.arange(held.shape[0], device=table.device)
    hole = torch.nonzero(~held & (place < total))[:, 0]
    mover = torch.nonzero(held & (place >= total))[:, 0]
    _ = [t.index_copy_(0, hole, t[mover]) for t in tensors]
    to = place.int()
    to[mover] = hole.int()
    table = torch.where(counts, to[table.long().clamp(min=0)], -1)
    return [table, lens, total.int().view(1)] + tensors


# ----------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "store": _exact_store, "decode": _exact_decode, "pages": _exact_pages}[case["op"]](s)


def _exact_softmax(q, k, v, ok, scale):
    """softmax(q k^T scale) v of one head's rows, 64 bits; rows with nothing give zeros."""
    x = (q @ k.T) * scale
    x = torch.where(ok, x, -math.inf)
    top = x.max(1).values
    e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top)[:, None])
    e = torch.where(ok, e, 0.0)
    den = e.sum(1)
    return torch.where(den[:, None] > 0, (e @ v) / den[:, None], 0.0)


def _exact_prompt(s):
    if work({k: s[k] for k in ("op", "B", "L", "ragged", "prefix", "Hq", "Hkv", "D", "causal", "lens")})["flops"] > 4e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cq, ck, G = s["cu_q"].tolist(), s["cu_k"].tolist(), s["Hq"] // s["Hkv"]
    for b in range(s["B"]):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        for h in range(s["Hkv"]):
            k, v = (t[ck[b]:ck[b + 1], h].double() for t in (s["k"], s["v"]))
            for lo in range(0, nq, 4096):
                hi = min(nq, lo + 4096)
                end = nk - nq + hi if s["causal"] else nk
                i = torch.arange(lo, hi, device="cuda") + (nk - nq)
                ok = torch.arange(end, device="cuda")[None] <= i[:, None] if s["causal"] else torch.ones(hi - lo, nk, dtype=torch.bool, device="cuda")
                for g in range(h * G, h * G + G):
                    rows = slice(cq[b] + lo, cq[b] + hi)
                    out[rows, g] = _exact_softmax(s["q"][rows, g].double(), k[:end], v[:end], ok, s["D"] ** -0.5)
    return out


def _exact_store(s):
    T, start, cn, ca = s["T"], s["start"].tolist(), s["cu_new"].tolist(), s["cu_all"].tolist()
    table = s["table"].tolist()
    got = []
    for codes, scale, x in ((s["kc"], s["ks"], s["k"]), (s["vc"], s["vs"], s["v"])):
        rows = []
        for b in range(s["B"]):
            pages = torch.tensor([p for p in table[b] if p >= 0], device="cuda")
            n = ca[b + 1] - ca[b]
            c = codes[pages].double().permute(0, 2, 1, 3).reshape(-1, s["Hkv"], s["D"])          # [tokens][Hkv][D]
            f = scale[pages].double().permute(0, 2, 1).reshape(-1, s["Hkv"])                     # [blocks][Hkv]
            new = x[cn[b]:cn[b + 1]].double()
            lo, first, last = start[b], start[b] // BLOCK, -(-n // BLOCK)
            pad = torch.zeros(((last - first) * BLOCK,) + new.shape[1:], dtype=torch.float64, device="cuda")
            pad[lo - first * BLOCK:n - first * BLOCK] = new
            top = pad.view(last - first, BLOCK, s["Hkv"], s["D"]).abs().amax((1, 3)) / 127
            was = torch.zeros_like(top)
            if lo % BLOCK:
                was[0] = f[first]
            sc = torch.maximum(top, was)
            q = torch.round(pad.view(last - first, BLOCK, s["Hkv"], s["D"]) / sc[:, None, :, None]).nan_to_num(0.0)
            if lo % BLOCK:
                ratio = torch.where(sc[0] > 0, was[0] / sc[0], 1.0)
                q[0, :lo % BLOCK] = torch.round(c[first * BLOCK:lo] * ratio[None, :, None])
            mine = (q * sc[:, None, :, None]).reshape(-1, s["Hkv"], s["D"])
            before = c[:first * BLOCK] * f[:first].repeat_interleave(BLOCK, 0)[:, :, None]
            rows.append(torch.cat([before, mine])[:n])
        got.append(torch.cat(rows))
    return got


def _exact_decode(s):
    T, G, lens = s["T"], s["Hq"] // s["Hkv"], s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(s["B"]):
        pages = s["table"][b, :-(-lens[b] // T)].long()
        for h in range(s["Hkv"]):
            k, v = ((c[pages, h].double().view(-1, BLOCK, s["D"]) * f[pages, h].double().view(-1, 1, 1)).view(-1, s["D"])[:lens[b]]
                    for c, f in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            ok = torch.ones(G, lens[b], dtype=torch.bool, device="cuda")
            out[b, h * G:h * G + G] = _exact_softmax(s["q"][b, h * G:h * G + G].double(), k, v, ok, s["D"] ** -0.5)
    return out


def _exact_pages(s):
    T, P = s["T"], s["kc"].shape[0]
    table, lens, src, dst = s["table"].tolist(), s["lens"].tolist(), s["src"].tolist(), s["dst"].tolist()
    held = {p for row, n in zip(table, lens) for p in row[:-(-n // T)]}
    fresh = sorted(set(range(P)) - held)[:s["forks"]]
    moves = []
    was_table, was_lens = [list(r) for r in table], list(lens)
    for i, (a, b) in enumerate(zip(src, dst)):
        n = -(-was_lens[a] // T)
        table[b] = was_table[a][:n] + [-1] * (len(table[b]) - n)
        lens[b] = was_lens[a]
        if lens[b] % T:
            moves.append((table[b][n - 1], fresh[i]))
            table[b][n - 1] = fresh[i]
    held = sorted({p for row, n in zip(table, lens) for p in row[:-(-n // T)]})
    there = set(held)
    to = dict(zip([p for p in held if p >= len(held)], [p for p in range(len(held)) if p not in there]))
    table = [[to.get(p, p) for p in row[:-(-n // T)]] + [-1] * (len(row) - -(-n // T)) for row, n in zip(table, lens)]
    tensors = [s[x].clone() for x in ("kc", "ks", "vc", "vs")]
    for t in tensors:
        for step in (moves, list(to.items())):
            if step:
                one, two = (torch.tensor(c, device="cuda") for c in zip(*step))
                t[two] = t[one]
    return [torch.tensor(table, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32), torch.tensor([len(held)], dtype=torch.int32)] + [
        t if t.dtype == torch.int8 else t.double() for t in tensors]
