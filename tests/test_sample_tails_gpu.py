"""Sampling from rows whose last words weigh next to nothing and are many: the tokens that
numbers close to 1 draw, against the definition in exact arithmetic, and the same row drawn
in batches of other sizes, which other numbers of CTAs take."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

getcontext().prec = 60
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    from int4_weight_quantized_gb300.build import build
    build()
    import int4_weight_quantized_gb300 as w4
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return w4


def _f(x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


def _numbers(tail, n):
    """n numbers of 24 bits (or as many as there are) spread over the last `tail` of [0, 1)."""
    last = 1 << 24
    first = max(0, last - max(1, int(tail * last)))
    return sorted({first + (last - 1 - first) * i // max(1, n - 1) for i in range(n)})


def _check(got, runs, u, M):
    """runs: the words in order, as (index of the j-th, count, weight); u in 2^-24.  What is allowed beside the exact word:
    a weight is off by 2^-39.7 of itself at most and a run's words all alike, so a border moves by 2^-38 of the run's words;
    u M is rounded to 53 bits twice, and M and the sums before a run to whole units of 2^-59 of M or less: 2^-50 M in all."""
    tokens, logps = got[0].tolist(), got[1].tolist()
    for b, k in enumerate(u):
        border = Decimal(k) / (1 << 24) * M
        before = Decimal(0)
        allowed = {}
        for place, count, w in runs:
            at = (border - before) / w
            slack = Decimal(count) * Decimal(2) ** -38 + M * Decimal(2) ** -50 / w
            for x in (at - slack, at, at + slack):
                if 0 <= x < count:
                    allowed[place(int(x))] = w
            before += count * w
        assert tokens[b] in allowed, (b, k, tokens[b], allowed)
        want = float((allowed[tokens[b]] / M).ln())
        # (the weight and M are off by 2^-39.7 each, and the result is rounded to fp32)
        assert abs(logps[b] - want) <= abs(want) * 2.0 ** -24 + 2.0 ** -38, (b, logps[b], want)


def _step(T, d):
    return (Decimal(-d) / Decimal(torch.tensor(T, dtype=torch.float32).item())).exp()


# one word and, a step of fp16 (2^-6) below it, all the others
TAILS = [1e-3, 9e-4, 7.5e-4, 5e-2, 1.2e-3]


def _two_levels(w4, V, T, at, first, n=64):
    x = torch.full((1, V), first - 2.0 ** -6, dtype=torch.float16)
    x[0, at] = first
    w = _step(T, 2.0 ** -6)
    M = 1 + (V - 1) * w
    u = _numbers(float((V - 1) * w / M), n)
    got = w4.sample(x.cuda().expand(len(u), -1), _f(u) / 2 ** 24, _f([T] * len(u)))
    others = lambda j: j + (j >= at)      # noqa: E731
    _check(got, [(lambda j: at, 1, Decimal(1)), (others, V - 1, w)], u, M)


# the first value and the next one in one group of 32 values, and in two
@pytest.mark.parametrize("first", [20.484375, 20.0])
@pytest.mark.parametrize("T", TAILS)
@pytest.mark.parametrize("V,at", [(524272, 7), (524272, 524271), (262145, 131072), (70000, 30000)])
def test_one_step_below_the_first(w4, V, at, T, first):
    _two_levels(w4, V, T, at, first)


# weights of 2^-36.4 to 2^-42: of these a few numbers below 1 draw, each among thousands of words
@pytest.mark.parametrize("T", [6.2e-4, 6.07e-4, 6e-4, 5.91e-4, 5.8e-4, 5.71e-4, 5.63e-4, 5.55e-4, 5.5e-4, 5.45e-4, 5.4e-4, 5.37e-4])
@pytest.mark.parametrize("first", [20.484375, 20.0])
def test_words_that_few_numbers_reach(w4, T, first):
    for at in (0, 262144, 524271):
        _two_levels(w4, 524272, T, at, first)


@pytest.mark.parametrize("T", [0.3, 4e-3, 1.1e-3, 8e-4, 7.1e-4])
@pytest.mark.parametrize("V,n", [(524272, 200000), (300001, 65536), (131072, 1000)])
def test_many_first_words(w4, V, n, T):
    x = torch.full((1, V), 20.484375 - 2.0 ** -6, dtype=torch.float16)
    x[0, V - n:] = 20.484375
    w = _step(T, 2.0 ** -6)
    M = n + (V - n) * w
    for tail in (1.0, float((V - n) * w / M)):
        u = _numbers(tail, 64)
        got = w4.sample(x.cuda().expand(len(u), -1), _f(u) / 2 ** 24, _f([T] * len(u)))
        _check(got, [(lambda j: V - n + j, n, Decimal(1)), (lambda j: j, V - n, w)], u, M)


@pytest.mark.parametrize("T", [0.02, 0.0301, 0.11])
def test_three_levels(w4, T):
    # 5 words, 1000 of the same 32 values' group, and 260000 of another group
    V, first = 261005, 20.484375
    x = torch.full((1, V), first - 0.75, dtype=torch.float16)
    x[0, 100:1100] = first - 2.0 ** -5
    x[0, -5:] = first
    w1, w2 = _step(T, 2.0 ** -5), _step(T, 0.75)
    M = 5 + 1000 * w1 + 260000 * w2
    for tail in (float((1000 * w1 + 260000 * w2) / M), float(260000 * w2 / M), 1.0):
        u = _numbers(tail, 64)
        got = w4.sample(x.cuda().expand(len(u), -1), _f(u) / 2 ** 24, _f([T] * len(u)))
        runs = [(lambda j: V - 5 + j, 5, Decimal(1)), (lambda j: 100 + j, 1000, w1), (lambda j: j if j < 100 else j + 1000, 260000, w2)]
        _check(got, runs, u, M)


@pytest.mark.parametrize("V,B", [(30000, 200), (131072, 160), (262144, 64)])
def test_a_row_alone_and_in_a_batch(w4, V, B):
    """The words of a row are dealt out to 8 CTAs where it is alone and to as few as its words need in a batch: the sums are
    the same integers, so that tokens and log-probabilities are."""
    drawn = 0
    for seed in range(12):
        g = torch.Generator().manual_seed(seed)
        T = 0.2 + 0.02 * float(torch.rand(1, generator=g))
        # one word, and weights of about 2^-38 to 2^-44 in a few dozen groups of 32 values
        x = (torch.rand((1, V), generator=g) * 0.9 + 9.6 + (0.6 if V < 50000 else 0.0)).half()
        x[0, V // 3] = 16.0
        u = _f([(2 ** 24 - 1 - i) / 2 ** 24 for i in range(8)])
        d = x.cuda()
        many = w4.sample(d.expand(B, -1), u.repeat(B // 8), _f([T] * B))
        for i in range(8):
            one = w4.sample(d, u[i:i + 1], _f([T]))
            assert one[0].tolist() * (B // 8) == many[0][i::8].tolist(), (seed, i, one[0], many[0][i::8])
            assert one[1].tolist() * (B // 8) == many[1][i::8].tolist()
        drawn += len(set(many[0].tolist()) - {V // 3})
    assert drawn > 0 or V < 50000                                     # (the tail was drawn from)


def test_a_row_alone_and_in_a_batch_with_filters(w4):
    V, B = 131072, 160
    g = torch.Generator().manual_seed(5)
    x = (torch.randn((1, V), generator=g) * 2.5).half().cuda()
    u, T = torch.rand(B, generator=g).cuda(), _f([0.3 + 0.01 * b for b in range(B)])
    k = torch.randint(-3, 3000, (B,), generator=g, dtype=torch.int32).cuda()
    p, m = (torch.rand(B, generator=g) * 1.2).cuda(), (torch.rand(B, generator=g) * 0.02 - 0.01).cuda()
    many = w4.sample(x.expand(B, -1), u, T, k, p, m)
    for b in range(B):
        one = w4.sample(x, *(t[b:b + 1] for t in (u, T, k, p, m)))
        assert one[0].item() == many[0][b].item() and one[1].item() == many[1][b].item()
    assert math.isfinite(float(many[1].sum()))
