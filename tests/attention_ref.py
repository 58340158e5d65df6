"""Attention in 64 bits on the CPU, with the bound that the GPU tests hold the
kernels to.

The kernels form x = scale q.k in fp32 (products of fp16 values are exact in
it; a sum of D of them is off by at most 2 D 2^-24 sum |q_d k_d|, also where
the tensor cores truncate), the weight p = 2^(x log2 e - m) (a relative error
of 2^-20 covers the exponent's rounding and the exponential for |x| up to some
dozens), round p to fp16 for the product with v (2^-11 relative; at most 2^-25
absolute where that is below fp16's normal range, against a largest weight of
at least 1), sum n products in fp32 (n/16 accumulations, each off by 2^-23 of
the sum of magnitudes), and round the quotient to fp16 (2^-11 relative, 2^-25
below fp16's normal range).  With A = sum p|v| / sum p, dx the bound on x:
  |err| <= A (2^-11 + 2 (dx + 2^-20) + (n/16 + 2) 2^-22) + n 2^-25 max|v| / sum p + 2^-11 |o| + 2^-25.
"""
import torch


def attention(q, k, v, scale, see=None):
    """q [r][D], k, v [n][D] -> (out [r][D], bound [r][D]) in 64 bits; see: bool [r][n], which keys a row sees."""
    q, k, v = q.double(), k.double(), v.double()
    n, D = k.shape
    if n == 0:
        z = torch.zeros(q.shape, dtype=torch.float64)
        return z, z + 2.0 ** -25
    x = q @ k.T * scale
    dx = q.abs() @ k.abs().T * scale * 2 * D * 2.0 ** -24
    if see is not None:
        x = x.masked_fill(~see, -torch.inf)
        dx = dx.masked_fill(~see, 0.0)
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - top.masked_fill(top == -torch.inf, 0.0))
    tot = p.sum(1, keepdim=True)
    some = tot > 0
    tot = tot.masked_fill(~some, 1.0)
    o = (p @ v / tot).masked_fill(~some, 0.0)
    A = p @ v.abs() / tot
    rel = 2.0 ** -11 + 2 * (dx.amax(1, keepdim=True) + 2.0 ** -20) + (n / 16 + 2) * 2.0 ** -22
    bound = A * rel + n * 2.0 ** -25 * v.abs().max() / tot + 2.0 ** -11 * o.abs() + 2.0 ** -25
    return o, bound


def check(got, ref, bound, what=""):
    err = (got.double().cpu() - ref).abs()
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    assert worst <= 1.0, f"{what}: error {worst:.3g} times the bound"
