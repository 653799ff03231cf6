"""Attention in 64 bits and the bound its GPU results are held to.

Bound of one output value, from the number formats: with u the unit roundoff of
the type (2^-11 FP16, 2^-8 BF16) and A = sum_j p_j |v_j|,

    u |out|                 the output's rounding
  + u A                     the probabilities' rounding to matrix operands
  + n 2^-32 max|v|          FP16 only: operands below 2^-14 (the largest is at
                            least 2^6) are spaced 2^-24
  + (e_s + e_a) A           FP32 arithmetic

e_s = 2 (dim 2^-23 max_j sum_i |q_i k_ji| scale + 2^-20): a score's error is at
most dim rounded (or cut) additions, enters numerator and denominator, and
2^x is good to 2^-21; e_a = 2 (n/8 + 64) 2^-23: the products' sums and the joins.
"""
import numpy as np
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def attend(q, k, v, seen, scale):
    """q (m, d), k, v (n, d), seen (m, n) bool: (out, A, largest sum |q k|) in 64 bits; rows that see nothing are 0."""
    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.T) * scale
    s = torch.where(seen, s, torch.full_like(s, -np.inf))
    top = s.amax(1, keepdim=True)
    e = torch.where(seen, torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top))), torch.zeros_like(s))
    p = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    return p @ v, p @ v.abs(), (q.abs() @ k.abs().T).max() * scale


def assert_near(got, out, A, qk, n, dim, dtype, vmax):
    u = U[dtype]
    es = 2 * (dim * 2.0 ** -23 * qk + 2.0 ** -20)
    ea = 2 * (n / 8 + 64) * 2.0 ** -23
    tol = u * out.abs() + (u + es + ea) * A + (n * 2.0 ** -32 * vmax if dtype == torch.float16 else 0.0)
    d = (got.double() - out).abs()
    assert torch.isfinite(got).all()
    assert bool((d <= tol).all()), f"error {float(d.max()):.3e}, {float((d / tol.clamp(min=1e-300)).max()):.2f} of its bound"
