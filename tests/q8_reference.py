"""Codes of 8 bits under power-of-two scales, and attention over them, in 64 bits.

Bound of an attention output value over a cache of codes, from the number formats. With
u the unit roundoff of the rows' type (2^-11 FP16, 2^-8 BF16), A = sum_j p_j |v_j|, v_j
the values that the codes of V stand for, and `most` = top * the largest scale of V:

    u |out|, 2^-25            the output's rounding: FP16's values below 2^-14 lie 2^-24 apart,
                              so that one is off by up to 2^-25 there, however small it is
  + 2^-11 A                   the weights' (probability times scale) rounding to FP16 operands
  + n 2^-32 most              operands below FP16's normal range: half a step of 2^-24
                              where the largest is 2^7
  + (e_s + e_a) A             FP32 arithmetic, as in attention_reference: e_s = 2 (dim 2^-23
                              max_j sum_i |q_i k_ji| scale + 2^-19), e_a = 2 (n/8 + 64) 2^-23

A score is good to dim rounded additions, two factors more (2^-23 of it, in the first
term), and BF16 rows of q as FP16 operands under a power of two are exact but for
elements 2^-28 below the row's largest, off by 2^-39 of it: in the first term too.
2^x is good to 2^-21, for the probability and for the scale's factor.
"""
import numpy as np
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
BLOCK = 16


def scale_of(largest, store):
    """The smallest 2^e, e >= -126, with largest <= top 2^e; NaN of what is not finite."""
    top = TOP[store]
    m, e = np.frexp(largest)  # m in [1/2, 1)
    tm, te = np.frexp(top)
    e = np.where(largest > 0, e - te + (m > tm), -126)
    return np.where(np.isfinite(largest), np.ldexp(1.0, np.maximum(e, -126).astype(int)), np.nan)


def round_codes(y, store):
    """The nearest code's value, ties to even."""
    if store == torch.int8:
        return np.rint(y)
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))  # 3 bits behind the first, and subnormals of 2^-9
    return np.rint(y / step) * step


class Coded:
    """One sequence's K (or V) of one layer, block by block: code values and scales."""

    def __init__(self, store, heads, dim):
        self.store, self.heads, self.dim = store, heads, dim
        self.codes = np.zeros((0, heads, dim))
        self.scales = np.zeros((0, heads))

    def append(self, x):
        """x: (tokens, heads, dim) as they are given to one append."""
        x, old = np.asarray(x, dtype=np.float64), len(self.codes)
        self.codes = np.concatenate([self.codes, np.zeros_like(x)])
        at = 0
        while at < len(x):
            b = (old + at) // BLOCK
            here = min((b + 1) * BLOCK - old - at, len(x) - at)
            part = x[at:at + here]
            scale = scale_of(np.abs(part).max((0, 2)), self.store)
            kept = slice(b * BLOCK, old + at)
            if (old + at) % BLOCK == 0:
                self.scales = np.concatenate([self.scales, scale[None]])
            else:
                scale = np.where(np.isnan(self.scales[b]) | np.isnan(scale), np.nan, np.fmax(self.scales[b], scale))
                with np.errstate(invalid="ignore"):
                    self.codes[kept] = round_codes(self.codes[kept] * (self.scales[b] / scale)[None, :, None], self.store)
                self.scales[b] = scale
            with np.errstate(invalid="ignore"):
                self.codes[old + at:old + at + here] = round_codes(part / scale[None, :, None], self.store)
            at += here

    def values(self):
        return self.codes * np.repeat(self.scales, BLOCK, 0)[:len(self.codes), :, None]


def attend(q, k, v, scale):
    """q (m, d), k, v (n, d): (out, A, largest sum |q k|) in 64 bits."""
    q, k, v = q.double(), k.double(), v.double()
    p = torch.softmax((q @ k.T) * scale, 1)
    return p @ v, p @ v.abs(), (q.abs() @ k.abs().T).max() * scale


def assert_near(got, out, A, qk, n, dim, most, largest=0.0):
    u = U[got.dtype]
    es = 2 * (dim * 2.0 ** -23 * qk + 2.0 ** -19)
    ea = 2 * (n / 8 + 64) * 2.0 ** -23
    least = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    tol = (u * out.abs()).clamp(min=least) + (2.0 ** -11 + es + ea) * A + n * (2.0 ** -32 * most + 2.0 ** -126 * largest)
    d = (got.double() - out).abs()
    assert torch.isfinite(got).all()
    assert bool((d <= tol).all()), f"error {float(d.max()):.3e}, {float((d / tol.clamp(min=1e-300)).max()):.2f} of its bound"
