"""Plain 64-bit definitions of the rotation, cache and tree operators, and the
tolerances that follow from their roundings (each off by at most half a step:
2^-8 of the value for bf16)."""
import math

import numpy as np
import torch

import oracle

PAGE = 64
BF16 = 2.0 ** -8


def norm_rope(x, w, positions, inv_freq, interleaved, eps=1e-6):
    """x [..., tokens, d] float64, positions [tokens] -> (y, bound on |y - bf16 result|)."""
    x = x.double()
    d = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + eps) * w.double()
    rot = 2 * len(inv_freq)
    angle = positions.double()[:, None] * inv_freq.double()[None]
    c, s = angle.cos(), angle.sin()
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y, size = x.clone(), x.abs()
    xa, xb = x[..., a], x[..., b]
    y[..., a] = xa * c - xb * s
    y[..., b] = xb * c + xa * s
    both = xa.abs() + xb.abs()
    size[..., a], size[..., b] = both, both
    # fp32: the mean over d <= 128 values, rsqrt, two products and the rotation
    # stay within 16 roundings of 2^-24 of |a| + |b|; the angle within 2^-22 rad
    return y, BF16 * y.abs() + 2.0 ** -20 * size + 1e-37


def quantised(x):
    """Codes and scales of bf16 vectors [..., d], by the C oracle."""
    x = x.cpu().contiguous()
    n = x.numel() // x.shape[-1]
    codes, scales = oracle.quantize_e4m3(x, n)
    return (torch.from_numpy(codes).view(x.shape),
            torch.from_numpy(scales.astype(np.float32)).view(x.shape[:-1]))


def dequantised(codes, scales):
    values = torch.from_numpy(oracle.e4m3_values())
    return values[codes.cpu().long()] * scales.cpu().double()[..., None]


def tree(q, K, V, mask_bits, T):
    """One sequence: q [T, Hq, d], K, V [Hkv, len, d] float64 -> (o, bound).

    mask_bits: T ints, or None for a chain.  The kernels round P to bf16 and
    sum the rounded values, so o = sum p (1 + e) v / sum p (1 + e) with
    |e| <= 2^-8, which moves it by at most 2^-8 (sum p |v| / sum p + |o|); a
    score's fp32 error (128 products of up to a few hundred in all, and the
    exponent's rounding) adds at most 2^-11 to e; the result is rounded once.
    """
    T_, Hq, d = q.shape
    Hkv, n, _ = K.shape
    g = Hq // Hkv
    prefix = max(0, n - T)
    sees = torch.zeros(T_, n, dtype=torch.bool, device=q.device)
    sees[:, :prefix] = True
    for i in range(T_):
        for j in range(n - prefix):
            sees[i, prefix + j] = bool(((mask_bits[i] >> j) & 1) if mask_bits is not None else j <= i)
    o = torch.zeros(T_, Hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    for h in range(Hq):
        x = q[:, h].double() @ K[h // g].T / math.sqrt(d)
        x = torch.where(sees, x, -math.inf)
        some = sees.any(1)
        if not some.any():
            continue
        p = torch.zeros_like(x)
        p[some] = torch.softmax(x[some], -1)
        # a value that a token does not see is no part of its sum, NaN or not
        v = V[h // g]
        o[:, h] = torch.stack([p[i, sees[i]] @ v[sees[i]] for i in range(T_)])
        size = torch.stack([p[i, sees[i]] @ v[sees[i]].abs() for i in range(T_)])
        tol[:, h] = (BF16 + 2.0 ** -11) * (size + o[:, h].abs()) + BF16 * o[:, h].abs() + 1e-30
    return o, tol


def close(got, want, tol, what=""):
    err = (got.double().cpu() - want.cpu()).abs()
    bad = ~(err <= tol.cpu())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol.cpu()).nan_to_num(1e9).max()):.3g} of the bound"
