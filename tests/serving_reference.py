"""Plain implementations, in 64 bits on the CPU, of the single-token serving
operators, with the error each result may have.

Tolerances count roundings (u = half a step of the type the value is held
in) and are evaluated element by element next to the exact value:

  product   a sum of K terms held in fp32, in whatever order: (K / 16 + 8)
            2^-23 of the sum of magnitudes, as the tensor-core product's test
            counts it.  fp32 operands enter as two fp16 terms, 22 bits:
            2^-21 of the sum of magnitudes.
  softmax   an error dx of a score changes its weight by the factor e^dx, the
            quotient of two such sums by 2 dx; a weight rounded to fp16 is off
            by 2^-11 (two terms: 2^-21); exponential and logarithm by 2^-20.
            Weights are held times 2^11 (over a reference at most the largest
            weight) in fp16, whose spacing ends at 2^-24: below 2^-14 a weight
            is off by up to half of that, 2^-25, which is 2^-36 of the largest
            weight (one), whatever the weight's own size, so a result by 2^-36
            sum_j |v_j|.  MXFP4 holds w_j 2^(E_j) relative
            to the largest such product (E_j the token's largest block
            exponent, |v_j| <= 6 2^(E_j)): 2^-36 max_j(w_j 2^(E_j)) sum_j
            |v_j| 2^(-E_j).  With 2^(E_j) <= max_d |v_j| * 2 (the largest
            block holds a code of at least one half wherever it is not zero)
            this is computed from the values themselves.
  result    one rounding to the output's type.
"""
import numpy as np
import torch

import oracle

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], np.float64)
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def scale_values(fmt_nv):
    """The value of every scale byte, from its bit fields."""
    out = np.full(256, np.nan)
    for b in range(256):
        if not fmt_nv:
            out[b] = 2.0 ** (b - 127) if b < 255 else np.nan
        elif b & 127 != 127:
            e, m = (b >> 3) & 15, b & 7
            out[b] = (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) * (-1 if b & 128 else 1)
    return out


def decode(packed, scales, nv, g=1.0):
    """Values (64 bits) of packed [..., C/2] and scales [..., C/G]; g broadcast against the scales."""
    codes = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)
    s = scale_values(nv)[scales] * (np.asarray(g, np.float64) if nv else 1.0)
    return E2M1[codes] * np.repeat(s, 16 if nv else 32, -1)


def oracle_input(x: torch.Tensor):
    x = x.cpu().contiguous()
    return x.view(torch.int16).numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.numpy()


def quantize_rows(x: torch.Tensor, nv, g=None, rule=0):
    """The oracle's codes and scale bytes of x [T, H, D]; g fp32 [H]."""
    T, H, D = x.shape
    a = oracle_input(x)
    packed = np.zeros((T, H, D // 2), np.uint8)
    scales = np.zeros((T, H, D // (16 if nv else 32)), np.uint8)
    for h in range(H):
        rows = np.ascontiguousarray(a[:, h])
        r = oracle.nvfp4_quantize_with_g(rows, float(g[h])) if nv else oracle.mxfp4_quantize_rule(rows, rule)
        packed[:, h], scales[:, h] = r[0].reshape(T, -1), r[1].reshape(T, -1)
    return packed, scales


def attention(q, k, v, lens, scale, window, mx=False):
    """q [B, L, HQ, D]; k, v: lists of [n, H, D] arrays (64 bits).  Returns out, lse and their tolerances before the
    output's rounding is added (out_tol needs the output dtype's half step times |out| on top)."""
    B, L, HQ, D = q.shape
    two = q.dtype == torch.float32
    q = q.double().cpu().numpy()
    out, lse = np.zeros((B, L, HQ, D)), np.full((B, L, HQ), -np.inf)
    tol, ltol = np.zeros_like(out), np.zeros((B, L, HQ))
    for b in range(B):
        n = lens[b]
        group = HQ // k[b].shape[1]
        for i in range(L):
            p = n - L + i
            lo = max(0, p - window + 1) if window else 0
            if p < lo:
                continue
            for h in range(HQ):
                kk, vv = k[b][lo:p + 1, h // group], v[b][lo:p + 1, h // group]
                x = kk @ q[b, i, h] * scale
                mag = np.abs(kk) @ np.abs(q[b, i, h]) * abs(scale)
                dx = np.max(((D / 16 + 8) * 2.0 ** -23 + (2.0 ** -21 if two else 0)) * mag + 2.0 ** -21 * np.abs(x)) + 2.0 ** -20
                m = x.max()
                w = np.exp(x - m)
                s = w.sum()
                w /= s
                lse[b, i, h] = m + np.log(s)
                out[b, i, h] = w @ vv
                tol[b, i, h] = (2 * dx + (2.0 ** -21 if two else 2.0 ** -11) + ((p - lo + 1) / 16 + 8) * 2.0 ** -23) * (w @ np.abs(vv))
                if mx:
                    big = 2 * np.abs(vv).max(1)
                    unit = np.abs(vv) / np.where(big > 0, big, 1)[:, None] * 12
                    tol[b, i, h] += 2.0 ** -36 * (w * big).max() * unit.sum(0)
                else:
                    tol[b, i, h] += 2.0 ** -36 * w.max() * np.abs(vv).sum(0)
                ltol[b, i, h] = dx + 2.0 ** -22 * abs(lse[b, i, h]) + ((p - lo + 1) / 16 + 8) * 2.0 ** -23 + 2.0 ** -20
    return out, lse, tol, ltol


def linear(x, w):
    """x [rows, K] times w [N, K] (64 bits): y and its tolerance before the output's rounding."""
    a = x.double().cpu().numpy()
    y, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    K = x.shape[1]
    return y, ((K / 16 + 8) * 2.0 ** -23 + (2.0 ** -21 if x.dtype == torch.float32 else 0)) * mag
