"""64-bit references of the rotary, dense decode and eviction operators, and the
error bounds of the kernels' arithmetic.  Test-only, plain numpy on the host."""
from __future__ import annotations

import math

import numpy as np

BF16 = 2.0 ** -8    # half a step, relative
FP16 = 2.0 ** -11
FP32 = 2.0 ** -24


def rope(x, pos, axis, freqs, adjacent):
    """x [n][heads][dim] float64, pos int [axes][n] -> (y, bound)."""
    y, mag = x.copy(), np.zeros_like(x)
    half = len(axis)
    for i in range(half):
        a = pos[axis[i]].astype(np.float64) * freqs[i]
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        d0, d1 = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        x0, x1 = x[..., d0], x[..., d1]
        y[..., d0], y[..., d1] = x0 * c - x1 * s, x1 * c + x0 * s
        mag[..., d0] = mag[..., d1] = np.abs(x0) + np.abs(x1)
    # one rounding to BF16; the angle (reduced in 64 bits, then held in 32: pi * 2^-24 at most), sin, cos
    # (1 ulp) and three fp32 operations: below 8 half steps of fp32 on |x0| + |x1|
    return y, BF16 * np.abs(y) + 8 * FP32 * mag + 1e-30


def dense(q, k, v, scale, fp8):
    """One query: q [hq][256], k, v [n][hkv][256] (float64) -> out, lse, weights [n] (summed over heads) and bounds."""
    hq, (n, hkv) = q.shape[0], k.shape[:2]
    out, lse = np.zeros((hq, 256)), np.full(hq, -np.inf)
    w_sum, out_b, lse_b, w_b = np.zeros(n), np.zeros((hq, 256)), np.zeros(hq), np.zeros(n)
    if n == 0:
        return out, lse, w_sum, out_b, lse_b, w_b
    group = hq // hkv
    for h in range(hq):
        g = h // group
        z = scale * (k[:, g] @ q[h])
        m = z.max()
        e = np.exp(z - m)
        lse[h] = m + math.log(e.sum())
        w = np.exp(z - lse[h])
        out[h] = w @ v[:, g]
        # a logit: 256 exact products summed in fp32, each addition off by at most a step (2 half steps,
        # the tensor cores may truncate) of the sum of magnitudes, then the scale and the base-2 subtraction
        dz = (2 * 256 + 8) * FP32 * scale * np.max(np.abs(k[:, g]) @ np.abs(q[h])) + 8 * FP32 * (np.abs(z).max() + 1)
        # sums of n weights in fp32: split over tiles, at most 2 half steps per addition, n / 16 tiles deep
        ds = 2 * FP32 * (n / 16 + 64)
        # the weights entering P V: BF16 hi + lo leaves 2^-8 * 2^-8 half steps, FP16 half a step (and 2^-25 at least)
        dp = (FP16 + 2.0 ** -25) if fp8 else BF16 * BF16
        mag = w @ np.abs(v[:, g])
        out_b[h] = BF16 * np.abs(out[h]) + mag * (2 * dz + 2 * ds + dp) + (n * 2.0 ** -25 * np.abs(v[:, g]).max(0) / e.sum()
                                                                       if fp8 else 0) + 1e-30
        lse_b[h] = dz + ds + 8 * FP32 * (np.abs(lse[h]) + 1)
        w_sum += w
        w_b += w * (2 * dz + 2 * ds + 16 * FP32 * (np.abs(lse[h]) + 1)) + 2.0 ** -100
    return out, lse, w_sum, out_b, lse_b, w_b


def block_sums(x):
    nb = -(-len(x) // 4)
    y = np.zeros(nb * 4)
    y[:len(x)] = x
    return y.reshape(nb, 4).sum(1)


def keep_blocks(mass, length, budget, sink, recent):
    """Kept complete blocks, ascending.  A NaN ranks below every number; -0 ties with +0."""
    nb = length // 4
    if nb <= budget:
        return list(range(nb))
    rank = lambda b: (1, 0.0) if math.isnan(mass[b]) else (0, -float(mass[b]))
    mid = sorted(range(sink, nb - recent), key=lambda b: (rank(b), b))[:budget - sink - recent]
    return sorted(list(range(sink)) + mid + list(range(nb - recent, nb)))
