"""Inputs for the few-token MoE layer on which its matrix products are exact in fp32, and the
bound that its output then meets element by element.

Codes are integers, codebooks small integers and token scales powers of two, so g, u and the
products of down with the codes of h are exact in fp32 in any order of summation (below 2^24
units).  What is left, with e = 2^-24:

* h = silu(g) * u in fp32: an exponential and a division of at most 2 and 2.5 units in the
  last place and three roundings, at most 12 e |h|;
* the rotated h: d_u = 12 e times the sum of |h| over its block, or times 6 root of the sum of
  h^2 where that is less: the roundings of a block's values are independent, so by Hoeffding's
  inequality one in 3e7 sums leaves that (an error that all values share scales the whole row
  and moves no code).  It moves the scale s by d_u / max|u|, relatively, and another 2 e for
  its own roundings;
* v / s: at most 2 d_u / s (|v| <= max|u| = Q s) plus Q e for its rounding.
  Only a code whose exact v / s lies that close to a rounding border may differ, by one step;
* y: 40 e for the routing weight (its argument 8 e, exponentials, their sum, a division), 16 e
  for the sum over at most 16 rows and 8 e for the scale factors, times the rows' magnitudes.

So |dy| <= sum_rows w (|out| (64 e + d_u / max|u|) + s sum_(codes at risk) |W_down|)."""
import numpy as np

import datagen
import oracle

EPS = 2.0 ** -24


def _weights(rng, E, N, K, bits):
    vals = np.array([-4, -3, -2, -1, 1, 2, 3, 4], dtype=np.float16)
    return datagen.WeightSet(E, N, K, bits, rng.integers(0, 256, (E, N, K * bits // 8), dtype=np.uint8),
                             rng.choice(vals, (E, N, 1 << bits)).view(np.uint16))


def exact_layer(T, H, F, E, topk, n_shared, bits_gu, bits_d, act_bits, seed=0):
    """(codes q [T][H], token scales, logits, gate, up, down)"""
    rng = np.random.default_rng([seed, T, H, F, E, topk, n_shared, bits_gu, bits_d, act_bits])
    Q = 7 if act_bits == 4 else 127
    q = np.clip(np.rint(rng.standard_normal((T, H)) * Q / 3.5), -Q, Q).astype(np.int64)
    unit = -np.round(np.log2(Q / 3.5 * 2.7 * np.sqrt(H)))            # g and u of about unit size
    scales = (2.0 ** (unit + rng.integers(-1, 2, T))).astype(np.float32)
    n = E + n_shared
    return (q, scales, rng.standard_normal((T, E)).astype(np.float32), _weights(rng, n, F, H, bits_gu),
            _weights(rng, n, F, H, bits_gu), _weights(rng, n, H, F, bits_d))


def bound(want, down, act_bits):
    """The largest |dy| [T][H], want being oracle.moe_layer_few on inputs of exact_layer."""
    h, sh = np.abs(want["h"]), want["sh"].astype(np.float64)
    R, F = h.shape
    T, H = want["y"].shape
    b = oracle.block_size(F)
    Q = 7 if act_bits == 4 else 127
    u = oracle.reference.rotate_fp64(want["h"], b)
    top = np.abs(u).max(axis=1)
    s = np.where(top > 0, top / Q, 1.0)
    hb = h.reshape(R, F // b, b)
    d_u = 12 * EPS * np.minimum(hb.sum(axis=2), 6 * np.sqrt((hb * hb).sum(axis=2))).max(axis=1)
    r = u / s[:, None]
    near = 2 * d_u / s + Q * EPS
    risk = np.abs(r - np.floor(r) - 0.5) <= near[:, None]
    wts = np.concatenate([want["route"]["weights64"].ravel(), np.ones(R - want["route"]["weights64"].size)])
    tol = np.zeros((T, H))
    for i in range(R):
        row = np.abs(want["out"][i]) * (64 * EPS + d_u[i] / max(top[i], 1e-300))
        c = np.nonzero(risk[i])[0]
        if len(c):
            e = want["expert"][i]
            W = oracle.dequantize(oracle.unpack_indices(down.idx[e], F, down.bits), down.codebook[e])
            row = row + sh[i] * np.abs(W[:, c]).sum(axis=1)
        tol[want["token"][i]] += wts[i] * row
    return tol
