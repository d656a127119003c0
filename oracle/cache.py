"""The 4-bit key/value cache and the attention over it, restated in fp64.  Test infrastructure
like ``reference.py``, whose rotation it builds on."""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import numpy as np

from . import reference as ref

__all__ = ["E2M1_VALUES", "e2m1_decode", "e2m1_encode", "kv_quantise", "kv_dequantise", "kv_pack", "kv_unpack",
           "kv_places", "kv_attention"]

# nibble -> value: a sign, two bits of exponent, one of mantissa
E2M1_VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e2m1_decode(nibbles: np.ndarray) -> np.ndarray:
    return E2M1_VALUES[np.asarray(nibbles)]


def e2m1_encode(r: np.ndarray) -> np.ndarray:
    """Nibble of the value nearest to r, ties to the even index, at most 6, with r's sign bit."""
    r = np.asarray(r, dtype=np.float64)
    far = np.abs(np.minimum(np.abs(r), 6.0)[..., None] - E2M1_VALUES[:8])
    near = far == far.min(-1, keepdims=True)
    tie = near.sum(-1) == 2
    first = near.argmax(-1)                              # the lower index of a tie
    return (np.where(tie & (first % 2 == 1), first + 1, first) + 8 * np.signbit(r)).astype(np.uint8)


def _rotate(x: np.ndarray) -> np.ndarray:
    D = x.shape[-1]
    return (np.asarray(x, dtype=np.float64).reshape(-1, D) @ ref.sylvester_hadamard(D).astype(np.float64)).reshape(x.shape)


def kv_quantise(x: np.ndarray, rotate: bool) -> Tuple[np.ndarray, np.ndarray]:
    """Heads [..., D] -> (nibbles uint8 [..., D], scales fp32 [...])."""
    v = (_rotate(x) if rotate else np.asarray(x, dtype=np.float64)).astype(np.float32)
    s = np.abs(v).max(-1) / np.float32(6)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(s[..., None] > 0, v / s[..., None], np.float32(0))
    q = np.where(s[..., None] > 0, e2m1_encode(r), 0).astype(np.uint8)
    c = np.float32(1 / np.sqrt(x.shape[-1])) if rotate else np.float32(1)
    return q, (s * c).astype(np.float32)


def kv_dequantise(nibbles: np.ndarray, scales: np.ndarray, rotate: bool) -> np.ndarray:
    """The heads that codes and scales stand for, rotated back."""
    x = e2m1_decode(nibbles)
    if rotate:
        x = _rotate(x) / np.sqrt(x.shape[-1])
    return x * np.asarray(scales, dtype=np.float64)[..., None]


def kv_pack(nibbles: np.ndarray) -> np.ndarray:
    return (nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)).astype(np.uint8)


def kv_unpack(codes: np.ndarray) -> np.ndarray:
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def kv_places(T: int, lens: Sequence[int], offsets: Optional[Sequence[int]], table: np.ndarray, page: int,
              n_pages: int) -> np.ndarray:
    """Of each of T tokens: (sequence or -1, position, page or -1, place in the page)."""
    B = len(lens)
    if offsets is None:
        offsets = [b * (T // B) for b in range(B + 1)] if B else [0]
    out = np.full((T, 4), -1, dtype=np.int64)
    for b in range(B):
        for t in range(offsets[b], offsets[b + 1]):
            pos = int(lens[b]) - offsets[b + 1] + t
            out[t, :2] = b, pos
            if pos >= 0 and pos // page < table.shape[1] and 0 <= table[b, pos // page] < n_pages:
                out[t, 2:] = table[b, pos // page], pos % page
    return out


def kv_attention(k: np.ndarray, v: np.ndarray, held: np.ndarray, q: np.ndarray, pos: np.ndarray, length: int,
                 scale: float, causal: bool, window: int):
    """One sequence.  k, v: [L][n_kv][D] in fp64; held: [L], which positions hold anything; q:
    [n][n_q][D]; pos: [n].  Returns (out [n][n_q][D], p [n][n_q][L], a [n][n_q][L])."""
    n, n_q, D = q.shape
    L, n_kv = k.shape[0], k.shape[1]
    j = np.arange(L)
    out, ps, sc = np.zeros((n, n_q, D)), np.zeros((n, n_q, L)), np.full((n, n_q, L), -np.inf)
    for i in range(n):
        see = held & (j < length)
        if causal:
            see &= j <= pos[i]
        if window:
            see &= j > pos[i] - window
        at = np.flatnonzero(see)
        if len(at) == 0:
            continue
        for h in range(n_q):
            g = h // (n_q // n_kv)
            a = scale * (k[at, g] @ q[i, h])
            p = np.exp(a - a.max())
            p /= p.sum()
            out[i, h] = p @ v[at, g]
            ps[i, h, at], sc[i, h, at] = p, a
    return out, ps, sc
