"""Steps over a paged 4-bit cache for the tests: random caches whose unused places hold garbage, and
the oracle's attention with the bound its arithmetic gives."""
import numpy as np
import torch

import codebook_bit_quantized_amd as cbq
import oracle

DEV = "cuda:0"


class Step:
    """lens and new: cached and new tokens of each sequence; front, back: tokens of no sequence around them."""

    def __init__(self, seed, lens, new, n_kv, D, page, rotate=3, spare=2, front=0, back=0, max_pages=None, garbage=True,
                 table=True):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.new, self.n_kv, self.D, self.page, self.rotate = list(lens), list(new), n_kv, D, page, rotate
        B = len(lens)
        need = [max(0, -(-n // page)) for n in lens]
        self.max_pages = max_pages or max(need + [1])
        self.offsets = [front]
        for n in new:
            self.offsets.append(self.offsets[-1] + n)
        self.T = self.offsets[-1] + back
        if table:
            used = [min(n, self.max_pages) for n in need]
            self.n_pages = sum(used) + spare
            ids = rng.permutation(self.n_pages)
            self.table = np.full((B, self.max_pages), -1, dtype=np.int32)
            at = 0
            for b, n in enumerate(used):
                self.table[b, :n] = ids[at:at + n]
                at += n
        else:
            self.n_pages = max(1, B * self.max_pages)
            self.table = np.arange(B * self.max_pages, dtype=np.int32).reshape(B, self.max_pages)
        self.has_table = table
        shape = (self.n_pages, n_kv, page)
        self.codes = [rng.integers(0, 256, shape + (D // 2,), dtype=np.uint8) for _ in "kv"]
        self.scales = [(0.1 + rng.random(shape)).astype(np.float32) * np.float32(0.5) for _ in "kv"]
        if garbage:                                       # what no sequence holds is NaN, infinite or large
            held = np.zeros((self.n_pages, page), dtype=bool)
            for b in range(B):
                for j in range(min(max(self.lens[b], 0), self.max_pages * page)):
                    p = self.table[b, j // page]
                    if 0 <= p < self.n_pages:
                        held[p, j % page] = True
            bad = np.array([np.nan, np.inf, -np.inf, 3e38, -3e38], dtype=np.float32)
            for s in self.scales:
                m = np.broadcast_to(~held[:, None, :], s.shape)
                s[m] = bad[rng.integers(0, len(bad), m.sum())]

    def device(self):
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        self.cache = cbq.KVCache(up(self.codes[0]), up(self.codes[1]), up(self.scales[0]), up(self.scales[1]), self.rotate)
        self.d_lens = up(np.array(self.lens, dtype=np.int32))
        self.d_offsets = up(np.array(self.offsets, dtype=np.int32))
        self.at = dict(block_table=up(self.table) if self.has_table else None, offsets=self.d_offsets)
        return self

    def places(self):
        return oracle.kv_places(self.T, self.lens, self.offsets, self.table, self.page, self.n_pages)

    def sequence(self, b):
        """(k, v) [L][n_kv][D] of sequence b in fp64 (rotated back), and which positions hold anything."""
        L = min(max(self.lens[b], 0), self.max_pages * self.page)
        j = np.arange(L)
        p = self.table[b, j // self.page]
        held = (p >= 0) & (p < self.n_pages)
        p = np.where(held, p, 0)
        out = []
        for i in range(2):
            s = np.where(held[:, None], self.scales[i][p, :, j % self.page], 0)
            out.append(oracle.kv_dequantise(oracle.kv_unpack(self.codes[i][p, :, j % self.page]), s, bool(self.rotate >> i & 1)))
        return out[0], out[1], held

    def attention(self, q, scale, causal=True, window=0):
        """(out [T][n_q][D] fp64, bound of the same shape, rows that belong to a sequence)."""
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        mine = np.zeros(self.T, dtype=bool)
        for b in range(len(self.lens)):
            t0, t1 = self.offsets[b], self.offsets[b + 1]
            if t0 == t1:
                continue
            mine[t0:t1] = True
            k, v, held = self.sequence(b)
            pos = np.arange(t0, t1) + self.lens[b] - t1
            out[t0:t1], tol[t0:t1] = attention_and_bound(k, v, held, q[t0:t1], pos, self.lens[b], scale, causal, window)
        return out, tol, mine


def attention_and_bound(k, v, held, q, pos, length, scale, causal, window):
    """The oracle's attention of one sequence, and how far a result may be from it.

    The bound, with u = 2^-11 of fp16 and everything relative to a row's largest value:
    a score moves by at most d = |scale| |q||k| (u + 2^-17) (the rotated queries in fp16, fp32
    sums of 128 products), so a weight by 2 d and u of its own; a weight below fp16's normal
    range by 2^-25 of the largest one; the exponential, its argument and the normalisation
    in fp32 by 2^-18 of a score's size at most.  The rotation back keeps lengths.  Then half a step of bf16."""
    with np.errstate(invalid="ignore", over="ignore"):
        out, p, a = oracle.kv_attention(k, v, held, q, pos, length, scale, causal, window)
    n, n_q, D = q.shape
    tol = np.zeros(q.shape)
    for i in range(n):
        for h in range(n_q):
            w = p[i, h]
            at = np.flatnonzero(w)
            if len(at) == 0:
                continue
            g = h // (n_q // k.shape[1])
            kn, vn = np.linalg.norm(k[at, g], axis=1), np.linalg.norm(v[at, g], axis=1)
            d = abs(scale) * np.linalg.norm(q[i, h]) * kn.max() * (2.0 ** -11 + 2.0 ** -17)
            d += np.abs(a[i, h, at]).max() * 2.0 ** -18
            err = (w[at] * vn).sum() * (np.expm1(2 * d) + 2.0 ** -11 + 2.0 ** -18)
            # an E2M1 row's error is at most 6 sqrt(D) of its scale, its length at least half of it
            err += len(at) * 2.0 ** -25 * 12 * np.sqrt(D) * (w[at] * vn).max()
            tol[i, h] = err
    return out, tol + 2.0 ** -8 * np.abs(out) + 1e-37


def bf16_values(rng, shape, spread=1.0):
    x = torch.from_numpy(rng.normal(size=shape).astype(np.float32) * np.float32(spread)).to(torch.bfloat16)
    return x, x.double().numpy()


def check_attention(step, n_q, q_spread=1.5, scale=None, causal=True, window=0, **kw):
    scale = step.D ** -0.5 if scale is None else scale
    q, q64 = bf16_values(step.rng, (step.T, n_q, step.D), q_spread)
    want, tol, mine = step.attention(q64, scale, causal, window)
    out = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    got = cbq.kv_attention(step.cache, q.to(DEV), step.d_lens, scale=scale, causal=causal, window=window, out=out, **step.at, **kw)
    assert got is out
    g = got.double().cpu().numpy()
    assert np.all(g[~mine] == 77.0), "rows of no sequence were written"
    off = np.abs(g[mine] - want[mine])
    bad = ~(off <= tol[mine])
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs beyond the bound; worst {np.nanmax(off / tol[mine]):.2f} of it, " \
                          f"{np.isnan(g[mine]).sum()} NaN, first at {np.argwhere(bad)[0]}"
    return q, got, off.max(initial=0)
