"""Steps whose attention is known closely: every product and score of the kernels is exact, every term of an output is
non-negative where the values are held, and an output's channels show which keys took which share of the softmax.

Keys are of four types.  A key of type t holds one value in the channels c with c % 4 == t and zero in the others, with a scale
that makes code times scale 2; a query (rotated, where the keys are) holds levels of 0 to 3 in one channel of each residue,
so the score of a key in binades is the level that the query holds for its type.  A value holds one channel, that of its
type and of its place among D / 4 stretches of the sequence, again with code times scale 2.  So channel by channel the
output is twice the softmax's sum over the keys of one type in one stretch.

How far a result may be off, relative, with roundings that all point the same way: a weight's rounding to fp16, 2^-11; its
exponential and argument, 2^-18 (arguments below 16, four roundings of 2^-24 of them and one of the result); the sums of
non-negative terms in fp32, 2^-24 a term: at most a quarter of the keys in a lane for the softmax's sum, and one addition for
32 keys (and 64 at the joins) in the matrix cores, taken as 2^-23 each; the rotation back 2^-18; and half a step of bf16,
2^-8.  That holds channel by channel where the values are not rotated, and for the length of the difference where
they are, as the rotation keeps lengths."""
import math

import numpy as np
import torch

import oracle
from kv_steps import Step

LOG2E = np.float32(1.44269504088896341)
PAIRS = np.array([[0.5, 4.0], [1.0, 2.0], [2.0, 1.0], [4.0, 0.5]])     # a code's value and the scale that make 2


class ExactStep(Step):
    def __init__(self, seed, lens, new, n_q, n_kv, D, page, rotate=3, **kw):
        super().__init__(seed, lens, new, n_kv, D, page, rotate, **kw)
        rng, self.n_q = self.rng, n_q
        nibble = oracle.e2m1_encode(PAIRS[:, 0])
        for b in range(len(self.lens)):
            L = min(max(self.lens[b], 0), self.max_pages * page)
            j = np.arange(L)
            p = self.table[b, j // page]
            j, p = j[p >= 0], p[p >= 0]
            kind = rng.integers(0, 4, (len(j), n_kv))
            where = kind * (D // 4) + (j * (D // 4) // max(L, 1))[:, None]
            channel = np.arange(D)
            for i, holds in enumerate((channel % 4 == kind[..., None], channel == where[..., None])):
                pick = rng.integers(0, 4, (len(j), n_kv))
                self.codes[i][p, :, j % page] = oracle.kv_pack(np.where(holds, nibble[pick][..., None], 0).astype(np.uint8))
                self.scales[i][p, :, j % page] = PAIRS[pick, 1]
        levels = rng.integers(0, 4, (self.T, n_q, 4))
        x = np.zeros((self.T, n_q, D))
        t, h, kind = np.meshgrid(np.arange(self.T), np.arange(n_q), np.arange(4), indexing="ij")
        x[t, h, 4 * rng.integers(0, D // 4, levels.shape) + kind] = D * levels
        if rotate & 1:
            x = (x.reshape(-1, D) @ oracle.sylvester_hadamard(D)).reshape(x.shape) / D
        self.q = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
        assert np.array_equal(self.q.double().numpy(), x)
        # the kernels' factor of the queries is 2^-e: code * scale * D * level * factor = level
        c_q = np.float32(1 / math.sqrt(D)) if rotate & 1 else np.float32(1)
        self.scale = float(np.float32(math.log(2) / (2 * D) / float(c_q)))
        assert abs(float(np.float32(self.scale) * c_q * LOG2E) * 2 * D - 1) <= 2.0 ** -22

    def outputs(self, tokens, causal=True, window=0, scale=None, without=None):
        """The definition in 64 bits for some tokens: [tokens][n_q][D], and the largest relative error of each.
        without: (sequence, positions) that are taken to hold nothing."""
        q = self.q.double().numpy()
        out, rel = np.zeros((len(tokens), self.n_q, self.D)), np.zeros(len(tokens))
        for b in range(len(self.lens)):
            mine = np.flatnonzero((tokens >= self.offsets[b]) & (tokens < self.offsets[b + 1]))
            if len(mine) == 0:
                continue
            k, v, held = self.sequence(b)
            if without is not None and without[0] == b:
                held = held.copy()
                held[without[1]] = False
            pos = tokens[mine] + self.lens[b] - self.offsets[b + 1]
            out[mine] = oracle.kv_attention(k, v, held, q[tokens[mine]], pos, self.lens[b], scale or self.scale, causal, window)[0]
            L = len(held)
            rel[mine] = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -17 + L / 4 * 2.0 ** -24 + (L / 32 + 64) * 2.0 ** -23
        return out, rel

    def mine(self):
        return np.arange(self.offsets[0], self.offsets[-1])


def beyond(got, want, rel, rotated):
    """How many rows (or, not rotated, values) are further off than rel says."""
    off = got - want
    if rotated:
        off, want = np.linalg.norm(off, axis=-1), np.linalg.norm(want, axis=-1)
        rel = rel[:, None]
    else:
        rel = rel[:, None, None]
    return int((~(np.abs(off) <= rel * np.abs(want))).sum())


# lens, new tokens, query heads, key/value heads, D, page, rotate, causal, window
CASES = {
    # 16 rows a block, whole
    "one key": ([1], [1], 4, 2, 64, 16, 3, True, 0),
    "a tile and one": ([65], [1], 8, 2, 128, 16, 3, True, 0),
    "129": ([129], [1], 8, 1, 128, 64, 0, True, 0),
    "one of 1000": ([1000], [1], 32, 4, 128, 16, 3, True, 0),
    "ragged": ([0, 1, 5, 64, 130, 300, 17], [0, 1, 2, 5, 40, 7, 17], 6, 2, 64, 16, 3, True, 0),
    "ragged, not rotated": ([300, 20, 77], [3, 20, 9], 5, 5, 128, 32, 0, True, 0),
    "keys rotated": ([500, 90], [5, 1], 8, 2, 64, 64, 1, True, 0),
    "values rotated": ([500, 90], [5, 1], 8, 2, 128, 64, 2, True, 0),
    "every position": ([250, 111], [7, 7], 4, 2, 128, 16, 0, False, 0),
    "many heads": ([90], [2], 96, 1, 64, 16, 3, True, 0),
    "more than 64 sequences": ([50, 0, 900] + [7] * 70 + [1200, 33], [1, 0, 3] + [1] * 70 + [2, 2], 4, 2, 64, 64, 3, True, 0),
    "window 1": ([90, 200], [3, 3], 4, 2, 64, 32, 0, True, 1),
    "window 16": ([90, 200], [1, 1], 8, 2, 64, 32, 3, True, 16),
    "window 33": ([90, 200], [40, 3], 4, 2, 128, 32, 3, True, 33),
    "window 100": ([90, 200, 333], [1, 3, 1], 8, 2, 64, 32, 3, True, 100),
    # 16 rows a block, cut
    "one of 40000": ([40000], [1], 8, 1, 128, 64, 3, True, 0),
    "one of 40000, not rotated": ([40000], [1], 8, 1, 128, 64, 0, True, 0),
    "20000, 3000 and 1": ([20000, 3000, 1], [1, 1, 1], 4, 2, 64, 64, 3, True, 0),
    "20 of 9000": ([9000, 12], [20, 3], 8, 1, 64, 64, 3, True, 0),
    "drafted": ([2500, 1700], [5, 5], 16, 4, 128, 64, 3, True, 0),
    "300 of 5000": ([5000], [300], 2, 2, 128, 64, 0, True, 0),
    "window 2500": ([5000, 3000, 40], [1, 1, 1], 8, 1, 64, 64, 3, True, 2500),
    # 128 rows a block, whole
    "prompts": ([300, 130], [300, 130], 16, 2, 64, 32, 3, True, 0),
    "prompts, not rotated": ([140, 64], [140, 64], 40, 1, 128, 128, 0, True, 0),
    "prompts, window 70": ([260], [260], 20, 1, 128, 16, 3, True, 70),
    # 128 rows a block, cut
    "132 of 2600": ([2600], [132], 32, 1, 64, 32, 3, True, 0),
    "132 of 2600, not rotated": ([2600], [132], 32, 1, 128, 32, 0, True, 0),
    "every position of 5000": ([5000], [65], 64, 1, 64, 64, 3, False, 0),
}
CUT = {"one of 40000", "one of 40000, not rotated", "20000, 3000 and 1", "20 of 9000", "drafted", "300 of 5000", "window 2500",
       "132 of 2600", "132 of 2600, not rotated", "every position of 5000"}
MANY_ROWS = {"prompts", "prompts, not rotated", "prompts, window 70", "132 of 2600", "132 of 2600, not rotated",
             "every position of 5000"}


def step_of(name):
    lens, new, n_q, n_kv, D, page, rotate, causal, window = CASES[name]
    return ExactStep(len(name) + sum(lens), lens, new, n_q, n_kv, D, page, rotate), causal, window
