"""Weights far below their row's largest: one key takes nearly all of the softmax, and many others far below it add up in channels
where that key's value is zero; keys whose values are zeros beside large ones.  Scores of any size."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from kv_steps import DEV, Step  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


# cached and new tokens, query heads, channels: 16 rows a block, whole and cut; 128 rows a block, whole and cut
@pytest.mark.parametrize("length,new,n_q,D", [(700, 1, 4, 64), (1500, 3, 5, 128), (20000, 1, 8, 128), (900, 132, 32, 64),
                                              (5000, 130, 32, 128)])
@pytest.mark.parametrize("gap", [12, 21, 24, 27, 30])
def test_one_key_above_many(length, new, n_q, D, gap):
    """Key 0's score lies `gap` binades above the others', which are equal.  The score's product is exact: c = scale * log2(e) is 2^-4
    within 2^-23 of it, the query's values are bf16 and, times c, fp16 values.  So a weight's relative error is that of the
    exponential and its argument (gap * 2^-22 in all is ample) and its rounding to fp16, which is at most 2^-11 of it or 2^-32 of the
    row's largest weight, whichever is more.  All roundings may point the same way.  The sums of non-negative terms in fp32 add
    2^-24 a term of a lane's (a quarter of the keys at most).  Then half a step of bf16."""
    st = Step(length + gap, [length], [new], 1, D, 64, rotate=0, garbage=False)
    for c in st.codes:
        c[:] = 0
    for s in st.scales:
        s[:] = 1
    st.codes[1][..., :D // 4] = 0x77                           # the first half's channels are 6 in every value
    p = st.table[0, 0]
    st.codes[0][p, 0, 0, 0] = 0x07                             # key 0: 6 in channel 0
    st.codes[1][p, 0, 0, :D // 4], st.codes[1][p, 0, 0, D // 4:] = 0, 0x77
    st.device()
    scale = float(np.float32(math.log(2) / 16))
    assert abs(float(np.float32(scale) * np.float32(1.44269504088896341)) * 16 - 1) <= 2.0 ** -23
    q = torch.zeros((new, n_q, D), dtype=torch.bfloat16)
    q[..., 0] = gap * 16 / 6
    assert bool((q[..., 0].double() * 6 == gap * 16).all())
    got = cbq.kv_attention(st.cache, q.to(DEV), st.d_lens, scale=scale, **st.at).double().cpu().numpy()
    n = np.arange(length - new, length)[:, None]               # the other keys that a token attends
    w = 2.0 ** -gap
    for part, want, few in ((got[..., :D // 2], 6 * n * w / (1 + n * w), True), (got[..., D // 2:], 6 / (1 + n * w), False)):
        rel = max(2.0 ** -11, 2.0 ** -32 / w) if few else 2.0 ** -11
        rel += gap * 2.0 ** -22 + 2 * length / 4 * 2.0 ** -24 + 2.0 ** -8
        off = float((np.abs(part - want[..., None]) / want[..., None]).max())
        assert off <= rel, f"off by {off:.2e} of the value, at most {rel:.2e}"


@pytest.mark.parametrize("new,n_q", [(1, 2), (130, 32)])
@pytest.mark.parametrize("power", [-40, 0, 50, 60, 66])
def test_a_zero_value_beside_large_ones(new, n_q, power):
    """Half of the keys have a value of zeros (scale 0, which counts as 2^-64), half one of 6 * 2^power; all scores are 0.  The zero
    values' contributions lie 2^-(64 + power) below the others', and their weights still count in the softmax's sum."""
    length, D = 200, 64
    st = Step(abs(power) + new, [length], [new], 1, D, 16, rotate=0, garbage=False)
    pos = np.arange(length)
    for c in st.codes:
        c[:] = 0
    st.scales[1][:] = 0
    at = pos[pos % 2 == 1]
    st.codes[1][st.table[0, at // 16], 0, at % 16] = 0x77
    st.scales[1][st.table[0, at // 16], 0, at % 16] = 2.0 ** power
    st.device()
    q = torch.ones((new, n_q, D), dtype=torch.bfloat16, device=DEV)
    got = cbq.kv_attention(st.cache, q, st.d_lens, **st.at).double().cpu().numpy()
    seen = np.arange(length - new + 1, length + 1)
    want = 6 * 2.0 ** power * (seen // 2) / seen
    # the exponential and the sums in fp32, 2^-18 at most; fp16's and bf16's half steps
    off = float((np.abs(got - want[:, None, None]) / want[:, None, None]).max())
    assert off <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18


@pytest.mark.parametrize("length,new,n_q", [(1300, 1, 2), (700, 130, 32), (4000, 1, 2)])
@pytest.mark.parametrize("power", [10, 20, 23, 24, 25, 26, 28, 40])
def test_scores_of_any_size(length, new, n_q, power):
    """Scores near 2^power binades: key 0's, and the largest of the later tiles', which lies two steps of fp32 (of 8 binades, if these
    are smaller) above.  All are exact, so weights are powers of two: finite, and right to a step of bf16 and of fp16."""
    step = max(8.0, 2 * 2.0 ** (power - 23))
    st = Step(power + new, [length], [new], 1, 64, 64, rotate=0, garbage=False)
    for c in st.codes:
        c[:] = 0
    for s in st.scales:
        s[:] = 1
    j = np.arange(0, length - new, 64)                       # a key in each tile has a score
    st.codes[0][st.table[0, j // 64], 0, 0, 0] = 0x02         # 1 in channel 0
    st.scales[0][st.table[0, j // 64], 0, 0] = 2.0 ** power + step
    st.scales[0][st.table[0, 0], 0, 0] = 2.0 ** power
    st.codes[1][st.table[0, j // 64], 0, 0, :] = 0x77
    st.codes[1][st.table[0, 0], 0, 0, :] = 0x22              # 1, and 6 in the others
    st.device()
    scale = float(np.float32(math.log(2) / 16))
    while float(np.float32(np.float32(scale) * np.float32(1.44269504088896341))) != 2.0 ** -4:
        scale = float(np.nextafter(np.float32(scale), np.float32(1 if scale * 1.4426950408889634 < 2.0 ** -4 else 0)))
    q = torch.zeros((new, n_q, 64), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 16
    got = cbq.kv_attention(st.cache, q, st.d_lens, scale=scale, **st.at).double().cpu().numpy()
    n, w = len(j) - 1, 2.0 ** -step
    want = (6 * n + w) / (n + w)
    bad = int((~(np.abs(got / want - 1) <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18)).sum())
    assert bad == 0, f"{bad} of {got.size} values, {int((~np.isfinite(got)).sum())} of them not finite"
