"""The bound of kv_exact.py on results that are wrong: each must be rejected.  On the CPU, with the definition in 64 bits, rounded to
bf16, in the kernel's place."""
import numpy as np
import pytest
import torch

pytest.importorskip("codebook_bit_quantized_amd")
from kv_exact import CASES, beyond, step_of  # noqa: E402


def _bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def _tokens(st, n=6):
    """The first and last new tokens of the longest sequence, some between them, and others."""
    b = int(np.argmax(st.lens))
    own = np.arange(st.offsets[b], st.offsets[b + 1])
    return b, np.unique(np.r_[own[np.linspace(0, len(own) - 1, min(len(own), n)).astype(int)],
                              np.random.default_rng(0).choice(st.mine(), 2)])


@pytest.mark.parametrize("name", CASES)
def test_wrong_results_are_rejected(name):
    st, causal, window = step_of(name)
    b, at = _tokens(st)
    rotated = bool(st.rotate & 2)
    want, rel = st.outputs(at, causal, window)
    assert rel.max() < 0.006
    wrong = lambda x: beyond(_bf16(x), want, rel, rotated)  # noqa: E731
    assert wrong(want) == 0 and wrong(want * (1 + 2.0 ** -11)) == 0
    assert wrong(np.zeros_like(want)) and wrong(want * 1.02)
    L = st.lens[b]
    if L > 100 and not window == 1:
        for s in (0.98, 1.02, 1.05):
            assert wrong(st.outputs(at, causal, window, scale=s * st.scale)[0]), f"the scores {s} times what they are"
        assert wrong(np.roll(want, 1, axis=1)), "another head's results"
    if L == 1:
        return
    last = (L - 1) // 64                                   # the last whole tile that a token attends
    tiles = [last - 1] + ([0, last // 2] if not window else [])
    if L >= 200 and not window == 1:
        for t in tiles:
            assert wrong(st.outputs(at, causal, window, without=(b, slice(64 * t, 64 * t + 64)))[0]), f"without keys {64 * t} ..."
        every = np.arange(L)
        for w in (0, 5):                                   # what one of eight waves takes
            if (every // 64 % 8 == w).sum() and not window:
                assert wrong(st.outputs(at, causal, window, without=(b, every // 64 % 8 == w))[0]), f"without wave {w}'s tiles"
    if L <= 1200 and not window:
        assert wrong(st.outputs(at, causal, window, without=(b, [0]))[0]), "without key 0"
    if 1 < window <= 200 and L > window:
        assert wrong(st.outputs(at, causal, window + 1)[0]) and wrong(st.outputs(at, causal, window - 1)[0]), "the window one off"
    if causal and L <= 1200 and st.new[b] > 1:
        assert wrong(st.outputs(at, False, 0)[0]) , "not causal"
