"""Rows whose keys all lie in pages that were given back, beside rows of the same block that attend something: zeros, whatever
their queries hold."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from kv_steps import DEV, Step, check_attention  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


# lens, new tokens (the first `dead` of them see nothing but the pages `gone`), n_q, n_kv, D, page, window
CASES = [
    ([40], [40], 16, [0], 4, 1, 64, 16, 0),                    # 16 rows a block: pages end inside a tile of 64 keys
    ([32], [24], 8, [0], 1, 1, 128, 16, 0),                    # rows of both kinds in one block of 16 rows
    ([60], [60], 32, [0, 1], 3, 1, 64, 16, 0),
    ([90], [90], 48, [0, 1, 2], 2, 2, 128, 16, 0),
    ([3000], [40], 16, list(range(182, 186)), 3, 1, 64, 16, 40),  # windows that begin behind the keys they still hold
    ([140], [140], 32, [0], 32, 1, 64, 32, 0),                 # 128 rows a block
    ([200], [200], 16, [0], 64, 2, 128, 16, 0),
    ([2600], [140], 12, list(range(151, 156)), 32, 1, 64, 16, 30),
]


@pytest.mark.parametrize("lens,new,dead,gone,n_q,n_kv,D,page,window", CASES)
def test_queries_that_are_not_finite_over_pages_given_back(lens, new, dead, gone, n_q, n_kv, D, page, window):
    st = Step(sum(lens) + n_q, lens, new, n_kv, D, page)
    st.table[0, gone] = -1
    held = np.repeat(st.table[0] >= 0, page)
    for i in range(dead):                                      # the case is what it says
        pos = lens[0] - new[0] + i
        assert not held[max(0, pos + 1 - window if window else 0):pos + 1].any()
    assert held[lens[0] - 1]
    st.device()
    check_attention(st, n_q, window=window)
    q = torch.randn((st.T, n_q, D), device=DEV).to(torch.bfloat16)
    want = cbq.kv_attention(st.cache, q, st.d_lens, window=window, **st.at)
    zeros, some = not bool(want[:dead].any()), bool(want[dead:].any())
    assert zeros and some
    for bad in (float("nan"), float("inf"), float("-inf")):
        q[:dead] = bad
        got = cbq.kv_attention(st.cache, q, st.d_lens, window=window, **st.at)
        wrong = int((got[:dead] != 0).sum())
        assert wrong == 0, f"{bad}: {wrong} values of tokens that attend nothing are not zero"
        same = torch.equal(got[dead:], want[dead:])
        assert same, "the other tokens' results"
