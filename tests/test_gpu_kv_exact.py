"""cbq_kv_attention against a bound of half a percent: steps whose products and scores are exact (kv_exact.py), in every form of the
kernels.  test_kv_exact_bound.py has what the bound rejects."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from kv_exact import CASES, CUT, MANY_ROWS, ExactStep, beyond, step_of  # noqa: E402
from kv_steps import DEV  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


def _check(st, causal=True, window=0):
    """Whether row blocks were cut: a call of whole ones leaves its workspace alone."""
    st.device()
    ws = torch.full((cbq.kv_attention_workspace(st.cache, st.T, len(st.lens), st.n_q),), 255, dtype=torch.uint8, device=DEV)
    got = cbq.kv_attention(st.cache, st.q.to(DEV), st.d_lens, scale=st.scale, causal=causal, window=window, ws=ws, **st.at)
    at = st.mine()
    want, rel = st.outputs(at, causal, window)
    got = got.double().cpu().numpy()[at]
    bad = beyond(got, want, rel, bool(st.rotate & 2))
    norms = np.linalg.norm(want, axis=-1)
    worst = float((np.linalg.norm(got - want, axis=-1) / np.where(norms > 0, norms, 1)).max())
    assert bad == 0, f"{bad} beyond the bound; the largest relative distance of a row is {worst:.2e}, at most {rel.max():.2e}"
    return bool((ws != 255).any())


@pytest.mark.parametrize("name", CASES)
def test_cases(name):
    st, causal, window = step_of(name)
    assert _check(st, causal, window) == (name in CUT)
    many = -(-st.T // len(st.lens)) * st.n_q // st.n_kv > 128 and st.T * st.n_q > 4096
    assert many == (name in MANY_ROWS)


@pytest.mark.parametrize("rotate", [0, 1, 2, 3])
@pytest.mark.parametrize("D,lens,new,n_q,n_kv", [(64, [700, 1000, 5], [1, 5, 5], 32, 8), (128, [3000, 129], [1, 1], 16, 2),
                                                 (64, [700], [131], 32, 1), (128, [3000], [131], 32, 1)])
def test_rotations(D, lens, new, n_q, n_kv, rotate):
    _check(ExactStep(D + rotate, lens, new, n_q, n_kv, D, 32, rotate))


@pytest.mark.parametrize("new", [15, 16, 17, 33, 65])
@pytest.mark.parametrize("n_q,n_kv,length", [(8, 1, 200), (8, 2, 2500), (3, 1, 4200)])
def test_row_blocks(new, n_q, n_kv, length):
    _check(ExactStep(new + length, [length, 70], [new, new], n_q, n_kv, 64, 64))


@pytest.mark.parametrize("lens,n_kv,window", [([4400, 100] * 8, 8, 4200), ([2600, 70] * 12, 8, 2000), ([900] * 40, 8, 300)])
def test_windows_over_many_key_tiles(lens, n_kv, window):
    for offsets in (True, False):
        st = ExactStep(len(lens) + window, lens, [1] * len(lens), 2 * n_kv, n_kv, 64, 64, 0)
        device = st.device
        if not offsets:
            def without():
                device()
                st.at = dict(block_table=st.at["block_table"])
                return st
            st.device = without
        _check(st, window=window)


def test_one_prompt_among_decoding_sequences():
    _check(ExactStep(34, [2000] + [60] * 20, [500] + [1] * 20, 2, 1, 64, 64))
    _check(ExactStep(48, [1500] + [60] * 6, [1400] + [1] * 6, 4, 1, 64, 64, 0))
    _check(ExactStep(49, [2300] + [9] * 4, [700] + [2] * 4, 8, 1, 64, 64, 0))


def test_pages_given_back():
    for lens, new, n_q in (([700, 300], [3, 1], 8), ([700], [132], 32)):
        st = ExactStep(8, lens, new, n_q, 1, 64, 16, 0)
        st.table[0, 3:7], st.table[0, 30] = -1, st.n_pages + 9
        _check(st)


def test_windows_cut_among_many_sequences():
    """Two tokens a sequence, so that the window's rule for whole row blocks does not apply."""
    assert _check(ExactStep(4, [4400, 100] * 8, [2] * 16, 16, 8, 64, 64, 0), window=4200)
    assert _check(ExactStep(5, [5000, 4300, 20] * 6, [3, 1, 0] * 6, 16, 8, 64, 64), window=4200)
