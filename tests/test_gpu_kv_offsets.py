"""One token a sequence, with offsets that say so and without: the same call, so the same bits and the same way through the
kernels (a call whose row blocks stay whole leaves its workspace alone)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from kv_exact import ExactStep, beyond  # noqa: E402
from kv_steps import DEV, Step  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


@pytest.mark.parametrize("lens,n_q,n_kv,D,window", [
    ([4500, 70, 2000, 900] * 4, 32, 8, 64, 4096), ([4500, 100] * 16, 8, 8, 64, 4096), ([1100, 60] * 20, 8, 8, 64, 1000),
    ([3500, 700, 20, 90] * 7, 16, 4, 64, 0), ([3000] * 10, 20, 5, 64, 0), ([1500, 2000, 9], 8, 2, 128, 0), ([300] * 70, 16, 1, 128, 0),
    ([2000, 40], 64, 2, 64, 0)])
def test_one_token_a_sequence(lens, n_q, n_kv, D, window):
    B = len(lens)
    st = Step(sum(lens), lens, [1] * B, n_kv, D, 64).device()
    q = torch.randn((B, n_q, D), device=DEV).to(torch.bfloat16)
    got = []
    for offsets in (None, st.d_offsets):
        ws = torch.full((cbq.kv_attention_workspace(st.cache, B, B, n_q),), 255, dtype=torch.uint8, device=DEV)
        o = cbq.kv_attention(st.cache, q, st.d_lens, st.at["block_table"], offsets, window=window, ws=ws)
        got.append((o, bool((ws != 255).any())))
    same = torch.equal(got[0][0], got[1][0])
    assert got[0][1] == got[1][1], f"row blocks cut without offsets: {got[0][1]}, with them: {got[1][1]}"
    assert same


@pytest.mark.parametrize("lens,new", [([4500, 70, 2000, 0] * 4, [3, 1, 0, 0] * 4), ([500] * 40, [40] + [0] * 39),
                                      ([50] * 40, [0] * 39 + [40]), ([900] * 3, [1, 2, 0])])
def test_as_many_tokens_as_sequences_but_not_one_each(lens, new):
    """The host's count of row blocks still holds, with 17 query heads to a key/value head and with one."""
    for n_q in (34, 2):
        st = ExactStep(n_q, lens, new, n_q, 2, 64, 64, 0).device()
        got = cbq.kv_attention(st.cache, st.q.to(DEV), st.d_lens, scale=st.scale, **st.at)
        want, rel = st.outputs(st.mine())
        assert beyond(got.double().cpu().numpy(), want, rel, False) == 0
