"""kv_cache_read of keys or values alone."""
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


@pytest.mark.parametrize("lens,n_kv,D", [([20, 37], 2, 64), ([700, 900], 8, 128)])
def test_one_of_keys_and_values(lens, n_kv, D):
    st = Step(sum(lens), lens, lens, n_kv, D, 16).device()
    both = cbq.kv_cache_read(st.cache, st.d_lens, st.T, **st.at)
    k, none = cbq.kv_cache_read(st.cache, st.d_lens, st.T, want_v=False, **st.at)
    assert none is None and torch.equal(k, both[0])
    wide = torch.full((st.T, n_kv * D + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    none, v = cbq.kv_cache_read(st.cache, st.d_lens, st.T, v=wide[:, :n_kv * D], want_k=False, **st.at)
    assert none is None and torch.equal(v.reshape(both[1].shape), both[1]) and bool((wide[:, n_kv * D:] == 3).all())


def test_refusals():
    st = Step(1, [20], [20], 2, 64, 16).device()
    out = torch.zeros((20, 2, 64), dtype=torch.bfloat16, device=DEV)
    for bad in (dict(want_k=False, want_v=False), dict(k=out, want_k=False), dict(v=out, want_v=False)):
        with pytest.raises(ValueError):
            cbq.kv_cache_read(st.cache, st.d_lens, 20, **bad, **st.at)
    assert not bool(out.any())
