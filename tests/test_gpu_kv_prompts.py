"""GPU parity of cbq_kv_attention in its form for many query rows (more than 128 a sequence and 4096 in all): prompts and their
chunks against the oracle in 64 bits, and what must not reach a result."""
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


def _many(T, n_q):
    assert T * n_q > 4096
    return n_q


@pytest.mark.parametrize("length", [140, 2600])          # whole row blocks, and cut ones
@pytest.mark.parametrize("rotate", [0, 1, 2, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_rotations_and_windows(length, rotate, D):
    st = Step(D + rotate + length, [length], [132], 1, D, 32, rotate).device()
    check_attention(st, _many(132, 32))
    check_attention(st, 32, window=50)
    check_attention(st, 32, causal=False)


@pytest.mark.parametrize("n_q,n_kv,new", [(5, 1, 821), (6, 2, 700), (33, 1, 125), (40, 8, 103), (64, 64, 129), (1024, 1, 5),
                                          (1000, 8, 5), (1024, 2, 9)])
def test_heads(n_q, n_kv, new):
    """Row blocks that end inside a token's heads, and tokens of more heads than a row block."""
    check_attention(Step(n_q + new, [new + 33], [new], n_kv, 64, 16).device(), _many(new, n_q))


@pytest.mark.parametrize("lens,new", [([140, 1, 260], [130, 1, 7]), ([0, 64, 200, 5], [0, 64, 66, 5]), ([900, 31], [100, 31]),
                                      ([63, 64, 65], [63, 64, 65])])
@pytest.mark.parametrize("page", [16, 128])
def test_ragged_steps(lens, new, page):
    check_attention(Step(sum(lens) + page, lens, new, 1, 128, page, front=1, back=2).device(), _many(sum(new), 40))
    check_attention(Step(sum(lens) + page, lens, new, 1, 64, page, back=1).device(), _many(sum(new), 40), window=70)


@pytest.mark.parametrize("spread,scale", [(0.0, None), (1e-3, None), (30.0, None), (1.0, -0.2), (1.0, 0.0), (1e30, 1e-30), (1e-30, 1e30)])
def test_spreads_and_scales(spread, scale):
    check_attention(Step(41, [150], [130], 1, 64, 16).device(), _many(130, 32), q_spread=spread, scale=scale)


def test_scales_of_the_cache_far_apart():
    st = Step(42, [200], [140], 1, 64, 16, garbage=False)
    rng = np.random.default_rng(1)
    st.scales[1] = np.ldexp(st.scales[1], rng.integers(-40, 60, st.scales[1].shape)).astype(np.float32)
    st.scales[0] = np.ldexp(st.scales[0], rng.integers(-20, 3, st.scales[0].shape)).astype(np.float32)
    check_attention(st.device(), _many(140, 32))


def test_pages_that_hold_nothing_and_lengths_past_the_table():
    st = Step(46, [200, 64, 2000], [140, 3, 20], 1, 64, 16, max_pages=13)
    st.table[0, 3], st.table[0, 7], st.table[1, :] = -1, st.n_pages + 4, -1
    _, out, _ = check_attention(st.device(), _many(163, 32))
    assert bool(out[:140].any()) and not bool(out[140:143].any())


def test_what_a_later_token_holds_reaches_no_earlier_one():
    for length in (140, 2600):
        st = Step(3, [length], [135], 1, 128, 16).device()
        q = torch.randn((st.T, _many(135, 32), 128), device=DEV).to(torch.bfloat16)
        want = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
        p, j = st.table[0, (length - 1) // 16], (length - 1) % 16
        for bad in (float("nan"), float("inf"), 3e38):
            st.cache.k_scales[p, :, j] = bad
            st.cache.v_scales[p, :, j] = bad
            got = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
            assert torch.equal(got[:-1], want[:-1])
            if bad != 3e38:
                assert not bool(torch.isfinite(got[-1].float()).all())


def test_padding_queries_that_are_not_finite():
    for length in (140, 5000):
        st = Step(length, [length, 0, 200, -3], [130] * 4, 1, 64, 16)
        st.table[2, :] = -1
        st.device()
        q = torch.randn((st.T, _many(st.T, 8), 64), device=DEV).to(torch.bfloat16)
        want = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
        assert bool(want[:130].any()) and not bool(want[130:].any())
        for bad in (float("nan"), float("inf")):
            q[130:] = bad
            assert torch.equal(cbq.kv_attention(st.cache, q, st.d_lens, **st.at), want)


def test_offsets_that_do_not_ascend():
    st = Step(47, [200, 300, 150], [100] * 3, 2, 64, 16).device()
    q = torch.randn((st.T, _many(300, 16), 64), device=DEV).to(torch.bfloat16)
    for o in ([0, 200, 100, 300], [300, 0, 0, 300], [0, 300, -7, 2 ** 31 - 1], [0, 2 ** 31 - 1, -2 ** 31, 5]):
        out = torch.full_like(q, 7.0)
        cbq.kv_attention(st.cache, q, st.d_lens, st.at["block_table"], torch.tensor(o, dtype=torch.int32, device=DEV), out=out)
        assert bool((out == 7).all())


def test_one_prompt_among_decoding_sequences():
    """Row blocks that a wave counts together, in both the whole and the cut case."""
    check_attention(Step(48, [1500] + [60] * 6, [1500] + [1] * 6, 1, 64, 64).device(), _many(1506, 4))
    check_attention(Step(49, [2300] + [9] * 4, [700] + [2] * 4, 1, 64, 64).device(), _many(708, 8))


def test_strides_streams_repetition_and_graphs():
    D, n_q = 64, 16
    for length in (300, 3000):
        st = Step(length, [length], [270], 1, D, 64).device()
        x = torch.randn((st.T, 8 + n_q * D + 16), device=DEV).to(torch.bfloat16)
        q = x[:, 8:8 + n_q * D]
        want = cbq.kv_attention(st.cache, q.contiguous().view(st.T, _many(st.T, n_q), D), st.d_lens, **st.at)
        wide = torch.full((st.T, 8 + n_q * D + 8), 5.0, dtype=torch.bfloat16, device=DEV)
        ws = torch.full((cbq.kv_attention_workspace(st.cache, st.T, 1, n_q),), 255, dtype=torch.uint8, device=DEV)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        cbq.kv_attention(st.cache, q, st.d_lens, out=wide[:, 8:8 + n_q * D], ws=ws, stream=s, **st.at)
        torch.cuda.synchronize()
        assert torch.equal(wide[:, 8:8 + n_q * D], want.view(st.T, -1))
        assert bool((wide[:, :8] == 5).all()) and bool((wide[:, 8 + n_q * D:] == 5).all())
        out = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cbq.kv_attention(st.cache, q, st.d_lens, out=out.view(st.T, -1), ws=ws, **st.at)
        for n in (length, length - 1, 100, length):       # lengths change between replays
            st.d_lens.fill_(n)
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, cbq.kv_attention(st.cache, q, st.d_lens, **st.at).view(out.shape))
        assert torch.equal(out, want)


def test_equal_prompts_without_offsets_or_a_table():
    st = Step(50, [200, 150, 70], [70] * 3, 1, 64, 64, table=False, max_pages=4).device()
    st.at = {}
    check_attention(st, _many(210, 32))
    st = Step(51, [2500, 1900], [66] * 2, 2, 128, 64).device()
    st.at = dict(block_table=st.at["block_table"])
    check_attention(st, _many(132, 32), window=900)


def test_a_query_that_is_not_finite_stays_alone():
    """Rows of the same wave included."""
    for length in (200, 2600):
        st = Step(length + 7, [length, 60], [131, 10], 2, 64, 16).device()
        q = torch.randn((st.T, _many(141, 32), 64), device=DEV).to(torch.bfloat16)
        want = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
        for bad in (float("nan"), float("inf"), 3e38):
            q2 = q.clone()
            q2[17, 5, 3] = bad
            got = cbq.kv_attention(st.cache, q2, st.d_lens, **st.at)
            keep = torch.ones(got.shape[:2], dtype=torch.bool, device=DEV)
            keep[17, 5] = False
            assert torch.equal(got[keep], want[keep])
            if bad != 3e38:
                assert not bool(torch.isfinite(got[17, 5].float()).all())
