"""GPU parity of cbq_kv_attention against the oracle in fp64, element by element, with the bound that
its arithmetic gives (kv_steps.Step.attention); caches hold garbage wherever no sequence does."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from kv_steps import DEV, Step, bf16_values, check_attention  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 500, 1000])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_one_token_of_one_sequence(length, D, page):
    check_attention(Step(length, [length], [1], 2, D, page).device(), 8)


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (4, 4), (6, 2), (12, 1), (16, 1), (17, 1), (32, 1), (33, 1), (48, 1), (71, 1),
                                      (40, 8), (5, 5)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_layouts(n_q, n_kv, D):
    check_attention(Step(n_q, [70, 33, 200], [1, 1, 1], n_kv, D, 32).device(), n_q)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
def test_pages(page):
    check_attention(Step(page, [page - 1, page, page + 1, 3 * page + 7 if page < 512 else 5], [1, 2, 3, 4], 2, 64, page).device(), 4)


@pytest.mark.parametrize("rotate", [0, 1, 2, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_rotation_flags(rotate, D):
    check_attention(Step(rotate, [130, 40], [1, 40], 2, D, 16, rotate).device(), 8)


LENS = [0, 1, 5, 64, 65, 130, 300, 17]


@pytest.mark.parametrize("new", [[0, 1, 1, 1, 1, 1, 1, 1], [0, 1, 2, 3, 4, 5, 6, 7], [0, 1, 5, 64, 65, 130, 300, 17],
                                 [0, 0, 1, 0, 40, 0, 100, 0]])
@pytest.mark.parametrize("n_q,n_kv,D", [(8, 2, 128), (3, 3, 64), (16, 1, 64)])
def test_ragged_steps(new, n_q, n_kv, D):
    check_attention(Step(len(new) + sum(new), LENS, new, n_kv, D, 16, front=2, back=3).device(), n_q)


@pytest.mark.parametrize("window", [1, 2, 16, 33, 64, 100, 1000])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_windows(window, new):
    check_attention(Step(window + new, [90, 200, 333], [new] * 3, 2, 64, 32).device(), 8, window=window)


@pytest.mark.parametrize("new", [1, 7, 100])
def test_all_positions_attended(new):
    check_attention(Step(new, [100, 250, 111], [new] * 3, 2, 128, 16).device(), 4, causal=False)


def test_rows_that_attend_nothing():
    """Empty sequences, tokens before the start, pages given back: zeros."""
    st = Step(5, [0, 3, -2, 40, 64, 10], [2, 5, 1, 3, 30, 1], 2, 64, 16)
    st.table[3, :] = -1
    st.table[4, 1] = st.n_pages + 5
    st.table[4, 2] = -1
    _, out, _ = check_attention(st.device(), 4)
    o = out.cpu()
    assert not o[0:2].any() and not o[2:4].any() and bool(o[4:7].any()) and not o[7].any() and not o[8:11].any()


def test_lengths_past_the_table():
    """lens beyond max_pages * page: the positions past the table hold nothing."""
    check_attention(Step(6, [100, 90, 2000], [4, 1, 20], 2, 128, 16, max_pages=5).device(), 4)


@pytest.mark.parametrize("spread,scale", [(0.0, None), (1e-3, None), (30.0, None), (1.0, -0.2), (1.0, 0.0), (1e30, 1e-30), (1e-30, 1e30)])
def test_spreads_and_scales(spread, scale):
    """From equal weights to one key alone; negative and no scale; queries far from fp16's range."""
    check_attention(Step(9, [150, 70], [2, 60], 2, 64, 16).device(), 4, q_spread=spread, scale=scale)


def test_scales_of_the_cache_far_apart():
    """Value scales over 2^-40 ... 2^60 and zeros, key scales over many binades: a weight is relative to its row's largest."""
    st = Step(10, [120, 64, 33], [1, 9, 33], 2, 64, 16, garbage=False)
    rng = np.random.default_rng(0)
    st.scales[1] = np.ldexp(st.scales[1], rng.integers(-40, 60, st.scales[1].shape)).astype(np.float32)
    st.scales[0] = np.ldexp(st.scales[0], rng.integers(-20, 3, st.scales[0].shape)).astype(np.float32)
    zero = rng.random(st.scales[1].shape) < 0.2
    st.scales[1][zero] = 0
    st.codes[1][zero] = 0
    check_attention(st.device(), 4)


def test_a_value_row_of_zeros_takes_its_weight():
    """Key 0 has almost all the weight and a value of zeros: the others' share stays what it is."""
    for length in (2, 70):
        st = Step(length, [length], [1], 1, 64, 16, rotate=0, garbage=False)
        p = st.table[0]
        st.codes[1][p[0], 0, 0], st.scales[1][p[0], 0, 0] = 0, 0
        st.codes[0][p[0], 0, 0], st.scales[0][p[0], 0, 0] = 0x55, 1.0
        st.device()
        q = torch.full((1, 2, 64), 0.1, dtype=torch.bfloat16, device=DEV)
        want, tol, _ = st.attention(q.double().cpu().numpy(), 0.25)
        got = cbq.kv_attention(st.cache, q, st.d_lens, scale=0.25, **st.at).double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol) and np.all(np.abs(want) < 1) and want.any()


def test_what_a_later_token_holds_reaches_no_earlier_one():
    """The last new token's scales are NaN or infinite: every earlier token's result is bit for bit what it was."""
    for lens, new in (([130], [40]), ([20], [20]), ([300], [3])):
        st = Step(3, lens, new, 2, 128, 16).device()
        q = torch.randn((st.T, 8, 128), device=DEV).to(torch.bfloat16)
        want = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
        p, j = st.table[0, (lens[0] - 1) // 16], (lens[0] - 1) % 16
        for bad in (float("nan"), float("inf"), 3e38):
            st.cache.k_scales[p, :, j] = bad
            st.cache.v_scales[p, :, j] = bad
            got = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
            assert torch.equal(got[:-1], want[:-1])
            if bad != 3e38:
                assert not bool(torch.isfinite(got[-1].float()).all())


def test_a_sequence_that_is_not_finite_stays_alone():
    st = Step(4, [100, 60, 200], [1, 5, 40], 2, 64, 16).device()
    q = torch.randn((st.T, 4, 64), device=DEV).to(torch.bfloat16)
    want = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
    st.cache.k_scales[int(st.table[1, 0]), 0, 3] = float("nan")
    q2 = q.clone()
    q2[0, 0, 0] = float("nan")
    got = cbq.kv_attention(st.cache, q2, st.d_lens, **st.at)
    assert torch.equal(got[6:], want[6:]) and torch.equal(got[0, 1:], want[0, 1:]) and torch.equal(got[1:6, 2:], want[1:6, 2:])
    assert bool(torch.isnan(got[1:6, :2].float()).all())


def test_strided_queries_outputs_and_tables():
    D, n_q, n_kv = 64, 6, 2
    st = Step(12, [80, 31], [3, 4], n_kv, D, 16).device()
    x, x64 = bf16_values(st.rng, (st.T, 16 + n_q * D + 24))
    x = x.to(DEV)
    wide = torch.full((st.T, 8 + n_q * D + 16), 5.0, dtype=torch.bfloat16, device=DEV)
    tab = torch.full((2, st.max_pages + 3), 10 ** 6, dtype=torch.int32, device=DEV)
    tab[:, :st.max_pages] = st.at["block_table"]
    want, tol, _ = st.attention(x64[:, 16:16 + n_q * D].reshape(st.T, n_q, D), D ** -0.5)
    o = wide[:, 8:8 + n_q * D]
    cbq.kv_attention(st.cache, x[:, 16:16 + n_q * D], st.d_lens, tab[:, :st.max_pages], st.d_offsets, out=o)
    assert np.all(np.abs(o.double().cpu().numpy().reshape(want.shape) - want) <= tol)
    assert bool((wide[:, :8] == 5).all()) and bool((wide[:, 8 + n_q * D:] == 5).all())
    no = Step(13, [40, 64, 9], [2, 2, 2], n_kv, D, 16, table=False, max_pages=4).device()   # sequence b's own pages, T / B tokens each
    no.at = {}
    check_attention(no, n_q)


@pytest.mark.parametrize("n_q,n_kv,D,lens,new", [
    (8, 1, 128, [40000], [1]), (4, 2, 64, [20000, 3000, 1], [1, 1, 1]), (8, 1, 64, [9000, 12], [20, 3]),
    (2, 2, 128, [5000], [300])])
def test_long_axes_split_over_the_chip(n_q, n_kv, D, lens, new):
    check_attention(Step(sum(lens), lens, new, n_kv, D, 64).device(), n_q)


@pytest.mark.parametrize("new", [15, 16, 17, 31, 32, 33, 63, 65])
@pytest.mark.parametrize("n_q,n_kv,D,length", [(8, 1, 64, 200), (8, 2, 128, 2500), (3, 1, 64, 4200)])
def test_row_blocks(new, n_q, n_kv, D, length):
    """Around 128 query rows a sequence, where the form changes, in blocks that end inside a token's heads; whole and cut."""
    check_attention(Step(new + length, [length, 70], [new, new], n_kv, D, 64).device(), n_q)


@pytest.mark.parametrize("lens,n_kv,window", [([5000, 3000, 40], 1, 2500), ([4400, 100] * 8, 8, 4200), ([2600, 70] * 12, 8, 2000),
                                              ([900] * 40, 8, 300)])
def test_windows_over_many_key_tiles(lens, n_kv, window):
    """Whole and cut row blocks, as the host takes them by the window and their number."""
    st = Step(len(lens) + window, lens, [1] * len(lens), n_kv, 64, 64).device()
    check_attention(st, 2 * n_kv, window=window)
    st.at = dict(block_table=st.at["block_table"])        # one token a sequence: no offsets needed
    check_attention(st, 2 * n_kv, window=window)


def test_long_prompts_in_many_row_blocks():
    check_attention(Step(31, [700, 130], [700, 130], 2, 64, 32).device(), 8)          # self-attention, whole blocks
    check_attention(Step(32, [1500], [1200], 1, 64, 64).device(), 2, window=200)
    check_attention(Step(33, [6000, 40], [200, 40], 1, 128, 64).device(), 4, causal=False)


def test_one_prompt_among_decoding_sequences():
    """Few rows a sequence on average, one with many row blocks, which a wave counts together."""
    check_attention(Step(34, [3000] + [60] * 20, [1500] + [1] * 20, 1, 64, 64).device(), 1)
    lens = [50, 0, 2300] + [7] * 90 + [1200, 33]
    new = [1, 0, 300] + [1] * 90 + [120, 2]
    check_attention(Step(35, lens, new, 2, 64, 64).device(), 4)                       # more than 64 sequences


@pytest.mark.parametrize("lens,new", [([90], [70]), ([2600], [70])])         # whole row blocks, and cut ones
@pytest.mark.parametrize("rotate", [0, 1, 2, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_rotations_and_windows(lens, new, rotate, D):
    st = Step(D + rotate + lens[0], lens, new, 1, D, 32, rotate).device()
    check_attention(st, 4)
    check_attention(st, 4, window=50)
    check_attention(st, 4, causal=False)


@pytest.mark.parametrize("spread,scale", [(0.0, None), (1e-3, None), (30.0, None), (1.0, -0.2), (1.0, 0.0), (1e30, 1e-30), (1e-30, 1e30)])
def test_prompts_spreads_and_scales(spread, scale):
    check_attention(Step(41, [150], [90], 2, 64, 16).device(), 4, q_spread=spread, scale=scale)


def test_prompts_scales_of_the_cache_far_apart():
    st = Step(42, [200], [130], 1, 64, 16, garbage=False)
    rng = np.random.default_rng(1)
    st.scales[1] = np.ldexp(st.scales[1], rng.integers(-40, 60, st.scales[1].shape)).astype(np.float32)
    st.scales[0] = np.ldexp(st.scales[0], rng.integers(-20, 3, st.scales[0].shape)).astype(np.float32)
    check_attention(st.device(), 2)


@pytest.mark.parametrize("n_q,n_kv,new", [(1024, 1, 1), (1024, 1, 2), (1024, 1024, 1), (1024, 512, 3), (1000, 8, 1), (7, 7, 40), (96, 1, 2)])
def test_many_heads(n_q, n_kv, new):
    check_attention(Step(n_q + new, [40], [new], n_kv, 64, 16).device(), n_q)


def test_padding_queries_that_are_not_finite():
    """Rows that attend nothing get zeros whatever their queries hold: empty sequences, pages given back, tokens before the
    start; in both forms, with few and many key tiles."""
    for new, long in ((1, 40), (1, 5000), (100, 140), (100, 5000)):
        st = Step(new + long, [long, 0, 200, -3], [new, new, new, new], 1, 64, 16)
        st.table[2, :] = -1
        st.device()
        q = torch.randn((st.T, 4, 64), device=DEV).to(torch.bfloat16)
        want = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
        assert bool(want[:new].any()) and not bool(want[new:].any())
        for bad in (float("nan"), float("inf")):
            q[new:] = bad
            got = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
            assert torch.equal(got, want)


def test_offsets_that_do_not_ascend():
    """Nothing is written, in either form."""
    for new in (1, 100):
        st = Step(new, [200, 300, 150], [new] * 3, 2, 64, 16).device()
        q = torch.randn((st.T, 8, 64), device=DEV).to(torch.bfloat16)
        for o in ([0, 2 * new, new, 3 * new], [3 * new, 0, 0, 3 * new], [0, 3 * new, -7, 2 ** 31 - 1], [0, 2 ** 31 - 1, -2 ** 31, 5]):
            out = torch.full_like(q, 7.0)
            cbq.kv_attention(st.cache, q, st.d_lens, st.at["block_table"], torch.tensor(o, dtype=torch.int32, device=DEV), out=out)
            assert bool((out == 7).all())


def test_the_most_sequences():
    B, at = 65536, {0: 5, 1000: 70, 30000: 1, 30001: 16, 65535: 33}
    lens = [at.get(b, 0) for b in range(B)]
    check_attention(Step(43, lens, [min(n, 3) for n in lens], 1, 64, 16).device(), 2)


def test_two_graphs_that_share_a_workspace():
    """Replayed in turn, each with its own results."""
    steps = [Step(44, [2500, 80], [1, 1], 2, 64, 64).device(), Step(45, [3000], [150], 2, 64, 64).device()]
    qs = [torch.randn((s.T, 8, 64), device=DEV).to(torch.bfloat16) for s in steps]
    want = [cbq.kv_attention(s.cache, q, s.d_lens, **s.at) for s, q in zip(steps, qs)]
    n = max(cbq.kv_attention_workspace(s.cache, s.T, len(s.lens), 8) for s in steps)
    ws = torch.empty((n,), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(q) for q in qs]
    graphs = []
    for s, q, o in zip(steps, qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cbq.kv_attention(s.cache, q, s.d_lens, out=o, ws=ws, **s.at)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_a_table_for_2_to_the_30_positions():
    """Units of several key tiles: the count of a call's key tiles would pass 31 bits."""
    B, page = 150, 1024
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 3000, B).tolist()
    st = Step(36, lens, [1] * B, 2, 64, page).device()
    table = torch.full((B, (1 << 30) // page), -1, dtype=torch.int32, device=DEV)
    table[:, :st.max_pages] = st.at["block_table"]
    st.at["block_table"] = table
    check_attention(st, 4)


def test_many_sequences():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 90, 700).tolist()
    check_attention(Step(14, lens, [min(n, 1) for n in lens], 2, 64, 16).device(), 4)
    check_attention(Step(15, lens[:60], [min(n, int(m)) for n, m in zip(lens, rng.integers(0, 9, 60))], 1, 128, 16).device(), 4)


def test_the_same_call_twice_is_bit_for_bit_the_same():
    st = Step(16, [3000, 77, 900], [1, 2, 70], 2, 128, 64).device()
    q = torch.randn((st.T, 16, 128), device=DEV).to(torch.bfloat16)
    a = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
    ws = torch.full((cbq.kv_attention_workspace(st.cache, st.T, 3, 16),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        assert torch.equal(a, cbq.kv_attention(st.cache, q, st.d_lens, ws=ws, **st.at))


def test_another_stream_and_two_calls_at_once():
    st = Step(17, [2500, 80], [1, 1], 2, 128, 64).device()
    q = [torch.randn((2, 8, 128), device=DEV).to(torch.bfloat16) for _ in range(2)]
    want = [cbq.kv_attention(st.cache, x, st.d_lens, **st.at) for x in q]
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [cbq.kv_attention(st.cache, x, st.d_lens, stream=y, **st.at) for x, y in zip(q, s)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_decode_loop_captured_and_replayed():
    """Write and attention of a step in a graph, replayed while lengths and inputs change, against
    eager calls; the cache grows by a token a replay over page borders."""
    B, n_q, n_kv, D, page = 3, 8, 2, 128, 16
    lens0 = [14, 0, 130]
    st = Step(18, [n + 40 for n in lens0], [1] * B, n_kv, D, page).device()
    lens = torch.tensor(lens0, dtype=torch.int32, device=DEV)
    k, v = (torch.zeros((B, n_kv, D), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    q, out = (torch.zeros((B, n_q, D), dtype=torch.bfloat16, device=DEV) for _ in "qo")
    ws = torch.empty((cbq.kv_attention_workspace(st.cache, B, B, n_q),), dtype=torch.uint8, device=DEV)
    table = st.at["block_table"]

    def step(cache, o, w):
        cbq.kv_cache_write(cache, k, v, lens, table)
        cbq.kv_attention(cache, q, lens, table, out=o, ws=w)

    step(st.cache, out, ws)
    torch.cuda.synchronize()
    other = cbq.KVCache(*(t.clone() for t in (st.cache.k_codes, st.cache.v_codes, st.cache.k_scales, st.cache.v_scales)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(st.cache, out, ws)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)
    eager = torch.empty_like(out)
    for _ in range(40):
        lens += 1
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        step(other, eager, None)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and bool(torch.isfinite(out.float()).all())
    assert torch.equal(st.cache.k_codes, other.k_codes) and torch.equal(st.cache.v_codes, other.v_codes)
