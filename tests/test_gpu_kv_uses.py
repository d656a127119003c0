"""Uses of the key/value cache's calls that the formulas allow and that sit at the kernels' limits: shared pages, many sequences of many
rows, rows further apart than 32 bits, more row blocks than are cut, reading back in a graph."""
import numpy as np
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


def _within(st, got, causal=True, window=0):
    want, rel = st.outputs(st.mine(), causal, window)
    return beyond(got.double().cpu().numpy()[st.mine()], want, rel, bool(st.rotate & 2)) == 0


@pytest.mark.parametrize("lens,n_q", [([40 + b % 30 for b in range(70)], 8), ([2000 - 7 * b for b in range(70)], 4)])
def test_more_than_64_sequences_of_many_rows(lens, n_q):
    """128 rows a block, whole and cut, where a lane counts more than one sequence."""
    st = ExactStep(n_q, lens, [35] * 70, n_q, 1, 64, 64, 0).device()
    assert 35 * n_q > 128 and st.T * n_q > 4096
    ws = torch.full((cbq.kv_attention_workspace(st.cache, st.T, 70, n_q),), 255, dtype=torch.uint8, device=DEV)
    for offsets in (st.d_offsets, None):
        got = cbq.kv_attention(st.cache, st.q.to(DEV), st.d_lens, st.at["block_table"], offsets, scale=st.scale, ws=ws)
        assert _within(st, got)
    assert bool((ws != 255).any()) == (max(lens) == 2000)


def test_sequences_that_share_pages():
    """Three sequences with one prefix: the pages stand three times in the table, for attention and for reading back."""
    for new, n_q in ((2, 8), (70, 32)):
        st = ExactStep(new, [300, 300, 300], [new] * 3, n_q, 1, 64, 16, 0)
        st.table[1, :12] = st.table[2, :12] = st.table[0, :12]
        st.device()
        assert _within(st, cbq.kv_attention(st.cache, st.q.to(DEV), st.d_lens, scale=st.scale, **st.at))
    lens = torch.tensor([192] * 3, dtype=torch.int32, device=DEV)
    k, v = cbq.kv_cache_read(st.cache, lens, 3 * 192, st.at["block_table"])
    for x in (k, v):
        x = x.view(3, 192, 1, 64)
        same = torch.equal(x[0], x[1]) and torch.equal(x[0], x[2]) and bool(x.any())
        assert same


def test_rows_further_apart_than_32_bits():
    """Queries, results, keys and values whose rows lie 2^30 + 8 elements apart."""
    n, T, D, n_kv, n_q = (1 << 30) + 8, 4, 64, 2, 4
    big = torch.zeros((T - 1) * n + 1024, dtype=torch.bfloat16, device=DEV)
    rows = lambda w: big.as_strided((T, w), (n, 1))  # noqa: E731
    st = Step(3, [60], [T], n_kv, D, 16, garbage=False).device()
    x = torch.randn((T, n_kv * D), device=DEV).to(torch.bfloat16)
    other = cbq.KVCache(*(t.clone() for t in (st.cache.k_codes, st.cache.v_codes, st.cache.k_scales, st.cache.v_scales)))
    rows(n_kv * D).copy_(x)
    cbq.kv_cache_write(st.cache, rows(n_kv * D), rows(n_kv * D), st.d_lens, **st.at)
    cbq.kv_cache_write(other, x, x, st.d_lens, **st.at)
    assert torch.equal(st.cache.k_codes, other.k_codes) and torch.equal(st.cache.v_scales, other.v_scales)
    want = cbq.kv_cache_read(other, st.d_lens, T, want_v=False, **st.at)[0].view(T, -1)
    cbq.kv_cache_read(st.cache, st.d_lens, T, k=rows(n_kv * D), want_v=False, **st.at)
    assert torch.equal(rows(n_kv * D), want)
    q = torch.randn((T, n_q * D), device=DEV).to(torch.bfloat16)
    rows(n_q * D).copy_(q)
    want = cbq.kv_attention(st.cache, q, st.d_lens, **st.at)
    assert torch.equal(cbq.kv_attention(st.cache, rows(n_q * D), st.d_lens, **st.at), want)
    cbq.kv_attention(st.cache, q, st.d_lens, out=rows(n_q * D), **st.at)
    assert torch.equal(rows(n_q * D), want)


def test_more_row_blocks_than_are_cut():
    """2^24 of them: 65536 sequences of one token and 256 heads, which share a few pages."""
    B, n, D = 65536, 256, 64
    st = ExactStep(5, [9, 40, 64, 1], [1] * 4, n, n, D, 16, 0).device()
    pick = torch.arange(B, device=DEV) * 7 // 3 % 4
    q = st.q.to(DEV)[pick]
    lens, table = st.d_lens[pick].contiguous(), st.at["block_table"][pick].contiguous()
    ws = torch.full((cbq.kv_attention_workspace(st.cache, B, B, n),), 255, dtype=torch.uint8, device=DEV)
    got = cbq.kv_attention(st.cache, q, lens, table, scale=st.scale, ws=ws)
    one = cbq.kv_attention(st.cache, st.q.to(DEV), st.d_lens, scale=st.scale, **st.at)
    assert _within(st, one)
    same = torch.equal(got, one[pick])
    assert same and not bool((ws != 255).any())


def test_reading_back_in_a_graph():
    """Replayed with other lengths and pages, on the stream of the replay."""
    st = Step(9, [200, 30, 90], [20, 20, 20], 3, 64, 16).device()
    k, v = (torch.zeros((60, 3, 64), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    table = st.at["block_table"]
    cbq.kv_cache_read(st.cache, st.d_lens, 60, table, k=k, v=v)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cbq.kv_cache_read(st.cache, st.d_lens, 60, table, k=k, v=v)
    for lens in ([200, 30, 90], [25, 20, 21], [3, 0, 90], [200, 30, 90]):
        st.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        table.copy_(table.roll(1, 0))
        k.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        want = cbq.kv_cache_read(st.cache, st.d_lens, 60, table)
        # places that hold no number come back as the same bits
        assert torch.equal(k.view(torch.int16), want[0].view(torch.int16)) and torch.equal(v.view(torch.int16), want[1].view(torch.int16))


def test_a_step_on_a_stream_of_its_own():
    """Write, read and attention on another stream than the tensors', twice at once on two caches."""
    steps = [Step(20 + i, [300, 45], [5, 2], 2, 128, 16).device() for i in range(2)]
    xs = [torch.randn((7, 2, 128), device=DEV).to(torch.bfloat16) for _ in steps]
    qs = [torch.randn((7, 8, 128), device=DEV).to(torch.bfloat16) for _ in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    def step(s, x, q, stream):
        cbq.kv_cache_write(s.cache, x, -x, s.d_lens, stream=stream, **s.at)
        k, v = cbq.kv_cache_read(s.cache, s.d_lens, 7, stream=stream, **s.at)
        return k, v, cbq.kv_attention(s.cache, q, s.d_lens, stream=stream, **s.at)
    want = [step(s, x, q, None) for s, x, q in zip(steps, xs, qs)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [step(s, x, q, y) for s, x, q, y in zip(steps, xs, qs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("times,new,n_q,n_kv,causal", [(1 << 18, 1, 4, 1, True), (1 << 12, 5, 8, 2, False), (1 << 10, 131, 32, 1, False)])
def test_very_long_sequences(times, new, n_q, n_kv, causal):
    """The same 4096 positions `times` over, 2^30 in all at the most, by a table that repeats their pages: the result of attending
    them once.  A sum's terms lie in 256 workgroups of 8 waves of 4 lanes at least (of 4 waves, 2 workgroups a row block, with
    many rows), and each chain of parts is joined in order."""
    page, L, D = 1024, 4096, 64
    st = ExactStep(times, [L], [new], n_q, n_kv, D, page, 0).device()
    want, rel = st.outputs(st.mine(), causal=False)
    table = st.at["block_table"].repeat(1, times)
    lens = torch.tensor([L * times], dtype=torch.int32, device=DEV)
    q = st.q.to(DEV)
    got = cbq.kv_attention(st.cache, q, lens, table, scale=st.scale, causal=causal)
    chain = L * times / (8192 if new < 100 else 2 * 16) + 1024
    assert beyond(got.double().cpu().numpy(), want, rel + chain * 2.0 ** -24, False) == 0
    if causal:                                                # windows at the far end
        got = cbq.kv_attention(st.cache, q, lens, table, scale=st.scale, window=L)
        assert beyond(got.double().cpu().numpy(), want, rel, False) == 0
