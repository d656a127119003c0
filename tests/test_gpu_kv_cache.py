"""GPU parity of cbq_kv_cache_write and cbq_kv_cache_read: codes and scales bit for bit, every place
that no token names left as it was, values read back within half a bf16 step."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from kv_steps import DEV, Step, bf16_values  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


def _host(cache):
    return [t.cpu().numpy() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)]


def _check_write(st, x64, before, rotate):
    """The cache after a write of x64 = (k, v) [T][n_kv][D] against the oracle."""
    after = _host(st.cache)
    place = st.places()
    at = np.flatnonzero(place[:, 2] >= 0)
    for i in range(2):
        q, s = oracle.kv_quantise(x64[i], bool(rotate >> i & 1))
        codes, scales = before[i].copy(), before[2 + i].copy()
        codes[place[at, 2], :, place[at, 3]] = oracle.kv_pack(q)[at]
        scales[place[at, 2], :, place[at, 3]] = s[at]
        assert np.array_equal(after[i], codes)
        assert np.array_equal(after[2 + i].view(np.uint32), scales.view(np.uint32))
    return at, place


def _check_read(st, got, kept):
    """What was read against the cache's own codes: x = scale / sqrt(D) * H c, its two fp32 roundings
    (2^-24 each) and 1 / sqrt(D) in fp32 (2^-24), then half a bf16 step (2^-8)."""
    place = st.places()
    for i in range(2):
        g = got[i].double().cpu().numpy().reshape(st.T, st.n_kv, st.D)
        for t in range(st.T):
            b, _, p, j = place[t]
            if b < 0:
                assert np.all(g[t] == kept), "a row of no sequence was written"
                continue
            if p < 0:
                assert not g[t].any()
                continue
            codes, scales = _host(st.cache)[i][p, :, j], _host(st.cache)[2 + i][p, :, j]
            x = oracle.kv_dequantise(oracle.kv_unpack(codes), scales, bool(st.rotate >> i & 1))
            assert np.all(np.abs(g[t] - x) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(x) + 1e-40)


CASES = [  # lens, new, n_kv, D, page, rotate, front, back
    ([1], [1], 1, 128, 16, 3, 0, 0),
    ([5, 17, 33], [5, 1, 2], 2, 64, 16, 3, 0, 0),
    ([40, 0, 16, 100], [3, 0, 16, 7], 4, 128, 32, 3, 2, 3),
    ([64, 65], [64, 65], 5, 128, 64, 0, 0, 1),
    ([300, 20], [30, 20], 3, 64, 128, 1, 1, 0),
    ([70], [70], 1, 128, 1024, 2, 0, 0),
]


@pytest.mark.parametrize("lens,new,n_kv,D,page,rotate,front,back", CASES)
def test_write_and_read(lens, new, n_kv, D, page, rotate, front, back):
    st = Step(sum(lens), lens, new, n_kv, D, page, rotate, front=front, back=back).device()
    (k, k64), (v, v64) = bf16_values(st.rng, (st.T, n_kv, D), 2), bf16_values(st.rng, (st.T, n_kv, D), 0.1)
    before = _host(st.cache)
    cbq.kv_cache_write(st.cache, k.to(DEV), v.to(DEV), st.d_lens, **st.at)
    _check_write(st, (k64, v64), before, rotate)
    out = [torch.full((st.T, n_kv, D), 55.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    got = cbq.kv_cache_read(st.cache, st.d_lens, st.T, k=out[0], v=out[1], **st.at)
    assert got[0] is out[0] and got[1] is out[1]
    _check_read(st, got, 55.0)


@pytest.mark.parametrize("D", [64, 128])
def test_slices_of_a_fused_projection_and_no_table(D):
    n_kv, B, n = 3, 4, 5
    st = Step(7, [20, 5, 64, 33], [n] * B, n_kv, D, 16, table=False, max_pages=4).device()
    w = n_kv * D
    qkv, x = bf16_values(st.rng, (st.T, 8 + 3 * w + 8))
    qkv = qkv.to(DEV)
    before = _host(st.cache)
    cbq.kv_cache_write(st.cache, qkv[:, 8 + w:8 + 2 * w], qkv[:, 8 + 2 * w:8 + 3 * w].view(st.T, n_kv, D), st.d_lens)
    _check_write(st, [x[:, 8 + i * w:8 + (i + 1) * w].reshape(-1, n_kv, D) for i in (1, 2)], before, 3)
    wide = torch.full((st.T, 8 + 3 * w + 8), 9.0, dtype=torch.bfloat16, device=DEV)
    cbq.kv_cache_read(st.cache, st.d_lens, st.T, k=wide[:, 8:8 + w], v=wide[:, 16 + w:16 + 2 * w])
    _check_read(st, (wide[:, 8:8 + w], wide[:, 16 + w:16 + 2 * w]), 9.0)
    assert bool((wide[:, :8] == 9).all()) and bool((wide[:, 8 + w:16 + w] == 9).all()) and bool((wide[:, 16 + 2 * w:] == 9).all())


def test_one_of_keys_and_values_read_through_the_c_call():
    import ctypes
    st = Step(8, [20, 37], [20, 37], 2, 64, 16).device()
    both = cbq.kv_cache_read(st.cache, st.d_lens, st.T, **st.at)
    lib = cbq.load_library()
    c = st.cache._c_checked(st.d_lens.device)
    s = cbq._binding._kv_seqs(st.cache, st.d_lens.device, st.d_lens, st.at["block_table"], st.d_offsets)
    one = torch.zeros_like(both[0])
    for i in range(2):
        ptr = [None, None]
        ptr[i] = one.data_ptr()
        assert lib.cbq_kv_cache_read(ctypes.byref(c), ctypes.byref(s), ptr[0], 128, ptr[1], 128, st.T,
                                     torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(one, both[i])


def test_pages_that_hold_nothing_and_positions_outside():
    """Entries outside [0, n_pages), negative positions, positions past the table: not written, read as zeros."""
    st = Step(9, [50, 3, 200, -4], [50, 5, 10, 2], 2, 64, 16, max_pages=6)
    st.table[0, 1], st.table[0, 2] = -1, st.n_pages
    st.device()
    (k, k64), (v, v64) = bf16_values(st.rng, (st.T, 2, 64)), bf16_values(st.rng, (st.T, 2, 64))
    before = _host(st.cache)
    cbq.kv_cache_write(st.cache, k.to(DEV), v.to(DEV), st.d_lens, **st.at)
    at, place = _check_write(st, (k64, v64), before, 3)
    assert 0 < len(at) < st.T
    _check_read(st, cbq.kv_cache_read(st.cache, st.d_lens, st.T, **st.at), None)


def test_extreme_rows():
    """Zeros, negative zeros, subnormal and large values, values on the codes' borders, one value alone; rows that are not
    finite get a scale that is not finite and leave their neighbours alone."""
    D, n_kv = 128, 2
    rows = np.zeros((12, n_kv, D))
    rng = np.random.default_rng(3)
    rows[1, 0, 5] = 1
    rows[2] = -0.0
    rows[3] = rng.normal(size=(n_kv, D)) * 2.0 ** -130
    rows[4] = rng.normal(size=(n_kv, D)) * 1e36
    rows[5, 0] = np.tile([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5], D // 8)      # ties once not rotated
    rows[5, 1] = -rows[5, 0]
    rows[6] = 2.0 ** -133
    rows[7, 0, :] = 3.0
    rows[8:] = rng.normal(size=(4, n_kv, D))
    for rotate in (0, 3):
        st = Step(4, [12], [12], n_kv, D, 16, rotate, garbage=False).device()
        x = torch.from_numpy(rows.astype(np.float32)).to(torch.bfloat16)
        before = _host(st.cache)
        cbq.kv_cache_write(st.cache, x.to(DEV), x.flip(0).to(DEV), st.d_lens, **st.at)
        _check_write(st, (x.double().numpy(), x.flip(0).double().numpy()), before, rotate)
        y = x.clone()
        y[8, 0, 3], y[9, 1, 7] = float("nan"), float("inf")
        cbq.kv_cache_write(st.cache, y.to(DEV), x.flip(0).to(DEV), st.d_lens, **st.at)
        q, s = oracle.kv_quantise(x.double().numpy(), bool(rotate & 1))
        place = st.places()
        got_c, got_s = _host(st.cache)[0][place[:, 2], :, place[:, 3]], _host(st.cache)[2][place[:, 2], :, place[:, 3]]
        bad = np.zeros((12, n_kv), dtype=bool)
        bad[8, 0] = bad[9, 1] = True
        assert not np.isfinite(got_s[bad]).any()
        assert np.array_equal(got_s[~bad], s[~bad]) and np.array_equal(got_c[~bad], oracle.kv_pack(q)[~bad])


@pytest.mark.parametrize("lens,n_kv,D,page,rotate", [
    ([1024], 8, 128, 64, 3), ([1025], 8, 128, 64, 3),    # 8192 heads, and more: four lanes a head
    ([700, 400], 8, 64, 16, 3), ([300, 9, 800], 9, 128, 32, 0), ([9, 11], 1024, 64, 16, 3), ([6, 3], 1000, 128, 16, 2)])
def test_many_heads(lens, n_kv, D, page, rotate):
    """Each form of the kernels against the oracle; read back in one call as sequence by sequence."""
    st = Step(sum(lens) + D, lens, lens, n_kv, D, page, rotate, garbage=False).device()
    (k, k64), (v, v64) = bf16_values(st.rng, (st.T, n_kv, D), 3), bf16_values(st.rng, (st.T, n_kv, D), 0.2)
    k[0, 0, ::3] = -0.0                                   # a zero's sign stays
    k64[0, 0, ::3] = -0.0
    before = _host(st.cache)
    cbq.kv_cache_write(st.cache, k.to(DEV), v.to(DEV), st.d_lens, **st.at)
    _check_write(st, (k64, v64), before, rotate)
    whole = cbq.kv_cache_read(st.cache, st.d_lens, st.T, **st.at)
    for b, n in enumerate(lens):
        for t in range(0, n, 8000 // n_kv):               # positions t ... of sequence b
            m = min(8000 // n_kv, n - t)
            part = cbq.kv_cache_read(st.cache, torch.tensor([t + m], dtype=torch.int32, device=DEV), m, st.at["block_table"][b:b + 1])
            for i in range(2):
                assert torch.equal(whole[i][st.offsets[b] + t:st.offsets[b] + t + m], part[i])
    host = _host(st.cache)
    place = st.places()
    for i in range(2):
        x = oracle.kv_dequantise(oracle.kv_unpack(host[i][place[:, 2], :, place[:, 3]]), host[2 + i][place[:, 2], :, place[:, 3]],
                                 bool(rotate >> i & 1))
        assert np.all(np.abs(whole[i].double().cpu().numpy() - x) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(x) + 1e-40)


@pytest.mark.parametrize("D", [64, 128])
def test_many_heads_of_all_magnitudes(D):
    """Rotated rows whose values lie within or beyond 8 and 17 binades of their largest, near the ends of the exponent range, or are
    zero, neighbours in the kernel's groups of 16: codes and scales bit for bit the oracle's, which sums in fp64."""
    n_kv, T = 8, 1100
    st = Step(D, [T], [T], n_kv, D, 64, 3, garbage=False).device()
    rng = np.random.default_rng(D)
    depth = np.array([0, 1, 7, 8, 9, 10, 16, 17, 18, 25, 30])[rng.integers(0, 11, (T, n_kv, 1))]     # binades down to the least
    x = np.ldexp(1 + rng.integers(0, 128, (T, n_kv, D)) / 128, -rng.integers(0, 31, (T, n_kv, D)) % (depth + 1))
    x *= np.where(rng.random(x.shape) < 0.5, -1, 1) * (rng.random(x.shape) > 0.1)
    x[: T // 4] = np.abs(x[: T // 4])                     # sums as large as they get
    x = np.ldexp(x, np.array([0, 0, 0, 0, 100, -60, -90, -115])[rng.integers(0, 8, (T, n_kv, 1))])
    x[rng.random((T, n_kv)) < 0.05] = 0
    x[rng.random((T, n_kv)) < 0.02] = -0.0
    x[::50, 3] = np.sign(x[::50, 3]) * 1.0                # all of one magnitude
    x[1::50, 2] = np.ldexp(np.sign(x[1::50, 2]), -133)    # bf16's smallest
    y = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    x = y.double().numpy()                                # some have become subnormal or zero
    cbq.kv_cache_write(st.cache, y.to(DEV), (-y).to(DEV), st.d_lens, **st.at)
    place = st.places()
    for i, v in enumerate((x, -x)):
        q, want = oracle.kv_quantise(v, True)
        codes, scales = (_host(st.cache)[j][place[:, 2], :, place[:, 3]] for j in (i, 2 + i))
        fine = np.isfinite(want)                          # sums beyond fp32 leave a row that is not finite
        assert fine.mean() > 0.9 and not np.isfinite(scales[~fine]).any()
        assert np.array_equal(scales[fine].view(np.uint32), want[fine].view(np.uint32))
        assert np.array_equal(codes[fine], oracle.kv_pack(q)[fine])


def test_arguments_are_checked():
    cache = cbq.KVCache.empty(4, 2, 16, 64)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    lens = torch.tensor([3], dtype=torch.int32, device=DEV)
    table = torch.zeros((1, 4), dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    bad = [dict(k=x.half()), dict(k=x[:, :1]), dict(k=x[:2]), dict(k=x[:, :, :32]), dict(k=x.transpose(1, 2)), dict(k=x.cpu()),
           dict(k=x[..., None]), dict(lens=lens.long()), dict(lens=lens[None]), dict(lens=lens.cpu()), dict(block_table=table[0]),
           dict(block_table=table.long()), dict(block_table=table.expand(2, 4)), dict(offsets=offsets[:1]), dict(offsets=offsets.float()),
           dict(offsets=offsets.cpu())]
    for b in bad:
        a = dict(k=x, lens=lens, block_table=table, offsets=offsets)
        a.update(b)
        with pytest.raises((ValueError, RuntimeError)):
            cbq.kv_cache_write(cache, a["k"], x, a["lens"], a["block_table"], a["offsets"])
        with pytest.raises((ValueError, RuntimeError)):
            cbq.kv_cache_write(cache, x, a["k"], a["lens"], a["block_table"], a["offsets"] if "k" not in b else offsets[:1])
        with pytest.raises((ValueError, RuntimeError)):
            cbq.kv_cache_read(cache, a["lens"], 3, a["block_table"], a["offsets"], k=a["k"], v=x)
        if b.get("k") is None or b["k"].shape[0] != 2 and tuple(b["k"].shape[1:]) != (1, 64):
            with pytest.raises((ValueError, RuntimeError)):
                cbq.kv_attention(cache, a["k"], a["lens"], a["block_table"], a["offsets"])
    for b in (dict(window=-1), dict(window=1 << 32), dict(window=3, causal=False), dict(scale=float("nan")), dict(out=x[:2]),
              dict(out=x.float()), dict(ws=torch.empty((16,), dtype=torch.uint8, device=DEV)), dict(ws=x)):
        with pytest.raises((ValueError, RuntimeError)):
            cbq.kv_attention(cache, x, lens, table, offsets, **b)
    for i, t in enumerate((cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)):
        for other in (t[:3], t.cpu(), t.double(), t.transpose(1, 2)):
            parts = [cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales]
            parts[i] = other
            with pytest.raises((ValueError, RuntimeError)):
                cbq.kv_cache_write(cbq.KVCache(*parts), x, x, lens, table, offsets)
    assert not bool(cache.k_codes.any())


def test_codes_are_those_of_the_same_token_in_any_batch():
    n_kv, D = 4, 128
    st = Step(11, [500], [500], n_kv, D, 64).device()
    x = torch.randn((500, n_kv, D), device=DEV).to(torch.bfloat16)
    cbq.kv_cache_write(st.cache, x, x, st.d_lens, **st.at)
    whole = _host(st.cache)
    cache = cbq.KVCache.empty(st.n_pages, n_kv, 64, D)
    for n in (1, 2, 130, 499, 500):                      # token n - 1 alone, as a decode step writes it
        cbq.kv_cache_write(cache, x[n - 1:n], x[n - 1:n], torch.tensor([n], dtype=torch.int32, device=DEV),
                           st.at["block_table"])
        p, j = st.table[0, (n - 1) // 64], (n - 1) % 64
        for a, b in zip(_host(cache), whole):
            assert np.array_equal(a[p, :, j], b[p, :, j])


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes of codes: its last pages."""
    n_kv, D, page = 8, 128, 1024
    n_pages = (1 << 32) // (n_kv * page * D // 2) + 3
    cache = cbq.KVCache.empty(n_pages, n_kv, page, D)
    assert cache.k_codes.numel() > 1 << 32
    x = torch.randn((20, n_kv, D), device=DEV).to(torch.bfloat16)
    lens = torch.tensor([1030], dtype=torch.int32, device=DEV)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=DEV)
    small = cbq.KVCache.empty(2, n_kv, page, D)
    low = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    cbq.kv_cache_write(cache, x, -x, lens, table)
    cbq.kv_cache_write(small, x, -x, lens, low)
    for i, p in ((0, n_pages - 1), (1, n_pages - 2)):
        assert torch.equal(cache.k_codes[p], small.k_codes[i]) and torch.equal(cache.v_codes[p], small.v_codes[i])
        assert torch.equal(cache.k_scales[p], small.k_scales[i]) and torch.equal(cache.v_scales[p], small.v_scales[i])
    assert bool((small.k_scales != 0).any()) and not bool((cache.k_scales[:n_pages - 2] != 0).any())
    a, b = cbq.kv_cache_read(cache, lens, 20, table), cbq.kv_cache_read(small, lens, 20, low)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q = torch.randn((20, 2 * n_kv, D), device=DEV).to(torch.bfloat16)
    o = cbq.kv_attention(cache, q, lens, table, window=15)
    assert torch.equal(o, cbq.kv_attention(small, q, lens, low, window=15)) and bool((o != 0).any())


def test_no_tokens():
    cache = cbq.KVCache.empty(2, 2, 16, 64)
    x = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    z = torch.empty((0,), dtype=torch.int32, device=DEV)
    cbq.kv_cache_write(cache, x, x, z)
    cbq.kv_cache_write(cache, x, x, torch.tensor([5], dtype=torch.int32, device=DEV))
    k, v = cbq.kv_cache_read(cache, z, 0)
    assert k.shape == (0, 2, 64) and not cache.k_codes.any()
    assert cbq.kv_attention(cache, x, z).shape == (0, 2, 64)
