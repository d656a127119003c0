"""norm_rotate_quantize and combine_norm_residual against the fp64 oracle.

bf16 outputs: the kernel evaluates in fp64 (a few units of 2^-53 per operation, at most
16384 summands) what the oracle evaluates in fp64, then rounds the same two times, so an
output is one of the values that the oracle's result times 1 -+ 2^-38 rounds to (16384 sums
of positive squares err by at most 2^14 * 2^-53, and their root and the products by a few
units more).  The combined sums cancel, so there the bound is absolute in the row's largest
term.  Codes and scales are bit-exact against the oracle on the kernel's own bf16 rows."""
import numpy as np
import pytest
import torch

import datagen
import oracle

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from gpu_util import DEV, bf16_dev, bf16_to_bits, to_dev  # noqa: E402

REL = 2.0 ** -38


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


def _f64(bits):
    return oracle.reference.bf16_bits_to_f64(bits)


def _check_normed(got_bits, v64, w, eps):
    lo, hi = oracle.bf16_candidates(oracle.rms_norm(v64, w, eps), REL)
    assert np.all((got_bits == lo) | (got_bits == hi))


def _check_codes(normed_bits, codes, scales, had_block, act_bits):
    ref = oracle.rotate_quantize(normed_bits, had_block, act_bits)
    ok = ref["ok"].all(axis=1)             # tokens inside the transform's exactness bound
    assert ok.mean() > 0.5
    assert np.array_equal(codes.cpu().numpy()[ok], ref["codes"][ok])
    assert np.array_equal(scales.cpu().numpy()[ok], ref["scale"][ok])


def _weight(seed, K):
    return (1 + 0.25 * np.random.default_rng(seed).standard_normal(K)).astype(np.float32)


def _norm_case(T, K, act_bits, had_block=0, pad=0):
    xb = datagen.random_tokens(1000 + K + T, T, K + pad)
    if T > 2:
        xb[1] = 0                                          # a row of zeros
    w = _weight(K, K)
    x = bf16_dev(xb)[:, :K]
    normed, codes, scales = cbq.norm_rotate_quantize(x, to_dev(w), 1e-5, act_bits, had_block)
    nb = bf16_to_bits(normed)
    _check_normed(nb, _f64(xb[:, :K]), w, 1e-5)
    if T > 2:
        # n = 0 * w: a zero with the sign of w
        assert not (nb[1] & 0x7FFF).any() and not codes[1].any() and scales[1].item() == 0
    _check_codes(nb, codes, scales, had_block, act_bits)


@pytest.mark.parametrize("K", [32, 64, 96, 512, 768, 1056, 1408, 2048, 2080, 2560, 4096, 4128, 8192, 8224, 14336, 16384])
@pytest.mark.parametrize("act_bits", [4, 8])
def test_norm_shapes(K, act_bits):
    _norm_case(3, K, act_bits)


@pytest.mark.parametrize("T", [1, 2, 17, 1030])
def test_norm_token_counts(T):
    _norm_case(T, 768, 8)


@pytest.mark.parametrize("K,had_block", [(1024, 1), (1024, 2), (1024, 8), (1024, 16), (2048, 32), (2048, 512),
                                         (16384, 1), (16384, 8), (16384, 4096), (4096, 1024)])
def test_norm_blocks_and_row_stride(K, had_block):
    _norm_case(4, K, 4, had_block, pad=24)


def test_norm_parts_alone_and_in_place():
    T, K = 9, 2048
    xb = datagen.random_tokens(5, T, K)
    w = to_dev(_weight(1, K))
    full = cbq.norm_rotate_quantize(bf16_dev(xb), w, 1e-6, 4)
    n, c, s = cbq.norm_rotate_quantize(bf16_dev(xb), w, 1e-6, 0)
    assert c is None and s is None and torch.equal(n, full[0])
    n, c, s = cbq.norm_rotate_quantize(bf16_dev(xb), w, 1e-6, 4, want_normed=False)
    assert n is None and torch.equal(c, full[1]) and torch.equal(s, full[2])
    x = bf16_dev(xb)
    cbq.norm_rotate_quantize(x, w, 1e-6, 0, normed=x)
    assert torch.equal(x, full[0])


def test_norm_extreme_values():
    """Rows near the ends of bf16's range: the squares leave fp32's range, not fp64's."""
    K = 256
    rng = np.random.default_rng(3)
    xb = datagen.f32_to_bf16_bits((rng.standard_normal((3, K)) * np.array([[1e37], [1e-36], [1.0]])).astype(np.float32))
    w = _weight(2, K)
    normed, codes, scales = cbq.norm_rotate_quantize(bf16_dev(xb), to_dev(w), 1e-30, 8)
    nb = bf16_to_bits(normed)
    _check_normed(nb[[0, 2]], _f64(xb)[[0, 2]], w, 1e-30)
    _check_codes(nb[[0, 2]], codes[[0, 2]], scales[[0, 2]], 0, 8)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("K", [256, 16384])
def test_a_row_that_is_not_finite_says_so_and_stays_alone(bad, K):
    x = bf16_dev(datagen.random_tokens(8, 3, K))
    w = to_dev(_weight(1, K))
    want = cbq.norm_rotate_quantize(x, w, 1e-6, 8)
    x[1, 5] = bad
    got = cbq.norm_rotate_quantize(x, w, 1e-6, 8)
    for a, b in zip(want, got):
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    assert not torch.isfinite(got[2][1])
    rows = torch.randn((3, K), device=DEV)
    res = bf16_dev(datagen.random_tokens(9, 3, K))
    want = cbq.combine_norm_residual(rows, res, post_weight=w, next_weight=w, act_bits=8)
    rows[1, 7] = bad
    got = cbq.combine_norm_residual(rows, res, post_weight=w, next_weight=w, act_bits=8)
    for a, b in zip(want, got):
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    assert not torch.isfinite(got[0][1].float()).all() and not torch.isfinite(got[3][1])


def _block_case(T, H, topk, n_shared, bf16_rows, post, gate, nxt, act_bits=8, pad=0, in_place=False, scale=0.75):
    rng = np.random.default_rng(T * 7 + H + topk)
    n = T * topk + n_shared * T
    rows = rng.standard_normal((n, H + pad)).astype(np.float32) * np.float32(0.5)
    if bf16_rows:
        rb = datagen.f32_to_bf16_bits(rows)
        rows64, rows_t = _f64(rb), bf16_dev(rb)[:, :H]
    else:
        rows64, rows_t = rows.astype(np.float64), to_dev(rows)[:, :H]
    resb = datagen.random_tokens(T + H, T, H + pad)
    res_t = bf16_dev(resb)[:, :H]
    slots = rng.permutation(T * topk).reshape(T, topk).astype(np.int32) if topk else None
    tw = rng.random((T, topk)).astype(np.float32) if topk else None
    pw, w = (_weight(7, H) if post else None), _weight(8, H)
    gb = None if gate is None else datagen.f32_to_bf16_bits(
        rng.standard_normal((T if gate == "token" else 1, H + pad)).astype(np.float32))
    opt = lambda a: None if a is None else to_dev(a)  # noqa: E731
    got = cbq.combine_norm_residual(
        rows_t, res_t, opt(slots), opt(tw), n_shared, opt(pw), 1e-5, None if gate is None else bf16_dev(gb)[:, :H],
        scale, opt(w) if nxt else None, act_bits, out=res_t if in_place else None)
    out = got[0] if nxt else got
    want = oracle.combine_norm_residual(rows64[:, :H], _f64(resb[:, :H]), slots, tw, n_shared, pw, 1e-5,
                                        None if gate is None else _f64(gb[:, :H]), scale)
    ob = bf16_to_bits(out.contiguous())
    # the sum's terms may cancel: an error of REL times the largest of the row's terms
    big = np.abs(want).max(axis=1, keepdims=True) + 40 * 8
    f = oracle.round_f64_via_f32_to_bf16_bits
    assert np.all((ob == f(want - REL * big)) | (ob == f(want + REL * big)) | (ob == f(want)))
    if in_place:
        assert out.data_ptr() == res_t.data_ptr()
    if nxt:
        nb = bf16_to_bits(got[1])
        _check_normed(nb, _f64(ob), w, 1e-5)
        if act_bits:
            _check_codes(nb, got[2], got[3], 0, act_bits)


@pytest.mark.parametrize("topk,n_shared", [(0, 1), (1, 0), (2, 0), (6, 2), (8, 0), (8, 8), (0, 2)])
@pytest.mark.parametrize("bf16_rows", [False, True])
def test_block_row_sources(topk, n_shared, bf16_rows):
    _block_case(5, 768, topk, n_shared, bf16_rows, True, "channel", True)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("nxt", [False, True])
def test_block_options(post, gate, nxt):
    _block_case(4, 2048, 2, 1, False, post, gate, nxt, act_bits=4)


@pytest.mark.parametrize("T,H", [(1, 32), (1, 2048), (33, 1408), (3, 4096), (2, 8192), (2, 8224), (2, 14336), (700, 512)])
@pytest.mark.parametrize("bf16_rows", [False, True])
def test_block_shapes(T, H, bf16_rows):
    _block_case(T, H, 6, 2, bf16_rows, True, "token", True)


def test_block_strides_in_place_and_one_token_gate():
    _block_case(6, 1024, 2, 0, False, True, "token", True, pad=40)
    _block_case(6, 1024, 2, 0, True, False, "channel", True, pad=40, in_place=True)
    _block_case(1, 1024, 0, 1, True, True, "token", True, act_bits=0)


def test_empty_calls():
    w = to_dev(_weight(1, 64))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    n, c, s = cbq.norm_rotate_quantize(x, w)
    assert n.shape == (0, 64) and c.shape == (0, 32) and s.shape == (0,)
    o = cbq.combine_norm_residual(torch.empty((0, 64), device=DEV), x)
    assert o.shape == (0, 64)


def test_rows_behind_the_last_token_stay():
    T, K = 5, 1408
    xb = datagen.random_tokens(9, T, K)
    normed = torch.full((T + 2, K), 7.0, dtype=torch.bfloat16, device=DEV)
    codes = torch.full((T + 2, K // 2), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((T + 2,), -3.0, device=DEV)
    cbq.norm_rotate_quantize(bf16_dev(xb), to_dev(_weight(3, K)), normed=normed[:T], codes=codes[:T], scales=scales[:T])
    assert (normed[T:] == 7).all() and (codes[T:] == 0x5A).all() and (scales[T:] == -3).all()


def test_stream_and_graph_replay():
    """On another stream, and captured: every replay, with eager work between, on new inputs."""
    T, H = 12, 2048
    res = bf16_dev(datagen.random_tokens(21, T, H))
    rows = torch.randn((T, H), device=DEV)
    w, pw = to_dev(_weight(1, H)), to_dev(_weight(2, H))
    call = lambda st=None: cbq.combine_norm_residual(rows, res, post_weight=pw, next_weight=w, act_bits=4, stream=st)  # noqa: E731
    want = call()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = call(st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = call()
    for k in range(4):
        rows.normal_()
        eager = [t.clone() for t in call()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, cap)), k


def test_more_tokens_than_one_launch_takes():
    """2^21 tokens go in one launch; the tokens of the second give what a call of their own gives."""
    T, K = (1 << 21) + 3, 32
    x = torch.randn(T, K, device=DEV).to(torch.bfloat16)
    w = 1 + 0.1 * torch.randn(K, device=DEV)
    n, c, s = cbq.norm_rotate_quantize(x, w, 1e-6, 4)
    for a, b in ((0, 5), (T - 7, T)):
        n1, c1, s1 = cbq.norm_rotate_quantize(x[a:b], w, 1e-6, 4)
        assert torch.equal(n[a:b], n1) and torch.equal(c[a:b], c1) and torch.equal(s[a:b], s1)


@pytest.mark.parametrize("T,K", [(2200, 1920), (2100, 2048), (1100, 4064), (1300, 3712), (520, 8192), (300, 14336), (280, 16160)])
@pytest.mark.parametrize("act_bits", [4, 8])
def test_large_batches_match_single_tokens(T, K, act_bits):
    """The form of large batches (runs of channels, the last ones partly behind the row) against that of few tokens."""
    x = torch.randn(T, K + 32, device=DEV).to(torch.bfloat16)[:, :K]
    w = 1 + 0.1 * torch.randn(K, device=DEV)
    n, c, s = cbq.norm_rotate_quantize(x, w, 1e-6, act_bits)
    for t in (0, T // 2, T - 1):
        n1, c1, s1 = cbq.norm_rotate_quantize(x[t:t + 1], w, 1e-6, act_bits)
        assert torch.equal(n[t:t + 1], n1) and torch.equal(c[t:t + 1], c1) and torch.equal(s[t:t + 1], s1)
    cr, sr = cbq.rotate_quantize(n, act_bits)
    assert torch.equal(c, cr) and torch.equal(s, sr)


@pytest.mark.parametrize("act_bits", [4, 8])
def test_norm_extreme_values_row_by_row(act_bits):
    """Rows near the ends of bf16's range, subnormal values among them, rows of one value and a
    single value beside zeros: each row against the oracle, and each alone as in the batch."""
    K = 256
    rng = np.random.default_rng(3)
    mag = np.array([[1e37], [1e-36], [1e-38], [3e-40], [1.0]])
    v = (rng.standard_normal((5, K)) * mag).astype(np.float32)
    one = np.zeros((2, K), dtype=np.float32)
    one[0], one[1, 77] = 3.0e38, 1e-40
    xb = datagen.f32_to_bf16_bits(np.concatenate([v, one]))
    assert ((xb[2:4] & 0x7F80) == 0).any() and (xb[6] & 0x7FFF).any()    # subnormal inputs
    for eps in (1e-30, 1e-6):
        w = _weight(2, K)
        normed, codes, scales = cbq.norm_rotate_quantize(bf16_dev(xb), to_dev(w), eps, act_bits)
        nb = bf16_to_bits(normed)
        _check_normed(nb, _f64(xb), w, eps)
        ref = oracle.rotate_quantize(nb, 0, act_bits)
        assert np.array_equal(codes.cpu().numpy()[ref["ok"].all(axis=1)], ref["codes"][ref["ok"].all(axis=1)])
        assert ref["ok"].all(axis=1)[[0, 1, 4, 5]].all()
        for t in range(len(xb)):
            n1, c1, s1 = cbq.norm_rotate_quantize(bf16_dev(xb[t:t + 1]), to_dev(w), eps, act_bits)
            assert torch.equal(n1, normed[t:t + 1]) and torch.equal(c1, codes[t:t + 1]) and torch.equal(s1, scales[t:t + 1])
