"""codebook_adapter_gemm against the fp64 oracle.

Tolerance, normwise per token: the projection's K exact products are summed in fp32, an
error of at most K/16 * 2^-24 of the sum of magnitudes (MFMA steps of 16 or 32 products),
and so are the adapter's K and rank products.  The bound taken is 16384 / 16 * 2^-24 = 6.1e-5
of the magnitude sums, which the oracle forms beside the value."""
import numpy as np
import pytest
import torch

import datagen
import oracle

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from gpu_util import DEV, bf16_dev, to_dev, upload_weights  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


def _f64(bits):
    return oracle.reference.bf16_bits_to_f64(bits)


def _case(T, K, N, bits, act_bits, rank, n_ad, of=None, scale=True, blocked=True, pad=0, seed=0, check_rows=None):
    rng = np.random.default_rng(seed + T + K + N)
    w = datagen.random_weights(seed + 5, 1, N, K, bits)
    xb = datagen.random_tokens(seed + 6, T, K + pad)
    ab = datagen.f32_to_bf16_bits((rng.standard_normal((n_ad, rank, K)) / np.sqrt(K)).astype(np.float32))
    bb = datagen.f32_to_bf16_bits((0.2 * rng.standard_normal((n_ad, N, rank))).astype(np.float32))
    sc = (0.5 + rng.random(n_ad)).astype(np.float32) if scale else None
    if of is None:
        of = rng.integers(-1, n_ad, T)
    of = np.asarray(of, dtype=np.int32)
    x = bf16_dev(xb)[:, :K]
    codes, scales = cbq.rotate_quantize(x, act_bits)
    W = upload_weights(w)
    if blocked:
        W = cbq.prepack_weights(W)
    out = cbq.codebook_adapter_gemm(codes, scales, act_bits, W, x, bf16_dev(ab), bf16_dev(bb), to_dev(of),
                                    None if sc is None else to_dev(sc))
    assert out.dtype == torch.float32 and out.shape == (T, N)
    rows = np.arange(T) if check_rows is None else np.asarray(check_rows)
    q = oracle.unpack_codes(codes.cpu().numpy()[rows], K, act_bits)
    s = scales.cpu().numpy()[rows]
    Wd = oracle.dequantize(oracle.unpack_indices(w.idx[0], K, bits), w.codebook[0])
    x64 = _f64(xb[rows, :K])
    want = oracle.adapter_gemm(q, s, Wd, x64, _f64(ab), _f64(bb), of[rows], sc)
    mag = oracle.adapter_gemm(np.abs(q), s, np.abs(Wd), np.abs(x64), np.abs(_f64(ab)), np.abs(_f64(bb)), of[rows], sc)
    err = np.abs(out.cpu().numpy()[rows] - want)
    assert np.all(err <= 6.1e-5 * mag), float((err / mag).max())
    return out


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 64, 100, 257])
def test_token_counts(T):
    _case(T, 256, 192, 4, 4, 16, 5)


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("act_bits", [4, 8])
@pytest.mark.parametrize("blocked", [False, True])
@pytest.mark.parametrize("T", [6, 150])
def test_bits_and_layouts(bits, act_bits, blocked, T):
    _case(T, 288, 208, bits, act_bits, 24, 4, blocked=blocked)


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 120, 128])
@pytest.mark.parametrize("T", [3, 40])
def test_ranks(rank, T):
    _case(T, 320, 160, 3, 8, rank, 3)


@pytest.mark.parametrize("K,N", [(32, 16), (96, 48), (2560, 1024), (9728, 256), (16384, 32), (160, 9728)])
@pytest.mark.parametrize("T", [4, 48])
def test_sizes(K, N, T):
    _case(T, K, N, 4, 4, 16, 6)


def test_many_tiles_of_rows_and_columns():
    """Several 256-row tiles and both tile widths of the larger path; rows sampled."""
    T = 1300
    of = np.repeat([3, -1, 0, 2, 5, 1], [301, 7, 400, 256, 300, 36])
    _case(T, 128, 9728, 4, 4, 16, 6, of=of, check_rows=[0, 31, 300, 301, 307, 308, 707, 708, 963, 1263, 1264, 1299])
    _case(T, 128, 784, 3, 8, 32, 6, of=of, check_rows=np.arange(290, 330))


@pytest.mark.parametrize("T,K,N", [(900, 64, 2576), (2100, 64, 16384), (2304, 96, 9728), (4200, 32, 4112)])
@pytest.mark.parametrize("bits", [3, 4])
def test_tile_choices(T, K, N, bits):
    """Every tile shape of the larger path, ranks beyond one staging pass, ragged columns."""
    rng = np.random.default_rng(T)
    rows = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 40)]))
    _case(T, K, N, bits, 8, 48, 5, of=np.sort(rng.integers(-1, 5, T)), check_rows=rows)
    _case(T, K, N, bits, 4, 72, 9, check_rows=rows)


@pytest.mark.parametrize("T", [7, 70])
def test_orders_and_none(T):
    _case(T, 128, 64, 4, 8, 8, 4, of=np.full(T, 2))
    _case(T, 128, 64, 4, 8, 8, 70, of=np.arange(T)[::-1])           # every token another adapter
    _case(T, 128, 64, 4, 8, 8, 4, of=np.full(T, -1))
    _case(T, 128, 64, 4, 8, 8, 4, of=np.where(np.arange(T) % 2, 4, -2 ** 31))   # ids outside the set
    _case(T, 128, 64, 4, 8, 8, 4, scale=False, pad=24)


@pytest.mark.parametrize("T,n_ad", [(33, 40), (255, 20), (257, 300), (513, 33), (900, 1000)])
def test_many_adapters_in_random_order(T, n_ad):
    """Tiles order their tokens by adapter: ragged groups, ids up to the last, tokens with none."""
    rng = np.random.default_rng(T)
    of = rng.integers(-1, n_ad, T)
    of[[0, T - 1]] = n_ad - 1, -5
    of[T // 2] = 0x7FFFFFFF
    _case(T, 96, 48, 4, 8, 24, n_ad, of=of, pad=32)
    _case(T, 160, 144, 3, 4, 8, n_ad, of=np.sort(of))


@pytest.mark.parametrize("T,N,bits", [(300, 160, 4), (300, 160, 3), (2100, 4112, 4)])
def test_a_tokens_result_does_not_depend_on_the_order(T, N, bits):
    K, n_ad, rank = 160, 24, 40
    rng = np.random.default_rng(T + bits)
    W = cbq.prepack_weights(upload_weights(datagen.random_weights(3, 1, N, K, bits)))
    x = bf16_dev(datagen.random_tokens(4, T, K))
    codes, scales = cbq.rotate_quantize(x, 8)
    la = torch.randn(n_ad, rank, K, device=DEV).to(torch.bfloat16)
    lb = torch.randn(n_ad, N, rank, device=DEV).to(torch.bfloat16)
    of = torch.sort(to_dev(rng.integers(-1, n_ad, T).astype(np.int32))).values
    sorted_out = cbq.codebook_adapter_gemm(codes, scales, 8, W, x, la, lb, of)
    p = to_dev(rng.permutation(T))
    got = cbq.codebook_adapter_gemm(codes[p].contiguous(), scales[p].contiguous(), 8, W, x[p].contiguous(), la, lb,
                                    of[p].contiguous())
    assert torch.equal(got, sorted_out[p])


@pytest.mark.parametrize("T", [5, 80])
def test_no_adapter_is_the_plain_projection(T):
    K, N = 512, 256
    w = cbq.prepack_weights(upload_weights(datagen.random_weights(3, 1, N, K, 4)))
    x = bf16_dev(datagen.random_tokens(4, T, K))
    codes, scales = cbq.rotate_quantize(x, 4)
    a = torch.full((1, 8, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    b = torch.full((1, N, 8), float("inf"), dtype=torch.bfloat16, device=DEV)
    none = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    got = cbq.codebook_adapter_gemm(codes, scales, 4, w, x, a, b, none)
    want = cbq.codebook_lut_gemm(codes, scales, 4, [w])
    mag = cbq.codebook_lut_gemm(codes, scales, 4, [w]).abs().max()
    assert torch.isfinite(got).all()
    assert (got - want).abs().max() <= 1e-5 * mag


@pytest.mark.parametrize("T", [12, 90])
def test_another_adapters_infinities_stay_with_its_tokens(T):
    K, N = 256, 128
    w = cbq.prepack_weights(upload_weights(datagen.random_weights(3, 1, N, K, 4)))
    x = bf16_dev(datagen.random_tokens(4, T, K))
    codes, scales = cbq.rotate_quantize(x, 8)
    a = torch.randn((3, 16, K), device=DEV).to(torch.bfloat16)
    b = torch.randn((3, N, 16), device=DEV).to(torch.bfloat16)
    of = torch.arange(T, device=DEV, dtype=torch.int32) % 3
    clean = cbq.codebook_adapter_gemm(codes, scales, 8, w, x, a, b, of)
    a[1, 3], b[1, 5] = float("inf"), float("nan")
    x = x.clone()
    x[1::3] = float("nan")                                  # the rows of adapter 1
    got = cbq.codebook_adapter_gemm(codes, scales, 8, w, x, a, b, of)
    keep = of != 1
    assert torch.equal(got[keep], clean[keep])
    assert not torch.isfinite(got[~keep]).any()


def test_strided_output_and_neighbours():
    T, K, N = 37, 128, 96
    w = cbq.prepack_weights(upload_weights(datagen.random_weights(3, 1, N, K, 4)))
    x = bf16_dev(datagen.random_tokens(4, T, K))
    codes, scales = cbq.rotate_quantize(x, 4)
    a = torch.randn((2, 8, K), device=DEV).to(torch.bfloat16)
    b = torch.randn((2, N, 8), device=DEV).to(torch.bfloat16)
    for t in (5, T):
        of = torch.arange(t, device=DEV, dtype=torch.int32) % 3 - 1
        want = cbq.codebook_adapter_gemm(codes[:t], scales[:t], 4, w, x[:t], a, b, of)
        big = torch.full((t + 2, N + 32), 9.0, device=DEV)
        n = cbq.adapter_workspace(t, 8)
        ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        cbq.codebook_adapter_gemm(codes[:t], scales[:t], 4, w, x[:t], a, b, of, out=big[1:t + 1, :N], ws=ws[:n])
        assert torch.equal(big[1:t + 1, :N], want)
        assert (big[0] == 9).all() and (big[-1] == 9).all() and (big[:, N:] == 9).all() and (ws[n:] == 0xA5).all()
    empty = cbq.codebook_adapter_gemm(codes[:0], scales[:0], 4, w, x[:0], a, b, of[:0])
    assert empty.shape == (0, N)


@pytest.mark.parametrize("T", [9, 60])
def test_streams_and_graph_replay(T):
    K, N = 256, 160
    w = cbq.prepack_weights(upload_weights(datagen.random_weights(3, 1, N, K, 4)))
    x = bf16_dev(datagen.random_tokens(4, T, K))
    codes, scales = cbq.rotate_quantize(x, 4)
    a = torch.randn((4, 16, K), device=DEV).to(torch.bfloat16)
    b = torch.randn((4, N, 16), device=DEV).to(torch.bfloat16)
    of = torch.arange(T, device=DEV, dtype=torch.int32) % 5 - 1
    call = lambda st=None: cbq.codebook_adapter_gemm(codes, scales, 4, w, x, a, b, of, stream=st)  # noqa: E731
    want = call()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s1, s2):
        st.wait_stream(torch.cuda.current_stream())
    p, q = call(s1), call(s2)
    torch.cuda.synchronize()
    assert torch.equal(p, want) and torch.equal(q, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = call()
    for k in range(4):
        of.copy_(torch.randint(-1, 4, (T,), device=DEV, dtype=torch.int32))
        eager = call().clone()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap, eager), k


def test_argument_checks():
    T, K, N = 3, 64, 32
    w = upload_weights(datagen.random_weights(3, 1, N, K, 4))
    x = bf16_dev(datagen.random_tokens(4, T, K))
    codes, scales = cbq.rotate_quantize(x, 4)
    a = torch.zeros((2, 8, K), dtype=torch.bfloat16, device=DEV)
    b = torch.zeros((2, N, 8), dtype=torch.bfloat16, device=DEV)
    of = torch.zeros((T,), dtype=torch.int32, device=DEV)
    f = cbq.codebook_adapter_gemm
    for bad in (lambda: f(codes, scales, 4, w, x.float(), a, b, of), lambda: f(codes, scales, 4, w, x, a.float(), b, of),
                lambda: f(codes, scales, 4, w, x, a, b[:1], of), lambda: f(codes, scales, 4, w, x, a, b, of.long()),
                lambda: f(codes, scales, 4, w, x, a, b.transpose(1, 2).contiguous().transpose(1, 2), of),
                lambda: f(codes, scales, 8, w, x, a, b, of), lambda: f(codes, scales, 4, w, x, a, b, of[:2]),
                lambda: f(codes, scales, 4, w, x, a, b, of.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(cbq.CbqError):
        f(codes, scales, 4, w, x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), of)
    with pytest.raises(cbq.CbqError) as e:
        f(codes, scales, 4, w, x, a, b, of, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == cbq.CBQ_EWORKSPACE
