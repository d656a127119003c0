"""codebook_adapter_gemm where its large tiles sweep many steps of K and the middle vectors come
in parts, beyond 8192 tokens, and beyond 32-bit offsets.  The helper and its tolerance are those
of test_gpu_adapters."""
import numpy as np
import pytest
import torch

import datagen
import oracle

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from gpu_util import DEV, bf16_dev, to_dev, upload_weights  # noqa: E402
from test_gpu_adapters import _case, _gpu  # noqa: E402,F401


def _parts(T, K, rank, n_ad):
    """The host's rule for the parts of K in the first launch."""
    rt = (rank + 15) // 16
    zr = -(-rt // (4 if rt >= 4 else 2 if rt >= 2 else 1))
    most = 16 if T <= 32 else 4 if T <= 1024 else 2 if T <= 8192 else 1
    ny = min(n_ad, T if T < 16 else 16 if T <= 256 else 4)
    parts = 1
    while parts * 2 <= most and parts * 8 <= (K + 63) // 64 and (T + 15) // 16 * ny * zr * parts < 1024:
        parts *= 2
    return parts


# 4-bit codebooks take tiles of 256 rows from 256 of them on, 3-bit ones tiles of 256 columns
# from 512 of 128 rows on
@pytest.mark.parametrize("T,K,N,bits,act_bits,rank,order", [
    (2000, 2560, 4112, 4, 4, 16, "requests"), (2000, 2560, 8208, 3, 8, 72, "random"), (2000, 1056, 4112, 4, 8, 72, "random"),
    (2000, 1056, 4112, 4, 4, 16, "random"), (2000, 1056, 8208, 3, 4, 16, "requests"), (2000, 1056, 8208, 2, 8, 40, "random")])
def test_large_tiles_with_parts(T, K, N, bits, act_bits, rank, order):
    n_ad = 8
    assert _parts(T, K, rank, n_ad) == 2
    assert -(-N // 128) * -(-T // 256) >= 256 if bits == 4 else -(-N // 256) * -(-T // 128) >= 512
    rng = np.random.default_rng(T + K + rank)
    of = rng.integers(-1, n_ad, T)
    if order == "requests":
        of = np.sort(of)
    rows = np.unique(np.concatenate([[0, 255, 256, 1791, 1792, T - 1], rng.integers(0, T, 30)]))
    _case(T, K, N, bits, act_bits, rank, n_ad, of=of, check_rows=rows)


@pytest.mark.parametrize("T,K,N,bits,parts", [(900, 2560, 272, 4, 4), (300, 1120, 1040, 3, 4), (8200, 576, 784, 3, 1),
                                              (8200, 576, 4112, 4, 1)])
def test_other_tiles_with_long_sweeps(T, K, N, bits, parts):
    assert _parts(T, K, 24, 6) == parts
    rng = np.random.default_rng(T)
    rows = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 30)]))
    _case(T, K, N, bits, 8, 24, 6, of=rng.integers(-1, 6, T), check_rows=rows, pad=32)


def test_more_row_tiles_than_65536():
    """8.4 million tokens of a 32 x 16 projection: 65,569 row tiles."""
    T, K, N, rank, n_ad = (1 << 23) + 4133, 32, 16, 8, 3
    w = datagen.random_weights(3, 1, N, K, 3)
    x = torch.randn(T, K, device=DEV).to(torch.bfloat16)
    codes, scales = cbq.rotate_quantize(x, 8)
    a = torch.randn((n_ad, rank, K), device=DEV).to(torch.bfloat16)
    b = torch.randn((n_ad, N, rank), device=DEV).to(torch.bfloat16)
    of = torch.randint(-1, n_ad, (T,), device=DEV, dtype=torch.int32)
    out = cbq.codebook_adapter_gemm(codes, scales, 8, cbq.prepack_weights(upload_weights(w)), x, a, b, of)
    W = to_dev(oracle.dequantize(oracle.unpack_indices(w.idx[0], K, 3), w.codebook[0]).astype(np.float64))
    for lo in (0, T // 2, (1 << 16) * 128 - 350, T - 700):
        s = slice(lo, lo + 700)
        q = codes[s].view(torch.int8).double()
        want, mag = ((f(q) @ f(W).T) * scales[s, None].double() for f in (lambda v: v, torch.abs))
        for i in range(n_ad):
            mine = (of[s] == i)[:, None]
            want = want + mine * (x[s].double() @ a[i].double().T @ b[i].double().T)
            mag = mag + mine * (x[s].double().abs() @ a[i].double().abs().T @ b[i].double().abs().T)
        assert ((out[s] - want).abs() <= 6.1e-5 * mag).all()


@pytest.mark.parametrize("T", [3, 40])
def test_adapters_beyond_32_bit_offsets(T):
    """Adapter ids whose lora_a and lora_b lie 4.6 GB in, against the same adapters renumbered."""
    K, N, rank, n_ad = 16384, 16400, 128, 1100
    w = cbq.CodebookWeights(idx=torch.randint(0, 256, (1, N, K // 2), dtype=torch.uint8, device=DEV),
                            codebook=(torch.randn((1, N, 16), device=DEV) * 0.02).half(), K=K, bits=4)
    x = torch.randn(T, K, device=DEV).to(torch.bfloat16)
    codes, scales = cbq.rotate_quantize(x, 8)
    a = torch.empty((n_ad, rank, K), dtype=torch.bfloat16, device=DEV)
    b = torch.empty((n_ad, N, rank), dtype=torch.bfloat16, device=DEV)
    used = [2, 1057, 1099]
    for i in used:
        a[i] = (torch.randn((rank, K), device=DEV) / 128).to(torch.bfloat16)
        b[i] = torch.randn((N, rank), device=DEV).to(torch.bfloat16)
    pick = torch.arange(T, device=DEV) % 3
    of = torch.tensor(used, device=DEV, dtype=torch.int32)[pick]
    got = cbq.codebook_adapter_gemm(codes, scales, 8, w, x, a, b, of)
    want = cbq.codebook_adapter_gemm(codes, scales, 8, w, x, a[used], b[used], pick.int())
    # sums of K / 16 steps in another order (parts of K follow the number of adapters)
    assert (got - want).abs().max() <= 6.1e-5 * want.abs().max()
    base = cbq.codebook_lut_gemm(codes, scales, 8, [w])
    assert (got - base).abs().max() > 0.1 * base.abs().max()


@pytest.mark.parametrize("T", [5, 40])
def test_rows_of_x_beyond_32_bit_offsets(T):
    K, N, ld = 96, 64, (1 << 31) // (T - 1) // 8 * 8 + 4096
    big = torch.empty((T, ld), dtype=torch.bfloat16, device=DEV)
    x = big[:, :K]
    x.copy_(bf16_dev(datagen.random_tokens(4, T, K)))
    codes, scales = cbq.rotate_quantize(x.contiguous(), 4)
    w = cbq.prepack_weights(upload_weights(datagen.random_weights(3, 1, N, K, 4)))
    a = torch.randn((3, 16, K), device=DEV).to(torch.bfloat16)
    b = torch.randn((3, N, 16), device=DEV).to(torch.bfloat16)
    of = to_dev((np.arange(T) % 3).astype(np.int32))
    assert torch.equal(cbq.codebook_adapter_gemm(codes, scales, 4, w, x, a, b, of),
                       cbq.codebook_adapter_gemm(codes, scales, 4, w, x.contiguous(), a, b, of))


@pytest.mark.parametrize("T,N,rank,bits,act_bits,n_ad", [(32, 64, 128, 4, 4, 5), (32, 48, 128, 3, 8, 40), (17, 16, 8, 2, 8, 3)])
def test_decode_batches_with_the_most_splits(T, N, rank, bits, act_bits, n_ad):
    """K = 16384 on a narrow projection: 16 splits of K in a workgroup, the widest middle vectors beside them."""
    _case(T, 16384, N, bits, act_bits, rank, n_ad)


@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("mag", [(1e-39, 1e30, 1.0), (1e30, 1e-39, 1.0), (1e20, 1e-20, 1e-39), (3e-39, 1.0, 1e30), (1e-30, 1e-8, 1e30)])
def test_subnormal_factors(T, mag):
    """Subnormal x, lora_a or lora_b, and middle vectors near and below fp32's smallest normal value: the
    tolerance of the other tests and, beyond a decode batch, 2^-133 of the middle vector (half a step of
    its last part's, 2^-134, and of the fp32 sum's, 2^-150, are less)."""
    K, N, rank = 256, 64, 16
    w = cbq.prepack_weights(upload_weights(datagen.random_weights(3, 1, N, K, 4)))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T)
    rnd = lambda m, *s: (torch.randn(s, generator=gen, device=DEV) * m).to(torch.bfloat16)  # noqa: E731
    x, a, b = rnd(mag[0], T, K), rnd(mag[1], 1, rank, K), rnd(mag[2], 1, N, rank)
    codes = torch.zeros((T, K), dtype=torch.uint8, device=DEV)
    out = cbq.codebook_adapter_gemm(codes, torch.zeros(T, device=DEV), 8, w, x, a, b, torch.zeros(T, dtype=torch.int32, device=DEV))
    x, a, b = x.double(), a[0].double(), b[0].double()
    tol = 6.1e-5 * (x.abs() @ a.abs().T) @ b.abs().T + 2.0 ** -133 * b.abs().sum(1) + 2.0 ** -149
    assert ((out - (x @ a.T) @ b.T).abs() <= tol).all()
