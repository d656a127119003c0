"""moe_ffn_few on inputs whose matrix products are exact in fp32 (few_layer.py), so that what
its output may be off by is known element by element, and the codes of h that its two forms
take can be compared bit for bit."""
import numpy as np
import pytest
import torch

import datagen
import oracle

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from few_layer import bound, exact_layer  # noqa: E402
from gpu_util import to_dev, upload_weights  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


def _device(q, scales, lg, weights, act_bits, blocked=True):
    dev = [upload_weights(w) for w in weights]
    if blocked:
        dev = [cbq.prepack_weights(w) for w in dev]
    return to_dev(oracle.pack_codes(q.astype(np.int8), act_bits)), to_dev(scales), to_dev(lg), dev


def _check(T, H, F, E, topk, n_shared, bits_gu, bits_d, act_bits, renorm=True, blocked=True, y_dtype=torch.float32, seed=0):
    q, scales, lg, *weights = exact_layer(T, H, F, E, topk, n_shared, bits_gu, bits_d, act_bits, seed)
    codes, sc, L, dev = _device(q, scales, lg, weights, act_bits, blocked)
    y = cbq.moe_ffn_few(codes, sc, L, *dev, topk, n_shared, act_bits, renorm, y_dtype=y_dtype)
    want = oracle.moe_layer_few(q, scales, lg, *weights, topk, n_shared, act_bits, renorm)
    tol = bound(want, weights[2], act_bits)
    if y_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want["y"]) + tol)
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - want["y"])
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("H,F,E,topk,n_shared", [(32, 32, 8, 2, 0), (96, 64, 8, 8, 8), (2048, 768, 16, 8, 0), (64, 1408, 9, 6, 2),
                                                 (48 * 32, 160, 70, 3, 1), (64, 512, 130, 8, 0), (96, 1024, 8, 4, 1),
                                                 (128, 2048, 12, 6, 0), (128, 2048, 9, 8, 8), (64, 1536, 9, 8, 0),
                                                 (64, 2016, 20, 5, 0), (64, 800, 9, 7, 8), (64, 512, 200, 8, 8),
                                                 (64, 4096, 4, 2, 0)])
@pytest.mark.parametrize("act_bits", [4, 8])
def test_one_token(H, F, E, topk, n_shared, act_bits):
    _check(1, H, F, E, topk, n_shared, 4, 3, act_bits)
    _check(1, H, F, E, topk, n_shared, 3, 2, act_bits, renorm=False, blocked=False)
    _check(1, H, F, E, topk, n_shared, 2, 4, act_bits, y_dtype=torch.bfloat16, seed=1)


@pytest.mark.parametrize("T", [2, 7, 16, 17, 32])
@pytest.mark.parametrize("H,F,E,topk,n_shared,bits_gu,bits_d", [(256, 192, 16, 4, 1, 3, 2), (320, 1408, 5, 2, 2, 4, 4),
                                                                (64, 8224, 3, 1, 0, 2, 3), (4096, 256, 40, 8, 0, 4, 3)])
@pytest.mark.parametrize("act_bits", [4, 8])
def test_batches(T, H, F, E, topk, n_shared, bits_gu, bits_d, act_bits):
    _check(T, H, F, E, topk, n_shared, bits_gu, bits_d, act_bits)


@pytest.mark.parametrize("T,F,act_bits", [(2, 16384, 8), (17, 12288, 8), (3, 10240, 4), (1, 16384, 4)])
def test_widest_h(T, F, act_bits):
    """Rotation blocks of 2048 to 16384 channels of h, across all waves of a workgroup."""
    _check(T, 64, F, 3, 2, 1, 3, 4, act_bits)


@pytest.mark.parametrize("F", [96, 128, 256, 768, 1408, 512, 1024, 1536, 2048])
@pytest.mark.parametrize("act_bits", [4, 8])
def test_a_token_alone_has_the_codes_of_h_that_it_has_in_a_batch(F, act_bits):
    """With one expert a token and one chunk of 128 channels in each row of down, y is an exact
    sum of that chunk's codes of h, times their scale: one rounding, and equal bit for bit
    where the codes and the scale are."""
    T, H, E = 32, 64, 8
    for seed in range(2):
        q, scales, lg, gate, up, down = exact_layer(T, H, F, E, 1, 0, 4, 4, act_bits, seed)
        idx = np.random.default_rng(seed).integers(1, 16, (E, H, F))
        idx[:, np.arange(F) // 128 != (np.arange(H) % ((F + 127) // 128))[:, None]] = 0
        down.idx, down.codebook[..., 0] = datagen.pack_lsb_first(idx, 4), 0
        codes, sc, L, dev = _device(q, scales, lg, (gate, up, down), act_bits)
        run = lambda a, b: cbq.moe_ffn_few(codes[a:b], sc[a:b], L[a:b], *dev, 1, 0, act_bits, y_dtype=torch.float32)  # noqa: E731
        assert torch.equal(torch.cat([run(t, t + 1) for t in range(T)]), run(0, T))
