"""Arguments that the calls around a block would not use, or would misread, are refused."""
import pytest
import torch

import datagen

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from gpu_util import DEV, upload_weights  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


def test_output_tensors_that_would_stay_unwritten():
    T, K = 3, 64
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(K, device=DEV)
    codes = torch.empty((T, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, device=DEV)
    normed = torch.empty_like(x)
    for kw in (dict(codes=codes), dict(scales=scales), dict(codes=codes, scales=scales)):
        with pytest.raises(ValueError, match="act_bits"):
            cbq.norm_rotate_quantize(x, w, act_bits=0, **kw)
        with pytest.raises(ValueError, match="act_bits"):
            cbq.combine_norm_residual(x, x, next_weight=w, **kw)
    for kw in (dict(codes=codes), dict(scales=scales), dict(normed=normed), dict(normed=normed, act_bits=4, codes=codes)):
        with pytest.raises(ValueError, match="next_weight"):
            cbq.combine_norm_residual(x, x, **kw)
    n, c, s = cbq.norm_rotate_quantize(x, w, act_bits=4, normed=normed, codes=codes, scales=scales)
    assert n is normed and c is codes and s is scales
    out = cbq.combine_norm_residual(x, x, next_weight=w, act_bits=4, normed=normed, codes=codes, scales=scales)
    assert out[1] is normed and out[2] is codes and out[3] is scales
    assert cbq.combine_norm_residual(x, x, act_bits=4).shape == x.shape


def test_codebooks_of_another_16_bit_type():
    """fp16 patterns come as float16, int16 or uint16; bfloat16 values are not fp16 patterns."""
    T, K, N = 2, 64, 32
    w = upload_weights(datagen.random_weights(3, 1, N, K, 4))
    x = torch.randn((T, K), device=DEV).to(torch.bfloat16)
    codes, scales = cbq.rotate_quantize(x, 4)
    a = torch.zeros((1, 8, K), dtype=torch.bfloat16, device=DEV)
    b = torch.zeros((1, N, 8), dtype=torch.bfloat16, device=DEV)
    of = torch.zeros(T, dtype=torch.int32, device=DEV)
    run = lambda v: cbq.codebook_adapter_gemm(  # noqa: E731
        codes, scales, 4, cbq.CodebookWeights(w.idx, w.codebook.view(v), K, 4), x, a, b, of)
    want = run(torch.int16)
    assert torch.equal(run(torch.float16), want) and torch.equal(run(torch.uint16), want)
    with pytest.raises(ValueError, match="codebook"):
        run(torch.bfloat16)
    # the same tensors as a layer of one expert
    down = upload_weights(datagen.random_weights(4, 1, K, N, 4))
    bad = cbq.CodebookWeights(w.idx, w.codebook.view(torch.bfloat16), K, 4)
    with pytest.raises(ValueError, match="codebook"):
        cbq.moe_ffn_few(codes, scales, torch.zeros((T, 1), device=DEV), w, bad, down, 1)
