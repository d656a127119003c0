"""Arguments that the calls around a block would not use, or would misread, are refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from gpu_util import DEV  # noqa: E402


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
