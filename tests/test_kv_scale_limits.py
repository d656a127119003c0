"""The softmax scale near the ends of fp32's range."""
import ctypes
import os

import pytest
import torch

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from kv_steps import DEV, Step, check_attention  # noqa: E402

P = ctypes.c_void_p(0x1000)


def test_scales_whose_binary_logarithm_factor_overflows_are_refused():
    """The kernels take scale * log2(e) in fp32."""
    if not os.path.exists(cbq.LIB_PATH):
        pytest.skip("libcbq.so not built")
    lib = cbq.load_library()
    for rotate in (0, 3):
        cache = ctypes.byref(cbq._binding.cbq_kv_cache(0x1000, 0x1000, 0x1000, 0x1000, 8, 2, 16, 64, rotate))
        seqs = ctypes.byref(cbq._binding.cbq_kv_seqs(0x1000, 4, 4, 0x1000, 0x1000, 3))
        for scale, rc in ((2.0 ** 127, cbq.CBQ_EWORKSPACE), (-2.0 ** 127, cbq.CBQ_EWORKSPACE), (2.0 ** 127 * 1.001, cbq.CBQ_EINVAL),
                          (-3e38, cbq.CBQ_EINVAL), (0.0, cbq.CBQ_EWORKSPACE)):
            assert lib.cbq_kv_attention(cache, seqs, P, 256, 6, 4, scale, 1, 0, P, 256, None, 0, None) == rc, scale


@pytest.mark.gpu
@pytest.mark.parametrize("new,n_q", [(3, 4), (140, 32)])
@pytest.mark.parametrize("rotate", [0, 3])
def test_scales_at_the_ends(new, n_q, rotate):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for scale in (2.0 ** 127, -2.0 ** 127, 2.0 ** -126):
        spread = 1 / abs(scale) if abs(scale) > 1 else 1.0
        check_attention(Step(7, [200], [new], 1, 64, 16, rotate).device(), n_q, q_spread=spread, scale=scale)
        check_attention(Step(7, [200], [new], 1, 64, 16, rotate).device(), n_q, q_spread=0.0, scale=scale)
