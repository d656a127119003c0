"""The norms around a block on tensors of more than 2^31 elements: the last tokens give what a
call of their own gives."""
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


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_norm_beyond_32_bit_offsets():
    T, K = (1 << 31) // 16384 + 300, 16384
    x = torch.empty((T, K), dtype=torch.bfloat16, device=DEV).normal_()
    w = 1 + 0.1 * torch.randn(K, device=DEV)
    got = cbq.norm_rotate_quantize(x, w, 1e-6, 8)
    for lo in (0, 131071, T - 3):
        assert _same([t[lo:lo + 3] for t in got], cbq.norm_rotate_quantize(x[lo:lo + 3], w, 1e-6, 8))


@pytest.mark.parametrize("dtype,H,T", [(torch.bfloat16, 8192, 33000), (torch.float32, 4096, 66000)])
def test_combine_beyond_32_bit_offsets(dtype, H, T):
    topk = 8
    rows = torch.empty((T * topk, H), dtype=dtype, device=DEV).normal_()
    res = torch.empty((T, H), dtype=torch.bfloat16, device=DEV).normal_()
    slots = torch.randperm(T * topk, device=DEV).view(T, topk).int()
    tw = torch.rand((T, topk), device=DEV)
    w = 1 + 0.1 * torch.randn(H, device=DEV)
    got = cbq.combine_norm_residual(rows, res, slots, tw, post_weight=w, next_weight=w, act_bits=4)
    for lo in (0, T - 5):
        s = slots[lo:lo + 5].long()
        own = cbq.combine_norm_residual(rows[s.flatten()], res[lo:lo + 5],
                                        torch.arange(5 * topk, device=DEV, dtype=torch.int32).view(5, topk),
                                        tw[lo:lo + 5].contiguous(), post_weight=w, next_weight=w, act_bits=4)
        assert _same([t[lo:lo + 5] for t in got], own)
