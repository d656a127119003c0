"""The workspace of cbq_kv_attention on the host: a buffer made for the most tokens of a step serves every smaller one."""
import ctypes
import os

import pytest

cbq = pytest.importorskip("codebook_bit_quantized_amd")

P = ctypes.c_void_p(0x1000)
TOKENS = [1, 2, 17, 64, 65, 127, 128, 129, 500, 1024, 1025, 4096, 4097, 70000, 1 << 20]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cbq.LIB_PATH):
        pytest.skip("libcbq.so not built")
    return cbq.load_library()


@pytest.mark.parametrize("n_q,n_kv,D", [(32, 4, 128), (32, 8, 64), (1, 1, 128), (5, 5, 64), (1024, 2, 128)])
def test_a_buffer_for_the_most_tokens_serves_fewer_in_any_batch(lib, n_q, n_kv, D):
    cache = ctypes.byref(cbq._binding.cbq_kv_cache(0x1000, 0x1000, 0x1000, 0x1000, 8, n_kv, 16, D, 3))
    least = 0
    for T in TOKENS:
        sizes = [lib.cbq_kv_attention_workspace(cache, T, B, n_q) for B in (1, 2, 3, 64, 1000, T, 65536) if B <= 65536]
        assert min(sizes) > 0 and min(sizes) >= least, f"T = {T}: {sizes} bytes by the batch, {least} for fewer tokens"
        least = max(sizes)


def test_the_call_takes_no_more_than_the_query_says(lib):
    """A buffer of one byte for sequences whose tokens do not divide into it: the call names what it needs."""
    cache = ctypes.byref(cbq._binding.cbq_kv_cache(0x1000, 0x1000, 0x1000, 0x1000, 8, 4, 16, 128, 3))
    for T, B in ((1024, 1), (1024, 1024), (5000, 7), (1, 1), (200, 100)):
        seqs = ctypes.byref(cbq._binding.cbq_kv_seqs(0x1000, 4, 4, 0x1000, 0x1000, B))
        rc = lib.cbq_kv_attention(cache, seqs, P, 32 * 128, T, 32, 0.1, 1, 0, P, 32 * 128, P, 1, None)
        assert rc == cbq.CBQ_EWORKSPACE
        needs = int(lib.cbq_last_error().split(b"workspace of ")[1].split()[0])
        assert 1 < needs <= min(lib.cbq_kv_attention_workspace(cache, T, b, 32) for b in (1, B, T))
