"""The attention half of a decoder block as it is used: norm, fused projection, cache, attention, output
projection, residual; a prompt and then single tokens, against the oracle fed the same inputs at each call."""
import numpy as np
import pytest
import torch

import datagen
import oracle

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from gpu_util import DEV, upload_weights  # noqa: E402
from kv_steps import Step, attention_and_bound  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


def test_prompt_then_tokens():
    H, n_q, n_kv, D, page, act = 256, 4, 2, 64, 16, 8
    qw, kw = n_q * D, n_kv * D
    w_qkv = cbq.prepack_weights(upload_weights(datagen.random_weights(21, 1, qw + 2 * kw, H, 4)))
    w_out = cbq.prepack_weights(upload_weights(datagen.random_weights(22, 1, H, qw, 4)))
    norm_w = torch.ones(H, device=DEV)
    lens = [37, 5]
    st = Step(1, [n + 8 for n in lens], [1, 1], n_kv, D, page).device()
    ref = {(b, i): [] for b in range(2) for i in range(2)}      # the tokens' keys and values as the oracle holds them
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)

    def step(new):
        nonlocal lens
        T = sum(new)
        offs = [0, new[0], T]
        d_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        at = dict(block_table=st.at["block_table"], offsets=torch.tensor(offs, dtype=torch.int32, device=DEV))
        x = torch.randn((T, H), generator=gen, device=DEV).to(torch.bfloat16)
        _, codes, scales = cbq.norm_rotate_quantize(x, norm_w, 1e-6, act, want_normed=False)
        qkv = cbq.codebook_lut_gemm(codes, scales, act, [w_qkv]).to(torch.bfloat16)
        cbq.kv_cache_write(st.cache, qkv[:, qw:qw + kw], qkv[:, qw + kw:], d_lens, **at)
        o = cbq.kv_attention(st.cache, qkv[:, :qw], d_lens, **at)
        codes, scales = cbq.rotate_quantize(o, act)
        y = cbq.combine_norm_residual(cbq.codebook_lut_gemm(codes, scales, act, [w_out]), x)
        assert y.shape == x.shape and bool(torch.isfinite(y.float()).all())
        z = qkv.double().cpu().numpy()
        got = o.double().cpu().numpy().reshape(T, n_q, D)
        for b in range(2):
            for i in range(2):
                part = z[offs[b]:offs[b + 1], qw + i * kw:qw + (i + 1) * kw].reshape(-1, n_kv, D)
                ref[b, i].append(oracle.kv_dequantise(*oracle.kv_quantise(part, True), True))
            k, v = (np.concatenate(ref[b, i]) for i in range(2))
            assert len(k) == lens[b]
            q = z[offs[b]:offs[b + 1], :qw].reshape(-1, n_q, D)
            want, tol = attention_and_bound(k, v, np.ones(len(k), dtype=bool), q, np.arange(lens[b] - new[b], lens[b]), lens[b],
                                            D ** -0.5, True, 0)
            assert np.all(np.abs(got[offs[b]:offs[b + 1]] - want) <= tol), f"attention of sequence {b}"

    step(lens)
    for _ in range(4):
        lens = [n + 1 for n in lens]
        step([1, 1])
    lens = [lens[0] + 3, lens[1] + 1]
    step([3, 1])
