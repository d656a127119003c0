"""Codes next to a border where the reciprocal of the scale is hardest to round: bit for bit the oracle's."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from kv_steps import DEV, Step  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


def _pieces(x):
    """x > 0 as a sum of positive bf16 values."""
    out = []
    while x > 0:
        e = np.floor(np.log2(x))
        p = np.floor(x / 2.0 ** (e - 7)) * 2.0 ** (e - 7)
        out.append(p)
        x -= p
    return out


def _row(D, largest, other):
    """A row of bf16 values whose transform has its largest value, `largest`, in channel 0 and `other` in channel 1."""
    x = np.zeros(D)
    for first, total in ((0, (largest + other) / 2), (1, (largest - other) / 2)):
        for i, p in enumerate(_pieces(total)):
            x[first + 2 * i] = p                           # channel 1's signs go by the index's lowest bit
    u = oracle.sylvester_hadamard(D) @ x
    assert u[0] == largest == np.abs(u).max() and u[1] == other
    return x


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [8, 2000])              # few and many lanes a head
def test_scales_whose_mantissa_is_all_ones(D, tokens):
    """largest / 6 = (2 - 2^-23) * 2^k: the code of 2^(k-1) is that of a quotient one step above 1/4."""
    largest = 12 - 2.0 ** -20
    s = np.float32(largest) / np.float32(6)
    assert s == np.float32(2 - 2.0 ** -23) and np.float32(0.5) / s == np.nextafter(np.float32(0.25), np.float32(1))
    n_kv = 8
    rows = np.array([_row(D, largest, b * 2) for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)] + [_row(D, 12.0, 0.5)])
    rows = np.concatenate([rows, -rows])
    t, h = np.meshgrid(np.arange(tokens), np.arange(n_kv), indexing="ij")
    x = rows[(t * n_kv + h) % len(rows)] * 2.0 ** ((t + h) % 9 * 12 - 48)[..., None]
    y = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    assert np.array_equal(y.double().numpy(), x)
    st = Step(D, [tokens], [tokens], n_kv, D, 64, 3, garbage=False).device()
    cbq.kv_cache_write(st.cache, y.to(DEV), (-y).to(DEV), st.d_lens, **st.at)
    place = st.places()
    for v, codes, scales in ((x, st.cache.k_codes, st.cache.k_scales), (-x, st.cache.v_codes, st.cache.v_scales)):
        q, want = oracle.kv_quantise(v, True)
        got = oracle.kv_unpack(codes.cpu().numpy()[place[:, 2], :, place[:, 3]])
        wrong = int((got != q).sum())
        assert wrong == 0, f"{wrong} codes, the first at {np.argwhere(got != q)[0]}: {got[got != q][0]}, not {q[got != q][0]}"
        assert np.array_equal(scales.cpu().numpy()[place[:, 2], :, place[:, 3]].view(np.uint32), want.view(np.uint32))
