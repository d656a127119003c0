"""Pins of the oracle's 4-bit key/value cache and attention: closed forms and brute force."""
import numpy as np
import pytest

import oracle


def test_e2m1_values_are_sign_exponent_mantissa():
    for n in range(16):
        e, m = (n >> 1) & 3, n & 1
        mag = 0.5 * m if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1)
        assert oracle.e2m1_decode(n) == (-mag if n & 8 else mag)
        assert oracle.e2m1_encode(np.array(oracle.e2m1_decode(n))) == n


def test_e2m1_ties_go_to_the_even_index_and_large_values_to_six():
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    want = [0, 2, 2, 4, 4, 6, 6]
    for r, w in zip(mid, want):
        assert oracle.e2m1_encode(np.array([r, -r])).tolist() == [w, w + 8]
        up, down = np.nextafter(r, 9), np.nextafter(r, 0)
        i = mid.index(r)
        assert oracle.e2m1_encode(np.array([down, up])).tolist() == [i, i + 1]
    assert oracle.e2m1_encode(np.array([6.5, 1e30, -7.0])).tolist() == [7, 7, 15]
    r = np.random.default_rng(0).normal(size=2000) * 3            # brute force: no value is nearer
    d = np.abs(oracle.e2m1_decode(oracle.e2m1_encode(r)) - np.clip(r, -6, 6))
    assert np.all(d <= np.abs(np.clip(r, -6, 6)[:, None] - oracle.E2M1_VALUES).min(1) + 1e-15)


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_round_trip(D, rotate):
    rng = np.random.default_rng(D)
    x = rng.normal(size=(3, 2, D))
    x[1, 1] = 0
    q, s = oracle.kv_quantise(x, rotate)
    assert np.array_equal(oracle.kv_unpack(oracle.kv_pack(q)), q) and s.dtype == np.float32
    assert s[1, 1] == 0 and not q[1, 1].any()
    back = oracle.kv_dequantise(q, s, rotate)
    # in the quantised space a value is off by at most one step of 2/6 at the top of the range (half of 4 .. 6)
    y = oracle.kv_dequantise(q, s, False)
    v = (x.reshape(-1, D) @ oracle.sylvester_hadamard(D) / np.sqrt(D)).reshape(x.shape) if rotate else x
    assert np.all(np.abs(y - v) <= np.abs(v).max(-1, keepdims=True) / 6 * (1 + 1e-6))
    # the rotation keeps lengths, so the error's length is the same in both spaces
    assert np.allclose(np.linalg.norm(back - x, axis=-1), np.linalg.norm(y - v, axis=-1), rtol=1e-9)
    # what is already on the grid comes back as it was
    q2, s2 = oracle.kv_quantise(back, rotate)
    full = np.abs(oracle.e2m1_decode(q)).max(-1) == 6
    assert np.allclose(oracle.kv_dequantise(q2, s2, rotate)[full], back[full], rtol=1e-6, atol=1e-7)


def test_places():
    table = np.array([[5, -1, 2], [9, 1, 0]])
    p = oracle.kv_places(7, [18, 33], [1, 4, 6], table, 16, 9)
    assert p.tolist() == [[-1, -1, -1, -1], [0, 15, 5, 15], [0, 16, -1, -1], [0, 17, -1, -1], [1, 31, 1, 15],
                          [1, 32, 0, 0], [-1, -1, -1, -1]]
    p = oracle.kv_places(4, [1, 60], None, table, 16, 9)           # before the start, and past the last page
    assert p.tolist() == [[0, -1, -1, -1], [0, 0, 5, 0], [1, 58, -1, -1], [1, 59, -1, -1]]


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    L, n_kv, n_q, D, n = 9, 2, 4, 8, 3
    k, v, q = rng.normal(size=(L, n_kv, D)), rng.normal(size=(L, n_kv, D)), rng.normal(size=(n, n_q, D))
    held, pos = np.ones(L, dtype=bool), np.arange(L - n, L)
    # equal keys: the mean of the attended values
    o, p, _ = oracle.kv_attention(np.ones_like(k), v, held, q, pos, L, 0.3, True, 0)
    for i in range(n):
        for h in range(n_q):
            assert np.allclose(o[i, h], v[:pos[i] + 1, h // 2].mean(0))
    # a window of one: the token's own value
    o, _, _ = oracle.kv_attention(k, v, held, q, pos, L, 0.3, True, 1)
    assert np.allclose(o[:, 0], v[pos, 0]) and np.allclose(o[:, 3], v[pos, 1])
    # a score far above the others: that value
    k2 = np.zeros_like(k)
    k2[4] = 1e4 * np.sign(q[0, 0])
    o, _, _ = oracle.kv_attention(k2, v, held, q[:1, :1].repeat(2, 1), pos[:1], L, 1.0, True, 0)
    assert np.allclose(o[0], v[4])
    # probabilities sum to one over what is seen; nothing held: zeros
    o, p, _ = oracle.kv_attention(k, v, held, q, pos, L - 1, 0.3, False, 0)
    assert np.allclose(p.sum(-1), 1) and np.all(p[..., L - 1] == 0)
    o, p, _ = oracle.kv_attention(k, v, ~held, q, pos, L, 0.3, True, 0)
    assert not o.any() and not p.any()
    # rotating queries and keys alike changes nothing
    R = oracle.sylvester_hadamard(D) / np.sqrt(D)
    a = oracle.kv_attention(k, v, held, q, pos, L, 0.3, True, 4)[0]
    b = oracle.kv_attention(k @ R, v @ R, held, q @ R, pos, L, 0.3, True, 4)[0] @ R
    assert np.allclose(a, b)
