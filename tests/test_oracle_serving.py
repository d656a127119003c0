"""Pins of the oracle's serving functions to something other than themselves."""
import math

import numpy as np
import pytest

import datagen
import oracle


def test_rounding_through_fp32_is_two_roundings():
    assert oracle.round_f64_via_f32_to_bf16_bits(np.array([1.0, -2.0, 0.0])).tolist() == [0x3F80, 0xC000, 0]
    # just above the midpoint of 1 and 1 + 2^-7 by 2^-30: fp32 drops it, the tie goes to even
    x = np.array([1 + 2.0 ** -8 + 2.0 ** -30])
    assert oracle.round_f64_via_f32_to_bf16_bits(x)[0] == 0x3F80
    assert oracle.round_f64_to_bf16_bits(x)[0] == 0x3F81
    lo, hi = oracle.bf16_candidates(np.array([1 + 2.0 ** -8]), 2.0 ** -20)
    assert lo[0] == 0x3F80 and hi[0] == 0x3F81


def test_rms_norm_closed_forms():
    w = np.arange(1, 5, dtype=np.float64)
    # rows of one magnitude c norm to +-1 / sqrt(1 + eps / c^2)
    v = np.array([[3.0, -3.0, 3.0, -3.0]])
    want = np.array([[1, -1, 1, -1]]) * w / math.sqrt(1 + float(np.float32(0.9)) / 9)
    assert np.allclose(oracle.rms_norm(v, w, 0.9), want, rtol=1e-15)
    assert np.array_equal(oracle.rms_norm(np.zeros((1, 4)), w, 1e-6), np.zeros((1, 4)))
    # scale invariance as eps vanishes
    x = np.random.default_rng(0).normal(size=(3, 64))
    assert np.allclose(oracle.rms_norm(8 * x, np.ones(64), 1e-30), oracle.rms_norm(x, np.ones(64), 1e-30), rtol=1e-14)


def test_combine_norm_residual_matches_a_loop():
    rng = np.random.default_rng(1)
    T, k, S, H = 3, 2, 1, 8
    rows = rng.normal(size=(T * k + S * T, H))
    slots = rng.permutation(T * k).reshape(T, k)
    w = rng.random((T, k))
    res, gate, pw = rng.normal(size=(T, H)), rng.normal(size=(1, H)), rng.normal(size=H)
    got = oracle.combine_norm_residual(rows, res, slots, w, S, pw, 0.25, gate, 0.5)
    for t in range(T):
        y = [sum(w[t, j] * rows[slots[t, j], c] for j in range(k)) + rows[T * k + t, c] for c in range(H)]
        r = 1 / math.sqrt(sum(v * v for v in y) / H + 0.25)
        for c in range(H):
            assert got[t, c] == pytest.approx(res[t, c] + 0.5 * gate[0, c] * y[c] * r * pw[c], rel=1e-13, abs=1e-13)
    # without norm and gate it is the combine added to the residual
    plain = oracle.combine_norm_residual(rows, res, slots, w, S, None, 1.0, None, 1.0)
    assert np.allclose(plain - res, oracle.combine(rows, slots, w, T, k, S), rtol=1e-13, atol=1e-13)


@pytest.mark.parametrize("renorm,S", [(True, 0), (False, 2)])
def test_moe_layer_few_matches_the_layer_oracle(renorm, S):
    """On the tokens' own codes the layer equals moe_layer up to h's rounding to bf16: g, u
    and routing are the same, and teacher-forced codes of h give the same output."""
    wl = datagen.Workload("few", 3100, "moe", 8, H=64, F=96, E=5, topk=2, n_shared=S, bits_gate_up=3, bits_down=2)
    gate, up, down = datagen.moe_weights(wl)
    x, lg = datagen.moe_tokens(wl, 4)
    base = oracle.moe_layer(x, lg, gate, up, down, 2, S, 8, renormalize=renorm)
    rq = base["rq"]
    slot = np.concatenate([base["route"]["slot_of"].ravel(), 8 + np.arange(4 * S)])   # this row -> the sorted row
    few = oracle.moe_layer_few(rq["q"].astype(np.int64), rq["scale"], lg, gate, up, down, 2, S, 8, renorm)
    g, u = base["gate"][slot], base["up"][slot]
    assert np.allclose(few["h"], g * u / (1 + np.exp(-g)), rtol=1e-12, atol=1e-15)
    qh, sh = base["rqh"]["q"].astype(np.int64)[slot], base["rqh"]["scale"][slot]
    forced = oracle.moe_layer_few(rq["q"].astype(np.int64), rq["scale"], lg, gate, up, down, 2, S, 8, renorm,
                                  codes_h=(qh, sh))
    assert np.allclose(forced["y"], base["y"], rtol=1e-6, atol=1e-7 * np.abs(base["y"]).max())
    # codes of h: absmax reaches the top level, and codes times scale lie within half a step
    Q = 127
    assert np.all(np.abs(few["qh"]).max(axis=1) == Q)
    b = oracle.block_size(96)
    H = oracle.sylvester_hadamard(b).astype(np.float64)
    uh = (few["h"].reshape(-1, b) @ H / math.sqrt(b)).reshape(few["h"].shape)
    assert np.all(np.abs(few["qh"] * few["sh"][:, None].astype(np.float64) - uh) <= 0.5001 * few["sh"][:, None])


def test_adapter_gemm_is_the_sum_of_two_products():
    rng = np.random.default_rng(2)
    T, K, N, R, A = 5, 32, 16, 8, 3
    q, sc, W = rng.integers(-7, 8, (T, K)), rng.random(T).astype(np.float32), rng.normal(size=(N, K))
    x, a, b = rng.normal(size=(T, K)), rng.normal(size=(A, R, K)), rng.normal(size=(A, N, R))
    of, s = np.array([2, -1, 0, 7, 2]), np.array([0.5, 2.0, 3.0])
    y = oracle.adapter_gemm(q, sc, W, x, a, b, of, s)
    for t in range(T):
        M = np.zeros((N, K)) if of[t] not in (0, 1, 2) else s[of[t]] * (b[of[t]] @ a[of[t]])
        assert np.allclose(y[t], sc[t].astype(np.float64) * (W @ q[t]) + M @ x[t], rtol=1e-12, atol=1e-12)
