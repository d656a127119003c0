"""The bound that the few-token layer's GPU tests use tells wrong outputs from right ones."""
import numpy as np
import pytest

import datagen
import oracle
from few_layer import bound, exact_layer

SHAPES = [(1, 256, 768, 16, 8, 0), (1, 128, 2048, 11, 8, 3), (1, 64, 1408, 9, 6, 2), (4, 64, 4096, 6, 2, 1),
          (5, 256, 192, 16, 4, 1), (2, 128, 96, 8, 2, 0)]


def _bf16(a):
    return datagen.bf16_bits_to_f32(datagen.f32_to_bf16_bits(a.astype(np.float32))).astype(np.float64)


@pytest.mark.parametrize("act_bits", [4, 8])
@pytest.mark.parametrize("T,H,F,E,topk,n_shared", SHAPES)
def test_the_bound_rejects_mutated_layers(T, H, F, E, topk, n_shared, act_bits):
    q, scales, lg, gate, up, down = exact_layer(T, H, F, E, topk, n_shared, 3, 4, act_bits)
    layer = lambda **k: oracle.moe_layer_few(q, scales, lg, gate, up, down, topk, n_shared, act_bits, **k)  # noqa: E731
    want = layer()
    tol = bound(want, down, act_bits)
    y = want["y"]
    assert np.all(tol > 0) and np.median(tol / np.abs(y)) < 2e-2
    # an fp32 h passes
    quant = lambda h: oracle.reference.quantize(  # noqa: E731
        oracle.reference.rotate_fp64(h, oracle.block_size(F)).astype(np.float32), oracle.block_size(F), act_bits)
    qh, sh = quant(want["h"].astype(np.float32).astype(np.float64))
    assert np.all(np.abs(layer(codes_h=(qh.astype(np.int64), sh))["y"] - y) <= tol)
    # every token scaled by 0.3 %, and one token alone
    assert np.any(np.abs(1.003 * y - y) > tol, axis=1).all()
    # h rounded to bf16, as long as that moves a code
    qh, sh = quant(_bf16(want["h"]))
    assert np.any(np.abs(layer(codes_h=(qh.astype(np.int64), sh))["y"] - y) > tol)
    # one code of one row off by one step, away from a border (8-bit steps are as small as
    # those that codes next to a border are granted)
    if act_bits == 4:
        off = want["qh"].copy()
        c = int(np.argmax(np.abs(oracle.reference.rotate_fp64(want["h"][:1], oracle.block_size(F)))))
        off[0, c] -= np.sign(off[0, c])             # the largest value sits on its code
        assert np.any(np.abs(layer(codes_h=(off, want["sh"]))["y"] - y) > tol)
    # a hundredth of the weight moved to another choice
    w = want["route"]["weights64"]
    if topk > 1:
        z = y + 1e-2 * (want["out"][0] - want["out"][1])
        assert w.shape == (T, topk) and np.any(np.abs(z - y)[want["token"][0]] > tol[want["token"][0]])


@pytest.mark.parametrize("act_bits", [4, 8])
def test_products_are_exact_in_fp32(act_bits):
    q, scales, lg, gate, up, down = exact_layer(3, 4096, 2048, 4, 2, 1, 4, 4, act_bits)
    want = oracle.moe_layer_few(q, scales, lg, gate, up, down, 2, 1, act_bits)
    assert np.all(np.log2(scales) % 1 == 0)
    assert np.abs(q).sum(axis=1).max() * 4 < 2 ** 24 and np.abs(want["qh"]).sum(axis=1).max() * 4 < 2 ** 24
    assert 0.1 < np.abs(want["h"]).mean() < 10
