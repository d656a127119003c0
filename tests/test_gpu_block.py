"""The calls around a block as a serving loop makes them, one after the other: input norm,
router, few-token MoE layer (or the single calls for a prefill), the residual with the next
norm, and a projection with adapters.  Every stage is checked on the stage before it as the
GPU gave it, and the whole decode step is captured and replayed."""
import numpy as np
import pytest
import torch

import datagen
import oracle

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from gpu_util import DEV, bf16_dev, bf16_to_bits, to_dev, upload_weights  # noqa: E402

H, F, E, TOPK, SHARED, N, R, A = 256, 192, 12, 3, 1, 160, 16, 4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


@pytest.fixture(scope="module")
def model():
    wl = datagen.Workload("block", 4900, "moe", 8, H=H, F=F, E=E, topk=TOPK, n_shared=SHARED, bits_gate_up=3, bits_down=4)
    host = datagen.moe_weights(wl)
    proj = datagen.random_weights(77, 1, N, H, 4)
    rng = np.random.default_rng(4)
    bf = lambda *s: datagen.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    m = dict(host=host, proj_host=proj, dev=[cbq.prepack_weights(upload_weights(w)) for w in host],
             proj=cbq.prepack_weights(upload_weights(proj)), router=(torch.randn((E, H), device=DEV) / 16))
    m.update({k: (1 + 0.1 * rng.standard_normal(H)).astype(np.float32) for k in ("w_in", "w_post", "w_next")})
    m.update(gate=bf(1, H), a=bf(A, R, H), b=bf(A, N, R))
    m["t"] = {k: to_dev(m[k]) for k in ("w_in", "w_post", "w_next")}
    m["t"].update({k: bf16_dev(m[k]) for k in ("gate", "a", "b")})
    return m


def _step(m, x, of, few):
    t = m["t"]
    normed, codes, scales = cbq.norm_rotate_quantize(x, t["w_in"], 1e-6, 8)
    logits = normed.float() @ m["router"].T
    if few:
        rows = cbq.moe_ffn_few(codes, scales, logits, *m["dev"], TOPK, SHARED, 8)
        slot, tw, sh = None, None, None
    else:
        rt = cbq.moe_route_gather(logits, TOPK, True, SHARED)
        h = cbq.codebook_lut_gemm(codes, scales, 8, m["dev"][:2], expert_offsets=rt["offsets"], row_token=rt["sorted_tokens"])
        ch, sh_ = cbq.rotate_quantize(h, 8)
        rows = cbq.codebook_lut_gemm(ch, sh_, 8, m["dev"][2:], expert_offsets=rt["offsets"])
        slot, tw, sh = rt["slot_of"], rt["weights"], SHARED
    out, n2, c2, s2 = cbq.combine_norm_residual(rows, x, slot, tw, sh, t["w_post"], 1e-6, t["gate"], 0.5,
                                                next_weight=t["w_next"], act_bits=8)
    y = cbq.codebook_adapter_gemm(c2, s2, 8, m["proj"], n2, t["a"], t["b"], of)
    return dict(normed=normed, codes=codes, scales=scales, logits=logits, rows=rows, slot=slot, tw=tw, out=out, n2=n2, c2=c2,
                s2=s2, y=y)


def _f64(t):
    return oracle.reference.bf16_bits_to_f64(bf16_to_bits(t.contiguous()))


@pytest.mark.parametrize("T,few", [(1, True), (5, True), (32, True), (5, False), (80, False)])
def test_block(model, T, few):
    m = model
    x = bf16_dev(datagen.random_tokens(T, T, H))
    of = to_dev((np.arange(T) % (A + 1) - 1).astype(np.int32))
    s = _step(m, x, of, few)
    n = lambda k: s[k].cpu().numpy()  # noqa: E731
    lo, hi = oracle.bf16_candidates(oracle.rms_norm(_f64(x), m["w_in"], 1e-6), 2.0 ** -38)
    got = bf16_to_bits(s["normed"])
    assert np.all((got == lo) | (got == hi))
    rq = oracle.rotate_quantize(got, 0, 8)
    assert np.array_equal(n("codes"), rq["codes"]) and np.array_equal(n("scales"), rq["scale"])
    lg = n("logits")
    if few:
        want = oracle.moe_layer_few(rq["q"].astype(np.int64), rq["scale"], lg, *m["host"], TOPK, SHARED, 8)["y"]
        err = np.abs(_f64(s["rows"]) - want)
        # bf16 output, and codes of h that differ by one step of 1 / 127 of a row's largest value
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + 4e-3 * np.abs(want).max())
        rows, slot, tw, sh = _f64(s["rows"]), None, None, 1
    else:
        rt = oracle.route(lg, TOPK, True, SHARED)
        assert np.array_equal(n("slot"), rt["slot_of"])
        rows, slot, tw, sh = n("rows"), n("slot"), n("tw"), SHARED
    v = oracle.combine_norm_residual(rows, _f64(x), slot, tw, sh, m["w_post"], 1e-6, oracle.reference.bf16_bits_to_f64(m["gate"]),
                                     0.5)
    f = oracle.round_f64_via_f32_to_bf16_bits
    e = 2.0 ** -38 * (np.abs(v).max(axis=1, keepdims=True) + 40 * 8)
    ob = bf16_to_bits(s["out"])
    assert np.all((ob == f(v - e)) | (ob == f(v + e)) | (ob == f(v)))
    lo, hi = oracle.bf16_candidates(oracle.rms_norm(_f64(s["out"]), m["w_next"], 1e-6), 2.0 ** -38)
    nb = bf16_to_bits(s["n2"])
    assert np.all((nb == lo) | (nb == hi))
    rq = oracle.rotate_quantize(nb, 0, 8)
    assert np.array_equal(n("c2"), rq["codes"]) and np.array_equal(n("s2"), rq["scale"])
    W = oracle.dequantize(oracle.unpack_indices(m["proj_host"].idx[0], H, 4), m["proj_host"].codebook[0])
    b = oracle.reference.bf16_bits_to_f64
    args = (oracle.reference.bf16_bits_to_f64(nb), b(m["a"]), b(m["b"]), of.cpu().numpy(), None)
    want = oracle.adapter_gemm(rq["q"], rq["scale"], W, *args)
    mag = oracle.adapter_gemm(np.abs(rq["q"]), rq["scale"], np.abs(W), *(np.abs(a) for a in args[:3]), args[3], None)
    assert np.all(np.abs(n("y") - want) <= 6.1e-5 * mag)


@pytest.mark.parametrize("T", [1, 12])
def test_block_captured(model, T):
    x = bf16_dev(datagen.random_tokens(3, T, H))
    of = torch.zeros((T,), dtype=torch.int32, device=DEV)
    _step(model, x, of, True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = _step(model, x, of, True)
    for k in range(5):
        x.copy_(bf16_dev(datagen.random_tokens(100 + k, T, H)))
        of.copy_(torch.randint(-1, A, (T,), device=DEV, dtype=torch.int32))
        eager = {q: v.clone() for q, v in _step(model, x, of, True).items() if v is not None}
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for q, v in eager.items():
            assert torch.equal(v, cap[q]), (k, q)
