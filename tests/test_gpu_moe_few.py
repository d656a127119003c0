"""moe_ffn_few against the fp64 oracle.

Errors of y against the oracle's fp64 layer.  g and u are sums of K exact products in fp32:
their error is below K/32 * 2^-24 of the sum of magnitudes, in practice a few 1e-7 of h's
scale.  A code of h differs from the oracle's only where v / s lies that close to a rounding
border, about 1e-6 a code (A4) and 2e-5 (A8), and then by one step of s.  A differing code
moves a row's output by its weight's column times s, s = max|u_h| / Q.  The tests bound
both: the share of differing codes is not seen directly, so y is compared with the oracle
whose codes of h come from its own h (free-running), allowing one differing code in each
row: |dy| <= sum over rows of w_row * s_row * max|W_down| plus 2e-5 of max|y| for fp32 sums,
and bf16 rounding 2^-8 |y| where y is bf16.  Most elements must meet the bound without
the differing codes (all rows but those few)."""
import numpy as np
import pytest
import torch

import datagen
import oracle

pytestmark = pytest.mark.gpu

cbq = pytest.importorskip("codebook_bit_quantized_amd")
from gpu_util import DEV, bf16_dev, to_dev, upload_weights  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cbq.load_library()


def _inputs(T, H, F, E, topk, n_shared, bits_gu, bits_d, act_bits, seed=0):
    wl = datagen.Workload("few", 4000 + seed, "moe", act_bits, H=H, F=F, E=E, topk=topk, n_shared=n_shared,
                          bits_gate_up=bits_gu, bits_down=bits_d)
    gate, up, down = datagen.moe_weights(wl)
    x, lg = datagen.moe_tokens(wl, T)
    return gate, up, down, x, lg


def _check_layer(T, H, F, E, topk, n_shared=0, bits_gu=4, bits_d=4, act_bits=4, renorm=True, blocked=True,
                 y_dtype=torch.float32, logits=None, seed=0):
    gate, up, down, x, lg = _inputs(T, H, F, E, topk, n_shared, bits_gu, bits_d, act_bits, seed)
    if logits is not None:
        lg = logits
    dev = [upload_weights(w) for w in (gate, up, down)]
    if blocked:
        dev = [cbq.prepack_weights(w) for w in dev]
    codes, scales = cbq.rotate_quantize(bf16_dev(x), act_bits)
    y = cbq.moe_ffn_few(codes, scales, to_dev(lg), *dev, topk, n_shared, act_bits, renorm, y_dtype=y_dtype)
    assert y.dtype == y_dtype and y.shape == (T, H)
    q = oracle.unpack_codes(codes.cpu().numpy(), H, act_bits)
    want = oracle.moe_layer_few(q, scales.cpu().numpy(), lg, gate, up, down, topk, n_shared, act_bits, renorm)
    got = y.float().cpu().numpy().astype(np.float64)
    big = np.abs(want["y"]).max()
    tight = 2e-5 * big + (2.0 ** -8 * np.abs(want["y"]) if y_dtype == torch.bfloat16 else 0)
    wts = np.concatenate([want["route"]["weights64"].ravel(), np.ones(T * n_shared)])
    wmax = max(np.abs(oracle.reference.f16_bits_to_f64(down.codebook)).max(), 0)
    loose = np.zeros((T, 1))
    np.add.at(loose[:, 0], want["token"], wts * want["sh"].astype(np.float64) * wmax)
    err = np.abs(got - want["y"])
    assert np.all(err <= tight + loose), (float(err.max()), float(big))
    # tokens with a differing code of h are rare: two in a hundred thousand codes
    off = np.mean(np.any(err > tight, axis=1))
    allowed = min(1.0, 2e-5 * (topk + n_shared) * F * (4 if act_bits == 8 else 1)) * T
    assert off * T <= max(1.0, 3 * allowed), (off, allowed)
    return y


@pytest.mark.parametrize("T", [1, 2, 3, 8, 15, 16, 17, 31, 32])
def test_token_counts(T):
    _check_layer(T, 256, 192, 16, 4, 1, 3, 2, 4)


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("act_bits", [4, 8])
@pytest.mark.parametrize("blocked", [False, True])
def test_bits_and_layouts(bits, act_bits, blocked):
    _check_layer(5, 320, 224, 12, 3, 0, bits, 6 - bits, act_bits, blocked=blocked)


@pytest.mark.parametrize("E,topk,n_shared", [(1, 1, 0), (1, 1, 8), (8, 8, 0), (8, 2, 0), (63, 6, 2), (64, 1, 0),
                                             (65, 8, 1), (128, 8, 0), (200, 7, 0), (256, 8, 2)])
@pytest.mark.parametrize("T", [1, 20])
def test_experts(E, topk, n_shared, T):
    _check_layer(T, 64, 96, E, topk, n_shared, 2, 4, 8)


@pytest.mark.parametrize("H,F", [(32, 32), (96, 64), (2048, 768), (2560, 160), (4096, 1408), (160, 2048), (64, 14336)])
def test_sizes(H, F):
    _check_layer(4, H, F, 6, 2, 1, 4, 3, 4)


@pytest.mark.parametrize("H,F,E,topk,n_shared", [(32, 32, 8, 2, 0), (96, 64, 8, 8, 8), (2048, 768, 16, 8, 0), (64, 1408, 9, 6, 2),
                                                 (48 * 32, 160, 70, 3, 1), (64, 512, 130, 8, 0), (96, 1024, 8, 4, 1),
                                                 (128, 2048, 12, 8, 3), (128, 2048, 9, 8, 8), (64, 2016, 20, 5, 0),
                                                 (64, 2080, 6, 2, 1), (64, 4096, 4, 2, 0)])
@pytest.mark.parametrize("act_bits", [4, 8])
def test_one_token(H, F, E, topk, n_shared, act_bits):
    _check_layer(1, H, F, E, topk, n_shared, 4, 3, act_bits)
    _check_layer(1, H, F, E, topk, n_shared, 2, 4, act_bits, renorm=False, blocked=False, y_dtype=torch.bfloat16)


@pytest.mark.parametrize("F,topk,n_shared", [(2048, 4, 2), (768, 8, 8), (800, 8, 8), (1536, 8, 0), (1568, 8, 0), (2048, 6, 1)])
def test_one_token_at_the_limits_of_its_form(F, topk, n_shared):
    """12288 values of h and 2048 a row are the one-token form's largest; beyond, the batch form runs."""
    _check_layer(1, 64, F, 9, topk, n_shared, 4, 3, 8)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
def test_weights_and_output_types(renorm, y_dtype):
    _check_layer(9, 512, 256, 40, 6, 2, 3, 3, 8, renorm=renorm, y_dtype=y_dtype)


def test_ties_and_one_expert_for_all():
    """Equal logits go to the lower id; one expert can hold every token."""
    T, E = 32, 24
    lg = np.zeros((T, E), dtype=np.float32)
    lg[::2] = -0.0
    lg[5, 3] = lg[5, 9] = 1.0
    _check_layer(T, 128, 64, E, 4, 0, 4, 4, 8, logits=lg)
    lg = np.full((T, E), -3.0e38, dtype=np.float32)          # masked experts, one left
    lg[:, 7] = 2.0
    _check_layer(T, 128, 64, E, 1, 0, 4, 4, 8, logits=lg)
    _check_layer(2, 128, 64, E, 3, 1, 4, 4, 8, logits=lg[:2])


def test_masked_experts_at_minus_infinity():
    """Experts ruled out by -inf logits keep their rank order and get weight 0."""
    T, E = 6, 10
    rng = np.random.default_rng(0)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    lg[:, 4:] = -np.inf
    lg[3, 1:] = -np.inf
    _check_layer(T, 128, 64, E, 3, 0, 4, 4, 8, logits=lg)
    _check_layer(T, 128, 64, E, 3, 0, 4, 4, 8, renorm=False, logits=lg)


def test_zero_token_and_zero_tokens():
    gate, up, down, x, lg = _inputs(3, 128, 64, 8, 2, 1, 4, 4, 4)
    dev = [cbq.prepack_weights(upload_weights(w)) for w in (gate, up, down)]
    x[1] = 0
    codes, scales = cbq.rotate_quantize(bf16_dev(x), 4)
    y = cbq.moe_ffn_few(codes, scales, to_dev(lg), *dev, 2, 1, 4)
    assert not y[1].any() and y[0].any() and torch.isfinite(y.float()).all()
    y = cbq.moe_ffn_few(codes[:0], scales[:0], to_dev(lg)[:0], *dev, 2, 1, 4)
    assert y.shape == (0, 128)


def test_same_result_alone_and_in_a_batch_and_twice():
    """A token's output does not depend on its batch's other tokens beyond fp32 sums' order,
    and the same call gives the same bits."""
    gate, up, down, x, lg = _inputs(12, 512, 256, 32, 4, 1, 3, 3, 8)
    dev = [cbq.prepack_weights(upload_weights(w)) for w in (gate, up, down)]
    codes, scales = cbq.rotate_quantize(bf16_dev(x), 8)
    L = to_dev(lg)
    run = lambda a, b: cbq.moe_ffn_few(codes[a:b], scales[a:b], L[a:b], *dev, 4, 1, 8, y_dtype=torch.float32)  # noqa: E731
    both = run(0, 12)
    assert torch.equal(both, run(0, 12))
    alone = torch.cat([run(t, t + 1) for t in range(12)])
    assert (both - alone).abs().max() <= 2e-3 * both.abs().max()


def test_strided_output_keeps_its_neighbours_and_ws_given():
    gate, up, down, x, lg = _inputs(5, 128, 96, 8, 2, 0, 4, 4, 8)
    dev = [cbq.prepack_weights(upload_weights(w)) for w in (gate, up, down)]
    codes, scales = cbq.rotate_quantize(bf16_dev(x), 8)
    want = cbq.moe_ffn_few(codes, scales, to_dev(lg), *dev, 2, 0, 8)
    big = torch.full((7, 160), 9.0, dtype=torch.bfloat16, device=DEV)
    n = cbq.moe_few_workspace(5, 2, 0, 128, 96, 8)
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    cbq.moe_ffn_few(codes, scales, to_dev(lg), *dev, 2, 0, 8, y=big[1:6, :128], ws=ws[:n])
    assert torch.equal(big[1:6, :128], want)
    assert (big[0] == 9).all() and (big[6] == 9).all() and (big[:, 128:] == 9).all() and (ws[n:] == 0xA5).all()


def test_streams_and_graph_replay():
    gate, up, down, x, lg = _inputs(6, 256, 128, 16, 4, 1, 3, 2, 4)
    dev = [cbq.prepack_weights(upload_weights(w)) for w in (gate, up, down)]
    codes, scales = cbq.rotate_quantize(bf16_dev(x), 4)
    L = to_dev(lg)
    call = lambda st=None: cbq.moe_ffn_few(codes, scales, L, *dev, 4, 1, 4, stream=st)  # noqa: E731
    want = call()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s1, s2):
        st.wait_stream(torch.cuda.current_stream())
    a, b = call(s1), call(s2)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = call()
    for k in range(4):
        L.normal_()
        eager = call().clone()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap, eager), k


def test_argument_checks():
    gate, up, down, x, lg = _inputs(3, 128, 64, 8, 2, 0, 4, 4, 4)
    dev = [upload_weights(w) for w in (gate, up, down)]
    codes, scales = cbq.rotate_quantize(bf16_dev(x), 4)
    L = to_dev(lg)
    with pytest.raises(ValueError):
        cbq.moe_ffn_few(codes[:, :32], scales, L, *dev, 2)
    with pytest.raises(ValueError):
        cbq.moe_ffn_few(codes, scales, L.double(), *dev, 2)
    with pytest.raises(ValueError):
        cbq.moe_ffn_few(codes, scales, L.cpu(), *dev, 2)
    with pytest.raises(ValueError):
        cbq.moe_ffn_few(codes, scales, L, *dev, 2, y_dtype=torch.float16)
    with pytest.raises(cbq.CbqError):
        cbq.moe_ffn_few(codes, scales, L, *dev, 9)
    with pytest.raises(cbq.CbqError) as e:
        cbq.moe_ffn_few(codes, scales, L, *dev, 2, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == cbq.CBQ_EWORKSPACE
    many = cbq.FEW_MAX_TOKENS + 1
    with pytest.raises(cbq.CbqError) as e:
        cbq.moe_ffn_few(codes[:1].repeat(many, 1), scales[:1].repeat(many), L[:1].repeat(many, 1), *dev, 2)
    assert e.value.status == cbq.CBQ_EUNSUPPORTED


@pytest.mark.parametrize("T", [2, 9])
def test_another_tokens_infinities_stay_with_it(T):
    """A masked-out token (all logits -inf) and one with an infinite scale leave the other
    tokens' outputs as they are, bit for bit."""
    gate, up, down, x, lg = _inputs(T, 256, 128, 16, 4, 1, 3, 2, 4)
    dev = [cbq.prepack_weights(upload_weights(w)) for w in (gate, up, down)]
    codes, scales = cbq.rotate_quantize(bf16_dev(x), 4)
    L = to_dev(lg)
    run = lambda s, l: cbq.moe_ffn_few(codes, s, l, *dev, 4, 1, 4, y_dtype=torch.float32)  # noqa: E731
    want = run(scales, L)
    masked = L.clone()
    masked[1] = float("-inf")
    got = run(scales, masked)
    keep = torch.arange(T, device=DEV) != 1
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[1]).all()
    huge = scales.clone()
    huge[1] = float("inf")
    got = run(huge, L)
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[1]).all()
    nan = L.clone()
    nan[1, 3:9] = float("nan")
    got = run(scales, nan)
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("T,E", [(32, 8), (32, 70), (1, 8)])
def test_logits_of_any_nan(T, E):
    """Whatever bits a NaN has, its token still takes distinct experts, so no other token's rows go missing."""
    gate, up, down, x, lg = _inputs(T, 64, 96, E, 8, 0, 3, 2, 4)
    dev = [cbq.prepack_weights(upload_weights(w)) for w in (gate, up, down)]
    codes, scales = cbq.rotate_quantize(bf16_dev(x), 4)
    L = to_dev(lg)
    L[:, 8:] -= 100.0                                        # every token visits the first eight
    run = lambda l: cbq.moe_ffn_few(codes, scales, l, *dev, 8, 0, 4, y_dtype=torch.float32)  # noqa: E731
    want = run(L)
    for bits in (-1, -2, 0x7FFFFFFF, 0x7FC00000, -0x400000):
        bad = L.clone()
        bad.view(torch.int32)[::2] = bits
        got = run(bad)
        assert torch.isnan(got[::2]).all() and torch.equal(got[1::2], want[1::2])
