"""Host-side checks of the calls around a block: invalid arguments give the documented status
before any HIP call, so every refusal runs on a machine without a GPU."""
import ctypes
import os

import pytest

cbq = pytest.importorskip("codebook_bit_quantized_amd")

P, U = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cbq.LIB_PATH):
        pytest.skip("libcbq.so not built")
    return cbq.load_library()


def _norm(weight=0x1000, eps=1e-6, had_block=0, act_bits=4, normed=0x1000, ldn=256, codes=0x1000, scales=0x1000):
    return ctypes.byref(cbq._binding.cbq_norm(weight, eps, had_block, act_bits, normed, ldn, codes, scales))


def test_norm_rotate_quantize_refusals(lib):
    f = lib.cbq_norm_rotate_quantize
    assert f(P, -1, 256, 256, _norm(), None) == cbq.CBQ_EINVAL
    assert f(P, 1 << 31, 256, 256, _norm(), None) == cbq.CBQ_EUNSUPPORTED
    assert f(P, 4, 250, 256, _norm(), None) == cbq.CBQ_EINVAL
    assert f(P, 4, 32768, 32768, _norm(), None) == cbq.CBQ_EUNSUPPORTED
    assert f(P, 4, 256, 248, _norm(), None) == cbq.CBQ_EINVAL
    assert f(P, 4, 256, 260, _norm(), None) == cbq.CBQ_EINVAL
    assert f(P, 4, 256, 256, None, None) == cbq.CBQ_EINVAL
    assert f(None, 4, 256, 256, _norm(), None) == cbq.CBQ_EINVAL
    assert f(U, 4, 256, 256, _norm(), None) == cbq.CBQ_EINVAL
    for bad in (dict(weight=None), dict(weight=0x1004), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(normed=None, codes=None), dict(normed=0x1008), dict(ldn=248),
                dict(ldn=260), dict(act_bits=5), dict(had_block=3), dict(had_block=512), dict(had_block=-2),
                dict(scales=None), dict(codes=0x1004)):
        assert f(P, 4, 256, 256, _norm(**bad), None) == cbq.CBQ_EINVAL, bad
        assert lib.cbq_last_error()
    assert f(None, 0, 256, 256, _norm(), None) == cbq.CBQ_OK


def test_combine_norm_residual_refusals(lib):
    def f(rows=P, rows_type=0, ldr=256, slot_of=P, topk_w=P, T=4, topk=2, n_shared=1, H=256, post_weight=P,
          post_eps=1e-6, gate=P, ldg=256, scale=1.0, residual=P, ldres=256, out=P, ldo=256, nxt=None):
        return lib.cbq_combine_norm_residual(rows, rows_type, ldr, slot_of, topk_w, T, topk, n_shared, H, post_weight,
                                             post_eps, gate, ldg, scale, residual, ldres, out, ldo, nxt, None)

    for bad in (dict(T=-1), dict(H=250), dict(rows_type=2), dict(topk=9), dict(topk=-1), dict(n_shared=9),
                dict(topk=0, n_shared=0), dict(ldr=252), dict(ldr=258), dict(rows_type=1, ldr=260), dict(ldres=248),
                dict(ldo=260), dict(ldg=8), dict(ldg=260), dict(post_eps=0.0), dict(rows=None), dict(residual=None),
                dict(out=None), dict(slot_of=None), dict(topk_w=None), dict(rows=U), dict(residual=U), dict(out=U),
                dict(post_weight=U), dict(gate=U), dict(nxt=_norm(eps=0.0)), dict(nxt=_norm(normed=None, codes=None))):
        assert f(**bad) == cbq.CBQ_EINVAL, bad
        assert lib.cbq_last_error()
    assert f(H=32768, ldr=32768, ldres=32768, ldo=32768, ldg=0) == cbq.CBQ_EUNSUPPORTED
    assert f(T=0, rows=None, residual=None, out=None) == cbq.CBQ_OK


def _w(E=10, N=96, K=128, bits=4, layout=0, idx=0x1000, cb=0x1000):
    return ctypes.byref(cbq.cbq_weights(idx, cb, E, N, K, bits, layout))


def test_moe_ffn_few_refusals(lib):
    need = lib.cbq_moe_few_workspace(4, 2, 2, 128, 96, 4)
    assert need > 0

    def f(codes=P, scales=P, act_bits=4, logits=P, T=4, E=8, topk=2, renorm=1, n_shared=2, gate=_w(), up=_w(),
          down=_w(N=128, K=96), y=P, y_type=0, ldy=128, ws=P, n=None):
        return lib.cbq_moe_ffn_few(codes, scales, act_bits, logits, T, E, topk, renorm, n_shared, gate, up, down, y,
                                   y_type, ldy, ws, need if n is None else n, None)

    for bad in (dict(T=-1), dict(topk=0), dict(topk=9), dict(E=1, n_shared=9), dict(n_shared=-1), dict(renorm=2),
                dict(act_bits=16), dict(gate=None), dict(up=None), dict(down=None), dict(gate=_w(E=9)),
                dict(up=_w(N=80)), dict(up=_w(bits=3)), dict(up=_w(layout=1)), dict(down=_w(N=96, K=128)),
                dict(gate=_w(idx=None)), dict(gate=_w(cb=0x1004)), dict(gate=_w(layout=7)), dict(y_type=2),
                dict(ldy=124), dict(ldy=130), dict(codes=None), dict(scales=None), dict(logits=None), dict(y=None),
                dict(codes=U), dict(y=U), dict(ws=U)):
        assert f(**bad) == cbq.CBQ_EINVAL, bad
        assert lib.cbq_last_error()
    assert f(T=33) == cbq.CBQ_EUNSUPPORTED
    assert f(E=257) == cbq.CBQ_EUNSUPPORTED
    assert f(gate=_w(bits=5)) == cbq.CBQ_EUNSUPPORTED
    assert f(ws=None) == cbq.CBQ_EWORKSPACE and f(n=need - 1) == cbq.CBQ_EWORKSPACE
    assert f(T=0, codes=None, logits=None, y=None, ws=None) == cbq.CBQ_OK
    wide = dict(gate=_w(N=16384 + 32), up=_w(N=16384 + 32), down=_w(N=128, K=16384 + 32))
    assert f(**wide) == cbq.CBQ_EUNSUPPORTED


def test_moe_few_workspace_sizes(lib):
    f = lib.cbq_moe_few_workspace
    assert f(0, 2, 0, 128, 96, 4) == 0 and f(33, 2, 0, 128, 96, 4) == 0 and f(1, 9, 0, 128, 96, 4) == 0
    assert f(32, 8, 8, 16384, 16384, 8) >= 32 * 16 * (4 + 1 + 4) * 16384


def test_codebook_adapter_gemm_refusals(lib):
    need = lib.cbq_adapter_workspace(4, 16)
    assert need >= 4 * 16 * 4 and lib.cbq_adapter_workspace(4, 12) == 0 and lib.cbq_adapter_workspace(0, 16) == 0

    def f(codes=P, scales=P, act_bits=4, T=4, W=_w(E=1), x=P, ldx=128, a=P, b=P, sc=None, n_ad=3, rank=16, of=P, out=P,
          ldo=96, ws=P, n=need):
        return lib.cbq_codebook_adapter_gemm(codes, scales, act_bits, T, W, x, ldx, a, b, sc, n_ad, rank, of, out, ldo,
                                             ws, n, None)

    for bad in (dict(W=None), dict(W=_w(E=2)), dict(W=_w(E=1, K=100)), dict(act_bits=5), dict(T=-1), dict(ldx=120),
                dict(ldx=130), dict(ldo=92), dict(ldo=98), dict(n_ad=0), dict(rank=0), dict(rank=12), dict(rank=136),
                dict(codes=None), dict(scales=None), dict(x=None), dict(a=None), dict(b=None), dict(of=None),
                dict(out=None), dict(codes=U), dict(x=U), dict(a=U), dict(b=U), dict(out=U), dict(ws=U)):
        assert f(**bad) == cbq.CBQ_EINVAL, bad
        assert lib.cbq_last_error()
    assert f(T=1 << 31) == cbq.CBQ_EUNSUPPORTED
    assert f(T=3 << 20) == cbq.CBQ_EUNSUPPORTED                       # out of 1 GiB or more
    assert f(W=_w(E=1, K=16416), ldx=16416) == cbq.CBQ_EUNSUPPORTED
    assert f(ws=None) == cbq.CBQ_EWORKSPACE and f(n=need - 1) == cbq.CBQ_EWORKSPACE
    assert f(T=0, codes=None, x=None, out=None, ws=None) == cbq.CBQ_OK
