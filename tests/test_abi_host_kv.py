"""Host-side checks of the key/value cache's calls: invalid arguments give the documented status before
any HIP call, so every refusal runs on a machine without a GPU."""
import ctypes
import os

import pytest

cbq = pytest.importorskip("codebook_bit_quantized_amd")

P, U = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cbq.LIB_PATH):
        pytest.skip("libcbq.so not built")
    return cbq.load_library()


def _cache(kc=0x1000, vc=0x1000, ks=0x1000, vs=0x1000, n_pages=8, n_kv=2, page=16, D=64, rotate=3):
    return ctypes.byref(cbq._binding.cbq_kv_cache(kc, vc, ks, vs, n_pages, n_kv, page, D, rotate))


def _seqs(table=0x1000, ld=4, max_pages=4, lens=0x1000, offsets=0x1000, B=3):
    return ctypes.byref(cbq._binding.cbq_kv_seqs(table, ld, max_pages, lens, offsets, B))


CACHE = [(dict(n_pages=0), "EINVAL"), (dict(n_kv=0), "EINVAL"), (dict(n_kv=1025), "EUNSUPPORTED"), (dict(n_pages=1 << 30), "EUNSUPPORTED"), (dict(page=8), "EINVAL"),
         (dict(page=48), "EINVAL"), (dict(page=0), "EINVAL"), (dict(page=-16), "EINVAL"), (dict(page=2048), "EINVAL"),
         (dict(D=96), "EUNSUPPORTED"), (dict(D=0), "EUNSUPPORTED"), (dict(D=256), "EUNSUPPORTED"), (dict(rotate=4), "EINVAL"),
         (dict(rotate=-1), "EINVAL"), (dict(kc=None), "EINVAL"), (dict(vc=None), "EINVAL"), (dict(ks=None), "EINVAL"),
         (dict(vs=None), "EINVAL"), (dict(kc=0x1008), "EINVAL"), (dict(vc=0x1004), "EINVAL"), (dict(ks=0x1008), "EINVAL"),
         (dict(vs=0x1004), "EINVAL")]
SEQS = [(dict(B=-1), "EINVAL"), (dict(B=65537), "EUNSUPPORTED"), (dict(max_pages=0), "EINVAL"), (dict(ld=3), "EINVAL"),
        (dict(max_pages=1 << 27, ld=1 << 27), "EUNSUPPORTED"), (dict(lens=None), "EINVAL"),
        (dict(table=None, max_pages=3), "EINVAL"), (dict(offsets=None, B=5), "EINVAL"), (dict(offsets=None, B=0), "EINVAL")]


def _all(f):
    for bad, st in CACHE:
        assert f(cache=_cache(**bad)) == getattr(cbq, "CBQ_" + st), bad
    for bad, st in SEQS:
        assert f(seqs=_seqs(**bad)) == getattr(cbq, "CBQ_" + st), bad
    assert f(cache=None) == cbq.CBQ_EINVAL and f(seqs=None) == cbq.CBQ_EINVAL
    assert f(T=-1) == cbq.CBQ_EINVAL and f(T=1 << 31) == cbq.CBQ_EUNSUPPORTED
    assert b"T" in cbq.load_library().cbq_last_error()
    assert f(T=0) == cbq.CBQ_OK and f(T=6, seqs=_seqs(B=0)) == cbq.CBQ_OK


def test_write_and_read_refusals(lib):
    for name in ("cbq_kv_cache_write", "cbq_kv_cache_read"):
        def f(cache=_cache(), seqs=_seqs(), k=P, ldk=128, v=P, ldv=128, T=6):
            return getattr(lib, name)(cache, seqs, k, ldk, v, ldv, T, None)

        _all(f)
        for bad in (dict(ldk=120), dict(ldk=132), dict(ldv=0), dict(ldv=-128), dict(k=U), dict(v=U)):
            assert f(**bad) == cbq.CBQ_EINVAL, bad
        assert f(ldk=(1 << 31) + 8) == cbq.CBQ_EUNSUPPORTED and f(ldv=1 << 62) == cbq.CBQ_EUNSUPPORTED
        assert f(k=None, v=None) == cbq.CBQ_EINVAL
    assert lib.cbq_kv_cache_write(_cache(), _seqs(), None, 128, P, 128, 6, None) == cbq.CBQ_EINVAL
    assert lib.cbq_kv_cache_write(_cache(), _seqs(), P, 128, None, 128, 6, None) == cbq.CBQ_EINVAL


def test_attention_refusals(lib):
    need = lib.cbq_kv_attention_workspace(_cache(), 6, 3, 4)
    assert need > 0

    def f(cache=_cache(), seqs=_seqs(), q=P, ldq=256, T=6, n_q=4, scale=0.125, causal=1, window=0, out=P, ldo=256, ws=P, n=need):
        return lib.cbq_kv_attention(cache, seqs, q, ldq, T, n_q, scale, causal, window, out, ldo, ws, n, None)

    _all(f)
    for bad in (dict(n_q=0), dict(n_q=3), dict(n_q=-2), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2),
                dict(causal=-1), dict(window=-1), dict(causal=0, window=5), dict(ldq=248), dict(ldq=260), dict(ldo=128),
                dict(ldo=258), dict(q=None), dict(out=None), dict(q=U), dict(out=U), dict(ws=U)):
        assert f(**bad) == cbq.CBQ_EINVAL, bad
        assert lib.cbq_last_error()
    assert f(n_q=1026, ldq=1 << 20, ldo=1 << 20) == cbq.CBQ_EUNSUPPORTED
    assert f(ldq=1 << 62) == cbq.CBQ_EUNSUPPORTED and f(ldo=(1 << 31) + 8) == cbq.CBQ_EUNSUPPORTED
    assert f(T=(1 << 30), n_q=2, seqs=_seqs(B=3)) == cbq.CBQ_EUNSUPPORTED            # T * n_q = 2^31
    assert f(ws=None) == cbq.CBQ_EWORKSPACE and f(n=need - 1) == cbq.CBQ_EWORKSPACE


def test_workspace_sizes(lib):
    f = lib.cbq_kv_attention_workspace
    for bad in ((None, 6, 3, 4), (_cache(), 0, 3, 4), (_cache(), 1 << 31, 3, 4), (_cache(), 6, 0, 4), (_cache(), 6, 65537, 4),
                (_cache(), 6, 3, 3), (_cache(), 6, 3, 0), (_cache(), 6, 3, 1026), (_cache(D=96), 6, 3, 4), (_cache(n_kv=0), 6, 3, 4)):
        assert f(*bad) == 0, bad
    assert f(_cache(D=128, n_kv=8), 1 << 20, 1, 64) < 1 << 30


def test_every_call_is_exported(lib):
    for name in ("cbq_kv_cache_write", "cbq_kv_cache_read", "cbq_kv_attention_workspace", "cbq_kv_attention"):
        assert name in cbq.EXPORTED and getattr(lib, name)
