"""The cache quantiser's division by one corrected product, on the CPU for every mantissa: y = fma(fma(-s, y0, 1), y0, y0) from a
start y0 within one step of 1 / s, q = v y, r = fma(fma(-q, s, v), y, q).

Where y is 1 / s rounded to nearest, r is v / s rounded to nearest for every v next to a border of the codes, so the
codes are those of the true quotient.  And y is that for every mantissa of s and every start, but for the mantissa whose
bits are all ones: there only the start that is 1 / s rounded gives it (test_gpu_kv_division.py has that scale on
the hardware)."""
import numpy as np

BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
F, G = np.float32, np.float64


def _fma(a, b, c):
    """fp32 a b + c rounded once: the product is exact in fp64, the sum is rounded to odd there, then to fp32."""
    p, c = a.astype(G) * b.astype(G), c.astype(G)
    s = p + c
    z = s - p
    err = (p - (s - z)) + (c - z)                          # what the sum has lost, exactly
    bits = s.view(np.int64)
    towards = np.where((err > 0) == (s > 0), 1, -1)
    odd = np.where((err != 0) & (bits & 1 == 0), bits + towards, bits)
    return odd.view(G).astype(F)


def _step(x, d):
    return (x.view(np.int32) + np.int32(d)).view(F)


def _mantissas(chunk=1 << 20):
    for m in range(0, 1 << 23, chunk):
        yield (np.arange(m, m + chunk, dtype=np.int32) | np.int32(0x3F800000)).view(F)


def test_fma_rounds_once():
    e = F(2.0 ** -12)
    one = np.array([1], F)
    # (1 + 2^-12)^2 + 2^-60 lies just above the middle of two fp32 values, and less 2^-60 just below
    a = one + e
    up = _fma(a, a, np.array([2.0 ** -60], F))
    down = _fma(a, a, np.array([-2.0 ** -60], F))
    assert up[0] == F(1 + 2.0 ** -11 + 2.0 ** -23) and down[0] == F(1 + 2.0 ** -11)


def test_one_step_gives_the_rounded_reciprocal():
    wrong = []
    for s in _mantissas():
        right = F(1) / s
        for d in (-1, 0, 1):
            y0 = _step(right, d)
            y = _fma(_fma(-s, y0, np.ones_like(s)), y0, y0)
            within = np.abs(y0.astype(G) - 1 / s.astype(G)) <= 2.0 ** -24 * (1 + 2.0 ** -20)      # 1 / s lies in (1/2, 1]
            assert d or within.all()
            wrong += [(float(x), d) for x in s[within & (y != right)]]
    ones = float(F(2 - 2.0 ** -23))
    assert {x for x, _ in wrong} <= {ones} and (ones, 0) not in wrong


def test_quotients_next_to_a_border_are_rounded():
    for s in _mantissas():
        y = F(1) / s
        for b in BORDERS:
            near = (F(b) * s).astype(F)
            for d in (-1, 0, 1):
                v = _step(near, d)
                q = v * y
                r = _fma(_fma(-q, s, v), y, q)
                assert np.array_equal(r, v / s)
