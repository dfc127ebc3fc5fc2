"""The quotient behind the codes of append_chunk: with r = fl(1 / s) and
q = fl(d r), q' = fl(fl(d - q s) r + q) is fl(d / s) for every fp16 scale s and
every fp32 d near the half of a code, where a rounding would change the code.
Each fused operation is computed exactly and rounded once."""
import numpy as np


def scales():
    s = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16)  # all positive finite ones, subnormal ones too
    return s.astype(np.float32)


def near(x, steps):
    """The fp32 numbers up to `steps` away from each of x (all positive)."""
    return (x.view(np.int32)[..., None] + np.arange(-steps, steps + 1, dtype=np.int32)).view(np.float32)


def fma32(a, b, c):
    """fl32(a b + c): the product of two fp32 numbers is exact in 64 bits; the sum
    is rounded to odd there, after which rounding to 32 bits is the only one."""
    p, c = a.astype(np.float64) * b.astype(np.float64), c.astype(np.float64)
    t = p + c
    v = t - p
    err = (p - (t - v)) + (c - v)
    bits = t.view(np.int64)
    odd = np.where(err != 0, (bits - (err * np.sign(t) < 0)) | 1, bits)
    return odd.view(np.float64).astype(np.float32)


def corrected(d, s):
    r = (1.0 / s.astype(np.float64)).astype(np.float32)
    q = (d.astype(np.float64) * r.astype(np.float64)).astype(np.float32)
    return fma32(fma32(-q, s, d), r, q)


def divided(d, s):
    return (d.astype(np.float64) / s.astype(np.float64)).astype(np.float32)  # 53 bits are enough for one rounding to 24


def test_fma32_against_integers():
    """The helper itself, where a sum rounded twice would differ: 1 + 2^-24 and a
    little more or less."""
    one, tiny = np.float32([1, 1, 1]), np.float32([2.0 ** -60, -(2.0 ** -60), 0])
    half = np.float32(2.0 ** -12)
    got = fma32(np.full(3, half), np.full(3, half), one)  # exactly half a step: to even
    assert (got == 1).all()
    a = np.float32([2.0 ** -12 * (1 + 2.0 ** -23), 2.0 ** -12 * (1 - 2.0 ** -24), 2.0 ** -12])
    assert fma32(a, np.full(3, half), one).tolist() == [1 + 2.0 ** -23, 1.0, 1.0]
    big = np.float32([1 + 2.0 ** -23] * 3)
    assert fma32(tiny, one, big).tolist() == [1 + 2.0 ** -23] * 3


def test_near_every_half_of_a_code():
    s = scales()
    for k in range(15):  # both widths: 3 codes' halves are among 15's
        half = ((k + 0.5) * s.astype(np.float64)).astype(np.float32)
        d = near(half, 6).reshape(-1)
        ss = np.repeat(s, 13)
        assert np.array_equal(corrected(d, ss), divided(d, ss)), k


def test_at_every_code_and_between():
    s = scales()
    rng = np.random.default_rng(1)
    for _ in range(8):
        d = (s.astype(np.float64) * rng.uniform(0, 15, s.shape)).astype(np.float32)
        assert np.array_equal(corrected(d, s), divided(d, s))
    for k in range(16):
        d = near((k * s.astype(np.float64)).astype(np.float32), 2).reshape(-1) if k else np.zeros_like(s)
        ss = np.repeat(s, 5) if k else s
        q = corrected(d, ss)
        assert np.array_equal(q, divided(d, ss))
        magic = (q + np.float32(12582912.0)).view(np.uint32) - np.uint32(0x4B400000)  # adding 1.5 x 2^23 leaves rint
        assert (magic == k).all()
