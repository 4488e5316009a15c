"""The arithmetic behind the INT8 codes, on CPU.

The row kernels take the code of a bf16 value y of a row with scale
s = fl32(amax / 127) from the product y * r, where r = fl32(1 / s) moved by 2^-21
towards the side of 63.5 that (amax / 2) / s lies on.  Checked here against the
quotient y / s rounded half to even, over every significand of amax and of y and
every exponent distance at which a code can be non-zero; scaling both by a power
of two scales s with them, so one exponent of amax stands for all normal ones.
"""
import numpy as np
import pytest


def _significands(bits):
    """All positive values of `bits` significant bits in [1, 2)."""
    return 1.0 + np.arange(1 << (bits - 1)) / (1 << (bits - 1))


def _codes(y, amax):
    """Codes of y (2D) for rows of largest magnitude amax (column), as the kernel forms them."""
    f = np.float32
    s = (amax.astype(f) / f(127)).astype(f)
    r = (f(1) / s).astype(f)
    side = 0.5 * amax - 63.5 * s.astype(np.float64)       # exact in fp64: its sign is the FMA's
    r64 = r.astype(np.float64)
    r = np.where(side > 0, r64 * (1 + 2.0 ** -21), np.where(side < 0, r64 * (1 - 2.0 ** -21), r64)).astype(f)
    k = np.rint(y * r.astype(np.float64))                 # the exact product (32 bits), rounded half to even by the FMA
    return k.astype(np.int64), s


@pytest.mark.parametrize("e", range(10))                   # codes are 0 from 2^-9 of amax down
def test_product_codes_equal_the_rounded_quotient(e):
    sig = _significands(8)
    a, y = sig[:, None], sig[None, :] * 2.0 ** -e
    got, s = _codes(np.broadcast_to(y, (128, 128)), a)
    want = np.rint(y / s.astype(np.float64)).astype(np.int64)
    fits = np.broadcast_to(y <= a, got.shape)
    assert np.array_equal(got[fits], want[fits])
    assert got[fits].max(initial=0) <= 127


def test_an_fp64_quotient_of_fp32_numbers_never_rounds_onto_a_tie():
    """The rounded fp64 quotient used as the reference decides ties as the exact one: for fp32 y and s and
    h = k + 1/2 (8 bits), y != h s differ by at least 2^-33 of y, far above the fp64 rounding."""
    rng = np.random.default_rng(3)
    s = rng.uniform(1, 2, 20000).astype(np.float32)
    h = rng.integers(0, 127, 20000) + 0.5
    y = (h * s).astype(np.float32)                         # the fp32 number next to the tie
    exact = y.astype(np.float64) - h * s.astype(np.float64)   # exact: 32-bit products
    q = y.astype(np.float64) / s.astype(np.float64)
    assert np.array_equal(np.sign(q - h), np.sign(exact))
