"""The quotient of kv_append_dynamic, x / s by a refined reciprocal, against
the division: every pair of 11-bit significands of x and of the row's largest
element, each format's divisor.  (Powers of two change nothing: the residual
does not underflow where the kernel takes this way.)  Arithmetic of the
kernel in numpy: fp32 roundings of float64 values, a fused multiply-add's exact
product and sum in float64 with its rounding error kept."""
import numpy as np
import pytest

F, D = np.float32, np.float64


def fma(a, b, c):
    """round32(a b + c) of fp32 values."""
    t, c = a.astype(D) * b.astype(D), np.broadcast_to(c.astype(D), np.broadcast_shapes(a.shape, b.shape, c.shape))
    hi = t + c                                       # the product is exact, the sum is hi + lo
    z = hi - c
    lo = (c - (hi - z)) + (t - z)
    r = hi.astype(F)
    # hi on the border of two fp32 numbers (or rounded onto it): lo decides
    up, down = np.nextafter(r, F(np.inf)), np.nextafter(r, F(-np.inf))
    mid_up, mid_down = (r.astype(D) + up.astype(D)) / 2, (r.astype(D) + down.astype(D)) / 2
    r = np.where((hi == mid_up) & (lo > 0), up, r)
    return np.where((hi == mid_down) & (lo < 0), down, r)


@pytest.mark.parametrize("qmax", [448.0, 57344.0, 127.0])
def test_every_pair_of_significands(qmax):
    a = np.arange(1024, 2048, dtype=D)
    s = (a / qmax).astype(F)                         # float64's 53 bits are more than 2 x 24 + 1: rounded twice, as once
    r = (1.0 / s.astype(D)).astype(F)
    x = np.arange(1024, 2048, dtype=F)[:, None]
    q = (x.astype(D) * r.astype(D)).astype(F)
    e = fma(q, np.broadcast_to(s, q.shape), -np.broadcast_to(x, q.shape))
    got = fma(-e, np.broadcast_to(r, q.shape), q)
    assert np.array_equal(got, (x.astype(D) / s.astype(D)).astype(F))
