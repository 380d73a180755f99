"""The FMA-pipe exp2 of the packed attention's softmax: its embedded quartic matches the fit of
polynomials that are exactly 1 at 0, and the emulated float32 arithmetic stays within the fit's
error and its own roundings of 2^x."""
import os
import re

import numpy as np

from block_sparse_long_06_b200 import exp2_poly_fit as F

SRC = os.path.join(os.path.dirname(os.path.dirname(__file__)), "block_sparse_long_06_b200",
                   "csrc", "packed_attn.cu")


def embedded():
    text = open(SRC).read()
    return [1.0] + [float(re.search(r"kC%d\s*=\s*([0-9.eE+-]+)f" % i, text).group(1))
                    for i in (1, 2, 3, 4)]


def test_embedded_coefficients_match_the_fit():
    c, err = F.remez_exp2_unit()
    assert c[0] == 1.0 and err < 3e-6
    assert np.allclose(np.float32(c), np.float32(embedded()), rtol=0, atol=2e-7)


def test_the_fit_alternates():
    """Five equal extrema of alternating sign in the weighted error: no polynomial of the kind
    does better."""
    c, err = F.remez_exp2_unit()
    x = np.linspace(-0.5, 0.5, 400001)
    e = np.sign(x) * (np.polyval(c[::-1], x) / 2.0 ** x - 1.0)
    peaks = np.sign(e[np.abs(e) > 0.999 * err])
    assert 1 + np.count_nonzero(peaks[1:] != peaks[:-1]) == 5


def emulate(x):
    """The kernel's float32 arithmetic; the multiply-adds are rounded twice here, once there."""
    c = [np.float32(v) for v in embedded()]
    x = np.maximum(x.astype(np.float32), np.float32(-127.0))
    shift = np.float32(12582912.0)
    r = x + shift
    f = x + (shift - r)
    p = (((c[4] * f + c[3]) * f + c[2]) * f + c[1]) * f + c[0]
    bits = p.view(np.uint32).astype(np.uint64) + (r.view(np.uint32).astype(np.uint64) << np.uint64(23))
    return (bits & np.uint64(0xFFFFFFFF)).astype(np.uint32).view(np.float32)


def test_emulated_exp2():
    """3e-6 of the fit; the last step rounds to 2^-24 and, before it, terms below 0.36 with four
    roundings each: below 6 2^-24. Whole numbers are exact, and -127 and below give 0."""
    x = np.concatenate([np.linspace(-125.0, 8.0, 2_000_001), np.linspace(-1, 1, 100001)])
    got, ref = emulate(x).astype(np.float64), 2.0 ** x.astype(np.float32).astype(np.float64)
    assert np.abs(got / ref - 1.0).max() < 3e-6 + 6 * 2.0 ** -24
    whole = np.arange(-126, 9)
    assert np.array_equal(emulate(whole), np.float32(2.0) ** whole.astype(np.float32))
    assert not emulate(np.array([-127.0, -1000.0, -np.inf])).any()
