"""f8 host quantizer at the ends of fp32's range."""
import numpy as np
import pytest

import f8_util as fu

MOST = 240.0 * 2.0 ** 120          # the largest code times the largest scale that fp32 still holds
FAR = [np.finfo(np.float32).max, 3.35e38, 3.31e38, 248.0 * 2.0 ** 120, 247.9 * 2.0 ** 120, 3.2e38, -3.4e38, 1e30, 0.0]


def capped(v):
    """The definition with a finite result for every finite value: codes of the scale 2^120 stop at 240."""
    q, e = fu.quantize_rows(np.asarray(v, np.float64)[None])
    return np.where(e[0][0] == 120, np.clip(q[0], -MOST, MOST), q[0])


def test_finite_weights_stay_finite():
    import quantized_weight_gemv_amd as q
    for first in range(len(FAR) - 2):
        w = np.array([FAR[first:]], np.float32)
        got, clean = fu.unpack_weights(q.qquantize_f8(w), 1, w.shape[1])
        assert clean and np.isfinite(got.astype(np.float32)).all()
        assert np.array_equal(got[0], capped(w[0])), first


def test_only_the_largest_scale_is_capped():
    """A block one step down keeps its code of 256 and more."""
    import quantized_weight_gemv_amd as q
    w = (np.array([[448.0, 300.0, 256.0, 250.0, -449.0 / 2]]) * 2.0 ** 119).astype(np.float32)
    got, _ = fu.unpack_weights(q.qquantize_f8(w), 1, 5)
    assert np.array_equal(got, fu.quantize_weights(w)[0])


def test_capped_reference():
    assert np.array_equal(capped([3.4e38, -3.4e38, 3.2e38]), [MOST, -MOST, 240.0 * 2.0 ** 120])
    assert float(np.float32(MOST)) == MOST and 256.0 * 2.0 ** 120 > float(np.finfo(np.float32).max)
