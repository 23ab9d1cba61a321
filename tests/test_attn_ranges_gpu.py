"""The attention step at the ends of the ranges that its calls accept, under bounds that follow from what a result
is, not from an option's size."""
import numpy as np
import pytest

import attn_util as au
from gpu_util import torch_cuda
from test_attn_gpu import _Batch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _np(t):
    torch_cuda().cuda.synchronize()
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ tanh caps
def _capped(b, scale, window, cap):
    """(out, bound of everything but the last rounding) with errors of a score relative to the score.

    A score's products and sums: dim / 8 + 16 roundings of their magnitudes.  The capped score, all relative to the
    score without a cap (tanh's slope is at most 1): its two factors, the scale and its conversion 4; near 0 the series
    and its product 4; far from 0 the exponential with its argument, the reciprocal and the difference, 8 of at least
    tanh(1/2); the cap and its product 2; the distance from the maximum 2 of the largest: under 24.  The rest as
    for scores without a cap (attn_util.attend)."""
    q = _np(b.q)
    B, M, H, D = q.shape
    share = H // b.kv
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for i, n in enumerate(b.lens):
        for j in range(M):
            end = n - M + j + 1
            t = np.arange(max(0, end - window) if window else 0, max(end, 0))
            if not len(t):
                continue
            at = b.table[i][t // b.page] * b.page + t % b.page
            for h in range(H):
                k, v = b.k[at, h // share], b.v[at, h // share]
                raw = k @ q[i, j, h] * scale
                step = (D / 8 + 16) * U * (np.abs(k) @ np.abs(q[i, j, h]) * abs(scale)) + 24 * U * np.abs(raw).max()
                s = cap * np.tanh(raw / cap)
                w = np.exp(s - s.max())
                w /= w.sum()
                out[i, j, h] = w @ v
                bound[i, j, h] = w @ np.abs(v) * (2 * step.max() + 2.0 ** -15 + (len(t) / 8 + 64) * U)
    return out, bound


CAPPED = [  # lens, M, heads, key heads, D, page, cache, q
    ([200, 33, 1, 0], 1, 4, 2, 128, 16, "float16", "float16"),
    ([150, 7], 3, 8, 1, 64, 32, "f8", "float16"),
    ([90, 260], 1, 6, 2, 192, 64, "f8", "bfloat16"),
    ([300], 5, 4, 1, 256, 16, "bfloat16", "bfloat16"),
]


@pytest.mark.parametrize("case", CAPPED)
@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0, 1e3, 1e4, 1e6, 1e8, 1e30, 3.4e38])
@pytest.mark.parametrize("window,wide", [(0, False), (60, True)])
def test_caps_of_every_size(case, cap, window, wide):
    """From caps that hold nearly every score to ones that hold none: a large cap is none, whatever its size."""
    b = _Batch(*case, width=40000 // case[5] if wide else None)
    scale = 2 * b.D ** -0.5
    y = b.run(scale=scale, window=window, softcap=cap)
    out, bound = _capped(b, float(np.float32(scale)), window, float(np.float32(cap)))
    au.assert_attend(_np(y), out, bound, b.q_type, f"cap {cap}")
