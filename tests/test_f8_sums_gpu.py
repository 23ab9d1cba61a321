"""16-bit outputs of the f8 products are fp32 sums rounded once, also where the
sum is small beside its products."""
import numpy as np
import pytest

import f8_util as fu
from gpu_util import qg, to_dev, torch_cuda

pytestmark = pytest.mark.gpu

HALVES = ("float16", "bfloat16")


def _np(t):
    torch_cuda().cuda.synchronize()
    return t.double().cpu().numpy()


def _bound(ref, s, terms, dtype):
    """fp32 sums (sum_bound), then one rounding to nearest: half a step of what is rounded."""
    b = fu.sum_bound(s, terms)
    return b + fu.HALF_STEP[dtype] * (np.abs(ref) + b) + fu.TINY[dtype]


def _cancelling(rows, cols, seed, signed):
    """Whole numbers that f8 holds exactly, one pair of 256 in each block of 128 columns whose products
    cancel (signed: the side with both signs) beside products of 1 to 6: two of 2^16 a block."""
    g = np.random.default_rng([rows, cols, seed])
    v = g.integers(1, 4 if signed else 3, size=(rows, cols)).astype(np.float32)
    for c in range(0, cols - 1, 128):
        at = c + int(g.integers(0, min(128, cols - c) - 1))
        v[:, at] = 256.0
        v[:, at + 1] = -256.0 if signed else 256.0
    return v


def _pair(M, N, K):
    """x [M][K] and w [N][K] whose pairs stand in the same columns."""
    x = _cancelling(M, K, 1, signed=True)
    w = np.random.default_rng([N, K]).integers(1, 3, size=(N, K)).astype(np.float32)
    w[:, np.abs(x[0]) == 256.0] = 256.0
    return x, w


# one of each tile shape: 64 x 128, 128 x 128 of both depths, 256 x 256, and the streaming kernels
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,N,K", [(9, 40, 256), (50, 300, 130), (100, 500, 256), (640, 4100, 200), (1030, 6000, 130),
                                   (2100, 8200, 256), (3600, 3399, 257)])
def test_sums_that_cancel(M, N, K, dtype):
    q, torch = qg(), torch_cuda()
    x, w = _pair(M, N, K)
    W, xq = to_dev(q.qquantize_f8(w)), q.qact_quantize_f8(to_dev(x))
    xd, wd = to_dev(x).double(), to_dev(w).double()
    assert torch.equal(q.qact_dequant_f8(xq, M, K).double(), xd) and torch.equal(q.qdequant_f8(W, N, K).double(), wd)
    ref, s = _np(xd @ wd.t().contiguous()), _np(xd.abs() @ wd.abs().t().contiguous())
    y = q.qgemm_f8(W, xq, M, N, K, dtype=getattr(torch, dtype))
    fu.assert_close(_np(y), ref, _bound(ref, s, K, dtype), f"{M}x{N}x{K} {dtype}")


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("P,T,k,N,K", [(4, 9, 2, 40, 256), (3, 300, 2, 130, 257), (2, 5000, 1, 260, 200)])
def test_sums_of_experts_that_cancel(P, T, k, N, K, dtype):
    q, torch = qg(), torch_cuda()
    x, w = _pair(T, P * N, K)
    w = w.reshape(P, N, K)
    pool = to_dev(np.concatenate([q.qquantize_f8(v) for v in w]))
    g = np.random.default_rng(T)
    flat = np.stack([g.permutation(P)[:k] for _ in range(T)]).reshape(-1)
    order = np.argsort(flat, kind="stable").astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=P))]).astype(np.int32)
    y = q.qmoe_gemm_f8(pool, P, q.qact_quantize_f8(to_dev(x)), T, to_dev(order), to_dev(off), N, K,
                       dtype=getattr(torch, dtype))
    yv = _np(y)
    for e in range(P):
        at = np.flatnonzero(flat == e)
        xs, ws = x[at // k].astype(np.float64), w[e].astype(np.float64)
        ref, s = xs @ ws.T, np.abs(xs) @ np.abs(ws).T
        fu.assert_close(yv[at], ref, _bound(ref, s, K, dtype), f"expert {e}")


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,N,K", [(70, 130, 1000), (300, 257, 640), (1500, 1490, 300), (2300, 4200, 520)])
def test_sums_of_wide_blocks(M, N, K, dtype):
    """Values over the whole range of the codes inside a block (w below 1, so that sums stay below 65504)."""
    q, torch = qg(), torch_cuda()
    g = np.random.default_rng([M, N, K])

    def wide(r, top):
        return (np.sign(g.normal(size=(r, K))) * np.exp2(top - g.uniform(0, 17.8, size=(r, K)))).astype(np.float32)

    W, xq = to_dev(q.qquantize_f8(wide(N, -2))), q.qact_quantize_f8(to_dev(wide(M, 8.8)))
    wv, xv = q.qdequant_f8(W, N, K).double(), q.qact_dequant_f8(xq, M, K).double()
    ref, s = _np(xv @ wv.t().contiguous()), _np(xv.abs() @ wv.abs().t().contiguous())
    y = q.qgemm_f8(W, xq, M, N, K, dtype=getattr(torch, dtype))
    fu.assert_close(_np(y), ref, _bound(ref, s, K, dtype), f"{M}x{N}x{K} {dtype}")
