"""f8 operators at the ends of the range: the largest finite values, blocks of
the smallest scales, extreme scales with 16-bit outputs."""
import numpy as np
import pytest

import f8_util as fu
from gpu_util import qg, to_dev, torch_cuda
from test_f8_range_host import FAR, MOST, capped

pytestmark = pytest.mark.gpu


def _np(t):
    torch_cuda().cuda.synchronize()
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_finite_activations_stay_finite(dtype):
    q, torch = qg(), torch_cuda()
    x = np.ones((6, 300), np.float32)
    x[0, :len(FAR)] = x[1, 120:120 + len(FAR)] = FAR
    x[2] = np.finfo(np.float32).max
    x[3, 299] = -3.38e38
    x[4, :2] = [3.38e38, np.inf]                 # beside what is not finite
    x[5, :2] = [np.nan, -3.38e38]
    xd = to_dev(x)
    if dtype == "bfloat16":                      # its largest finite value is 255 * 2^120
        xd = torch.where(torch.isfinite(xd), xd.clamp(-255.0 * 2.0 ** 120, 255.0 * 2.0 ** 120), xd).to(torch.bfloat16)
    xv = _np(xd)
    xq = q.qact_quantize_f8(xd)
    torch.cuda.synchronize()
    got = fu.unpack_acts(xq.cpu().numpy(), 6, 300)
    ok = np.isfinite(xv)
    want = np.concatenate([np.stack([capped(np.where(ok, xv, 0)[m, c:c + 128]) for m in range(6)])
                           for c in (0, 128, 256)], axis=1)
    assert np.array_equal(got[ok], want[ok]) and np.isnan(got[~ok]).all()
    for out in (torch.float32, torch.bfloat16):
        back = _np(q.qact_dequant_f8(xq, 6, 300, dtype=out))
        assert np.isfinite(back[ok]).all() and np.array_equal(back[ok], want[ok])
    # the same values inside the one-launch product: against 2^-110 they come back as they are held
    w = np.zeros((300, 300), np.float32)
    np.fill_diagonal(w, 2.0 ** -110)
    y = _np(q.qgemv_f8(to_dev(q.qquantize_f8(w)), xd[:4].contiguous(), 300, 300))
    assert np.array_equal(y, want[:4] * 2.0 ** -110)


def test_finite_weights_stay_finite_in_products():
    q = qg()
    N, K = 40, 130
    w = np.ones((N, K), np.float32)
    w[3, 5], w[30, 129] = np.finfo(np.float32).max, -3.35e38
    W = to_dev(q.qquantize_f8(w))
    wv = _np(q.qdequant_f8(W, N, K))
    assert wv[3, 5] == MOST and wv[30, 129] == -MOST
    for M in (3, 20, 80):
        x = np.zeros((M, K), np.float32)
        x[0, 5], x[1, 129] = 2.0 ** -100, 2.0 ** -100
        y = _np(q.qgemm_f8(W, q.qact_quantize_f8(to_dev(x)), M, N, K))
        assert np.array_equal(y, x.astype(np.float64) @ wv.T)


def _small(cols):
    """A block of the scale 2^-127: its codes stand for 2^-136 to 448 * 2^-127."""
    g = np.random.default_rng(cols)
    v = g.integers(1, 16, size=cols) * np.exp2(g.integers(-136, -122, size=cols).astype(np.float64))
    v[0] = 14 * 2.0 ** -122                       # 448 * 2^-127
    return v


@pytest.mark.parametrize("M", [2, 20, 80])
def test_blocks_of_the_smallest_scale(M):
    """Conversions are exact; a product's value is within 2^-133, half a step of bf16's subnormals or all of it."""
    q, torch = qg(), torch_cuda()
    N, K = 24, 128
    x = np.stack([np.roll(_small(K), m) for m in range(M)]).astype(np.float32)
    xr, e = fu.quantize_rows(x)
    assert (e == -127).all() and np.array_equal(xr.astype(np.float32), xr)
    xq = q.qact_quantize_f8(to_dev(x))
    assert np.array_equal(_np(q.qact_dequant_f8(xq, M, K)), xr)
    g = np.random.default_rng(M)
    w = (g.integers(-4, 5, size=(N, K)) * 2.0 ** 100).astype(np.float32)
    ref, off = xr @ w.T.astype(np.float64), 2.0 ** -133 * np.abs(w).sum(1)[None].astype(np.float64)
    bound = fu.sum_bound(np.abs(xr) @ np.abs(w).T + off, K) + off
    W = to_dev(q.qquantize_f8(w))
    fu.assert_close(_np(q.qgemm_f8(W, xq, M, N, K)), ref, bound, "gemm")
    if M <= 8:
        fu.assert_close(_np(q.qgemv_f8(W, to_dev(x), N, K)), ref, bound, "gemv")
    dy = to_dev(w[:M] if M <= N else np.tile(w, (M // N + 1, 1))[:M]).to(torch.bfloat16)   # [M][K], whole numbers
    dyv = _np(dy)
    off = 2.0 ** -133 * np.abs(dyv).sum(0)[:, None]
    fu.assert_close(_np(q.qgemm_f8_wgrad(dy, xq, M, K, K)), dyv.T @ xr,
                    fu.sum_bound(np.abs(dyv).T @ np.abs(xr) + off, M) + off, "weight gradient")
    # and as weights
    ws = np.stack([np.roll(_small(K), n) for n in range(N)]).astype(np.float32)
    wr, _ = fu.quantize_weights(ws)
    a = (g.integers(-4, 5, size=(M, K)) * 2.0 ** 100).astype(np.float32)
    off = 2.0 ** -133 * np.abs(a).sum(1)[:, None].astype(np.float64)
    Ws = to_dev(q.qquantize_f8(ws))
    assert np.array_equal(_np(q.qdequant_f8(Ws, N, K)), wr)
    fu.assert_close(_np(q.qgemm_f8(Ws, q.qact_quantize_f8(to_dev(a)), M, N, K)), a.astype(np.float64) @ wr.T,
                    fu.sum_bound(np.abs(a) @ np.abs(wr).T + off, K) + off, "weights")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("M", [2, 20, 80, 300])
def test_extreme_scales_with_16_bit_outputs(M, dtype):
    q, torch = qg(), torch_cuda()
    for ws, xs in ((2.0 ** 110, 2.0 ** -110), (2.0 ** -118, 2.0 ** 118), (2.0 ** 110, 2.0 ** -122), (2.0 ** -60, 2.0 ** 50)):
        N, K = 40, 256
        g = np.random.default_rng(5)
        w = (g.integers(-8, 9, size=(N, K)) * ws).astype(np.float32)
        x = (g.integers(-8, 9, size=(M, K)) * xs).astype(np.float32)
        ref = x.astype(np.float64) @ w.T.astype(np.float64)           # whole numbers: exact in fp32, then one rounding
        y = _np(q.qgemm_f8(to_dev(q.qquantize_f8(w)), q.qact_quantize_f8(to_dev(x)), M, N, K, dtype=getattr(torch, dtype)))
        fu.assert_close(y, ref, fu.HALF_STEP[dtype] * np.abs(ref) + fu.TINY[dtype], f"{ws} {xs}")
