"""GPU parity of the f8 operators against the binary64 references of f8_util:
conversions bit for bit, products within the stated bounds."""
import numpy as np
import pytest

import f8_util as fu
from gpu_util import qg, to_dev, torch_cuda

pytestmark = pytest.mark.gpu


def _dtype(name):
    return getattr(torch_cuda(), name)


def _x(x, name):
    """x on the device in a type, and the values that type holds in fp64."""
    t = to_dev(x.astype(np.float32)).to(_dtype(name))
    return t, t.double().cpu().numpy()


def _np(t):
    torch_cuda().cuda.synchronize()
    return t.double().cpu().numpy()


# -------------------------------------------------------------- conversions
@pytest.mark.parametrize("dtype", fu.TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (2, 129), (17, 640), (65, 1000), (5, 4096), (300, 257)])
def test_act_quantize(M, K, dtype):
    q = qg()
    x = fu.acts(M, K, seed=2)
    if K >= 128:
        x[0, :128] = 0.0                                                      # a zero block
        x[0, 0] = 0.0
        x[-1, :16] = 2.0 ** -9 * (np.arange(16) - 7.5)                        # ties of the subnormal codes
        x[-1, 16:32] = (16 + np.arange(16)) / 2.0 + 0.25                      # ties of normal ones
        x[-1, 127] = 448.0
    xd, xv = _x(x, dtype)
    xq = q.qact_quantize_f8(xd)
    ref, _ = fu.quantize_rows(xv)
    torch_cuda().cuda.synchronize()
    assert np.array_equal(fu.unpack_acts(xq.cpu().numpy(), M, K), ref)
    for out in fu.TYPES:
        back = q.qact_dequant_f8(xq, M, K, dtype=_dtype(out))
        want = torch_cuda().from_numpy(ref).to(_dtype(out)) if out != "float32" else torch_cuda().from_numpy(ref).float()
        assert torch_cuda().equal(back.cpu(), want), out


def test_act_quantize_ranges_and_strides():
    q, torch = qg(), torch_cuda()
    x = np.zeros((8, 130), np.float32)
    x[0, :3] = [3.0e38, -1.0e30, 1.0]
    x[1, :3] = [1e-45, -3e-45, 0.0]            # fp32 subnormals: the smallest scale
    x[2, :2] = [2.0 ** -118, -2.0 ** -127]
    x[3] = -0.0
    x[4, :2] = [448.0, 449.0]
    x[5, :130] = np.linspace(-1, 1, 130)
    xq = q.qact_quantize_f8(to_dev(x))
    torch.cuda.synchronize()
    ref, _ = fu.quantize_rows(x)
    assert np.array_equal(fu.unpack_acts(xq.cpu().numpy(), 8, 130), ref)
    assert np.array_equal(_np(q.qact_dequant_f8(xq, 8, 130)), ref)
    # rows of a wider buffer, at every alignment of an element
    wide = torch.randn(9, 401, device="cuda")
    for dtype in fu.TYPES:
        w = wide.to(_dtype(dtype))
        for off, K in ((0, 300), (1, 300), (3, 257), (7, 128)):
            v = w[:, off:off + K]
            a, b = q.qact_quantize_f8(v), q.qact_quantize_f8(v.contiguous())
            assert np.array_equal(fu.unpack_acts(a.cpu().numpy(), 9, K), fu.unpack_acts(b.cpu().numpy(), 9, K))
            assert np.array_equal(fu.unpack_acts(a.cpu().numpy(), 9, K), fu.quantize_rows(v.double().cpu().numpy())[0])


def test_act_quantize_non_finite_stays_in_its_place():
    q, torch = qg(), torch_cuda()
    x = fu.acts(4, 300, seed=5)
    ref, _ = fu.quantize_rows(x)
    y = x.copy()
    y[1, 7], y[2, 150], y[2, 299] = np.nan, np.inf, -np.inf
    y[1, 8] = x[1, 8]
    got = fu.unpack_acts(q.qact_quantize_f8(to_dev(y)).cpu().numpy(), 4, 300)
    bad = np.zeros((4, 300), bool)
    bad[1, 7] = bad[2, 150] = bad[2, 299] = True
    assert np.isnan(got[bad]).all()
    want, _ = fu.quantize_rows(np.where(bad, 0, y))
    assert np.array_equal(got[~bad], want[~bad])
    assert np.array_equal(got[[0, 3]], ref[[0, 3]])


@pytest.mark.parametrize("N,K", [(1, 1), (15, 130), (16, 128), (129, 257), (300, 1000)])
def test_weights_dequant_and_transpose(N, K):
    q, torch = qg(), torch_cuda()
    w = fu.weights(N, K, seed=3)
    packed = q.qquantize_f8(w)
    ref, _ = fu.quantize_weights(w)
    W = to_dev(packed)
    assert np.array_equal(_np(q.qdequant_f8(W, N, K)), ref)
    half = q.qdequant_f8(W, N, K, fp16=True)
    assert torch.equal(half.cpu(), torch.from_numpy(ref).to(torch.float16))
    nt = q.qpacked_bytes_f8(K, N)
    out = torch.full((nt + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    WT = q.qtranspose_f8(W, N, K, out=out[:nt])
    torch.cuda.synchronize()
    got, clean = fu.unpack_weights(WT.cpu().numpy(), K, N)
    assert clean and np.array_equal(got, ref.T)
    assert (out[nt:] == 0x5A).all()
    again = q.qtranspose_f8(WT, K, N)
    assert np.array_equal(again.cpu().numpy(), packed)


# ----------------------------------------------------------------- products
GEMV = [(1, 1, 1), (1, 16, 128), (2, 17, 129), (3, 300, 1000), (4, 33, 5000), (8, 130, 257), (5, 2048, 640),
        (1, 4096, 4096), (7, 100, 16384)]


@pytest.mark.parametrize("dtype", fu.TYPES)
@pytest.mark.parametrize("M,N,K", GEMV)
def test_gemv(M, N, K, dtype):
    q = qg()
    W, wv = to_dev(q.qquantize_f8(fu.weights(N, K, seed=4))), fu.quantize_weights(fu.weights(N, K, seed=4))[0]
    xd, xv = _x(fu.acts(M, K, seed=5), dtype)
    xr, _ = fu.quantize_rows(xv)
    y = _np(q.qgemv_f8(W, xd, N, K))
    fu.assert_close(y, xr @ wv.T, fu.sum_bound(np.abs(xr) @ np.abs(wv).T, K), f"gemv {M}x{N}x{K}")


GEMM = [(1, 1, 1), (1, 130, 257), (16, 128, 128), (17, 100, 640), (33, 300, 1500), (64, 48, 3000), (65, 127, 129),
        (100, 500, 1000), (129, 257, 385), (255, 300, 2000), (300, 64, 128), (1000, 200, 520), (1, 2000, 9000)]


@pytest.mark.parametrize("dtype", fu.TYPES)
@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm(M, N, K, dtype):
    q, torch = qg(), torch_cuda()
    w = fu.weights(N, K, seed=6)
    W, wv = to_dev(q.qquantize_f8(w)), fu.quantize_weights(w)[0]
    x = fu.acts(M, K, seed=7)
    xr, _ = fu.quantize_rows(x)
    xq = q.qact_quantize_f8(to_dev(x))
    buf = torch.full((M * N + 8,), 7.0, dtype=_dtype(dtype), device="cuda")
    y = q.qgemm_f8(W, xq, M, N, K, Y=buf[:M * N].view(M, N))
    ref, s = xr @ wv.T, np.abs(xr) @ np.abs(wv).T
    fu.assert_close(_np(y), ref, fu.product_bound(ref, s, K, dtype), f"gemm {M}x{N}x{K} {dtype}")
    assert (buf[M * N:] == 7.0).all()
    # an output that no vector store can take, and the same call again: the same bits
    off = torch.empty(M * N + 1, dtype=_dtype(dtype), device="cuda")[1:].view(M, N)
    assert torch.equal(q.qgemm_f8(W, xq, M, N, K, Y=off), y)


@pytest.mark.parametrize("M,N,K", [(2100, 4200, 384), (4100, 2050, 200), (8, 28672, 512)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gemm_large(M, N, K, dtype):
    """Tiles beyond one a CU; the reference is the fp64 product of the packed values, on the device."""
    q, torch = qg(), torch_cuda()
    w, x = fu.weights(N, K, seed=8), fu.acts(M, K, seed=9)
    W, xq = to_dev(q.qquantize_f8(w)), q.qact_quantize_f8(to_dev(x))
    wv = to_dev(fu.quantize_weights(w)[0])
    xr = to_dev(fu.quantize_rows(x)[0])
    ref, s = _np(xr @ wv.T.contiguous()), _np(xr.abs() @ wv.abs().T.contiguous())
    y = q.qgemm_f8(W, xq, M, N, K, dtype=_dtype(dtype))
    fu.assert_close(_np(y), ref, fu.product_bound(ref, s, K, dtype), f"gemm {M}x{N}x{K} {dtype}")


def test_products_of_whole_numbers_are_exact():
    """Small whole numbers: every product and sum is exact in any order, in fp32 and in bf16 outputs up to 256."""
    q, torch = qg(), torch_cuda()
    g = np.random.default_rng(3)
    for M, N, K in ((3, 40, 300), (40, 40, 300), (200, 300, 700), (70, 4000, 130)):
        w = g.integers(-1, 2, size=(N, K)).astype(np.float32)
        x = g.integers(-2, 3, size=(M, K)).astype(np.float32) * (g.random((M, K)) < 0.1)
        W, xq = to_dev(q.qquantize_f8(w)), q.qact_quantize_f8(to_dev(x))
        ref = x.astype(np.float64) @ w.T.astype(np.float64)
        for dtype in fu.TYPES:
            y = _np(q.qgemm_f8(W, xq, M, N, K, dtype=_dtype(dtype)))
            assert np.array_equal(y, ref), (M, N, K, dtype)


def test_one_hot_activations_return_weight_columns():
    q, torch = qg(), torch_cuda()
    N, K = 200, 300
    w = fu.weights(N, K, seed=10)
    W, wv = to_dev(q.qquantize_f8(w)), fu.quantize_weights(w)[0]
    x = np.eye(K, dtype=np.float32)[::-1].copy()
    y = _np(q.qgemm_f8(W, q.qact_quantize_f8(to_dev(x)), K, N, K))
    assert np.array_equal(y, wv.T[::-1])
    y = _np(q.qgemv_f8(W, to_dev(x[:8]), N, K))
    assert np.array_equal(y, wv.T[::-1][:8])


def test_non_finite_rows_stay_in_their_rows():
    q, torch = qg(), torch_cuda()
    for M, dtype in ((3, "float32"), (70, "bfloat16"), (70, "float32"), (30, "float16")):
        N, K = 150, 300
        w, x = fu.weights(N, K, seed=12), fu.acts(M, K, seed=13)
        W = to_dev(q.qquantize_f8(w))
        clean = q.qgemm_f8(W, q.qact_quantize_f8(to_dev(x)), M, N, K, dtype=_dtype(dtype))
        x[1, 5], x[2, 299] = np.nan, np.inf
        y = q.qgemm_f8(W, q.qact_quantize_f8(to_dev(x)), M, N, K, dtype=_dtype(dtype))
        rest = [m for m in range(M) if m not in (1, 2)]
        assert torch.isnan(y[[1, 2]]).all()
        assert torch.equal(y[rest], clean[rest])


def test_extreme_scales():
    """The largest and the smallest scales the quantizers write, against each other."""
    q = qg()
    for ws, xs in ((2.0 ** 110, 2.0 ** -110), (2.0 ** -118, 2.0 ** 118), (2.0 ** -60, 2.0 ** -60), (2.0 ** 50, 2.0 ** 50)):
        for M in (2, 80):
            N, K = 40, 256
            g = np.random.default_rng(5)
            w = (g.integers(-8, 9, size=(N, K)) * ws).astype(np.float32)
            x = (g.integers(-8, 9, size=(M, K)) * xs).astype(np.float32)
            ref = x.astype(np.float64) @ w.T.astype(np.float64)
            y = _np(q.qgemm_f8(to_dev(q.qquantize_f8(w)), q.qact_quantize_f8(to_dev(x)), M, N, K))
            assert np.array_equal(y, ref), (ws, xs, M)


# ----------------------------------------------------------------- backward
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (63, 8, 128), (64, 128, 128), (65, 129, 127), (200, 136, 300),
                                   (515, 40, 257), (1300, 130, 129), (4000, 64, 128), (2048, 256, 384)])
def test_wgrad(M, N, K):
    q, torch = qg(), torch_cuda()
    x = fu.acts(M, K, seed=14)
    xr, _ = fu.quantize_rows(x)
    dy, dyv = _x(fu.acts(M, N, seed=15) * 1e-3, "bfloat16")
    xq = q.qact_quantize_f8(to_dev(x))
    dw = q.qgemm_f8_wgrad(dy, xq, M, N, K)
    ref, s = dyv.T @ xr, np.abs(dyv).T @ np.abs(xr)
    b = fu.sum_bound(s, M)
    fu.assert_close(_np(dw), ref, b, f"wgrad {M}x{N}x{K}")
    assert torch.equal(q.qgemm_f8_wgrad(dy, xq, M, N, K), dw)          # the same bits again
    g = np.random.default_rng(2).normal(size=(N, K)).astype(np.float32)
    buf = torch.full((N * K + 4,), 3.0, device="cuda")
    acc = buf[:N * K].view(N, K)
    acc.copy_(to_dev(g))
    q.qgemm_f8_wgrad(dy, xq, M, N, K, dW=acc, accumulate=True)
    fu.assert_close(_np(acc), ref + g, b + 2.0 ** -23 * (np.abs(ref) + np.abs(g) + b), "wgrad accumulate")
    assert (buf[N * K:] == 3.0).all()


def test_wgrad_non_finite_gradient_reaches_its_row_only():
    q, torch = qg(), torch_cuda()
    M, N, K = 70, 64, 128
    xq = q.qact_quantize_f8(to_dev(fu.acts(M, K, seed=1)))
    dy = to_dev(fu.acts(M, N, seed=2)).bfloat16()
    clean = q.qgemm_f8_wgrad(dy, xq, M, N, K)
    dy[M - 1, 3] = float("inf")
    dw = q.qgemm_f8_wgrad(dy, xq, M, N, K)
    assert not torch.isfinite(dw[3]).any()
    keep = [n for n in range(N) if n != 3]
    assert torch.equal(dw[keep], clean[keep])


def test_gradients_against_differences():
    """dx and dw of L = sum G * (X W^T) on values that f8 holds exactly, against central differences of the
    product itself: L is linear in each element, so they are exact up to the roundings counted below."""
    q, torch = qg(), torch_cuda()
    g = np.random.default_rng(8)
    M, N, K = 66, 40, 130
    w = g.integers(-4, 5, size=(N, K)).astype(np.float32)
    x = g.integers(-4, 5, size=(M, K)).astype(np.float32)
    G = g.integers(-2, 3, size=(M, N)).astype(np.float32)

    def loss(x, w):
        y = q.qgemm_f8(to_dev(q.qquantize_f8(w)), q.qact_quantize_f8(to_dev(x)), M, N, K)
        return float((_np(y) * G).sum())

    W = to_dev(q.qquantize_f8(w))
    gd = to_dev(G).bfloat16()
    xq = q.qact_quantize_f8(to_dev(x))
    dx = _np(q.qgemm_f8(q.qtranspose_f8(W, N, K), q.qact_quantize_f8(gd), M, K, N))
    dw = _np(q.qgemm_f8_wgrad(gd, xq, M, N, K))
    for m, k in ((0, 0), (65, 129), (30, 127), (5, 128)):
        d = np.zeros_like(x)
        d[m, k] = 1.0
        assert dx[m, k] == (loss(x + d, w) - loss(x - d, w)) / 2          # whole numbers: no rounding at all
    for n, k in ((0, 0), (39, 129), (17, 127), (8, 128)):
        d = np.zeros_like(w)
        d[n, k] = 1.0
        assert dw[n, k] == (loss(x, w + d) - loss(x, w - d)) / 2


# ------------------------------------------------------------------ experts
def _slots(P, T, k, seed, drop=0.1, only=None):
    """idx [T][k] of different experts (-1: dropped), order, offsets."""
    g = np.random.default_rng([P, T, k, seed])
    pool = np.arange(P) if only is None else np.asarray(only)
    idx = np.stack([g.permutation(pool)[:k] for _ in range(T)])
    idx[g.random((T, k)) < drop] = -1
    flat = idx.reshape(-1)
    key = np.where(flat >= 0, flat, P)
    order = np.argsort(key, kind="stable").astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=P + 1)[:P])]).astype(np.int32)
    return flat, order, off


def _pool(P, N, K, seed):
    q = qg()
    ws = [fu.weights(N, K, seed=seed + e) for e in range(P)]
    return np.concatenate([q.qquantize_f8(w) for w in ws]), [fu.quantize_weights(w)[0] for w in ws]


MOE = [(1, 1, 1, 16, 128, None), (4, 3, 2, 33, 300, None), (16, 5, 4, 100, 257, None), (3, 200, 2, 130, 129, None),
       (8, 700, 3, 64, 256, (1, 2, 5)), (130, 9, 2, 20, 130, None), (5, 257, 1, 257, 384, (4,)), (2, 40, 1, 48, 1000, None)]


@pytest.mark.parametrize("dtype", fu.TYPES)
@pytest.mark.parametrize("P,T,k,N,K,only", MOE)
def test_moe_gemm(P, T, k, N, K, only, dtype):
    q, torch = qg(), torch_cuda()
    pool, wv = _pool(P, N, K, seed=20)
    flat, order, off = _slots(P, T, k, seed=1, only=only)
    x = fu.acts(T, K, seed=21)
    xr, _ = fu.quantize_rows(x)
    xq = q.qact_quantize_f8(to_dev(x))
    S = T * k
    ref, s = np.zeros((S, N)), np.zeros((S, N))
    for i, e in enumerate(flat):
        if e >= 0:
            ref[i], s[i] = wv[e] @ xr[i // k], np.abs(wv[e]) @ np.abs(xr[i // k])
    buf = torch.full((S * N + 8,), 7.0, dtype=_dtype(dtype), device="cuda")
    y = q.qmoe_gemm_f8(to_dev(pool), P, xq, T, to_dev(order), to_dev(off), N, K, Y=buf[:S * N].view(S, N))
    bound = np.where((flat >= 0)[:, None], fu.product_bound(ref, s, K, dtype), 0.0)      # dropped slots: zeros
    fu.assert_close(_np(y), ref, bound, f"moe {P} {T}x{k} {N}x{K} {dtype}")
    assert (buf[S * N:] == 7.0).all()


def test_moe_gemm_holds_bad_slots_to_its_buffers():
    """Entries of order and offsets out of range: nothing outside Y is written, the other rows stay right."""
    q, torch = qg(), torch_cuda()
    for P, T in ((4, 6), (2, 90)):
        N, K = 40, 200
        pool, wv = _pool(P, N, K, seed=30)
        flat, order, off = _slots(P, T, 1, seed=3, drop=0.0)
        xq = q.qact_quantize_f8(to_dev(fu.acts(T, K, seed=31)))
        good = q.qmoe_gemm_f8(to_dev(pool), P, xq, T, to_dev(order), to_dev(off), N, K)
        bad = order.copy()
        gone = [int(bad[0]), int(bad[-1])]
        bad[0], bad[-1] = -5, 2 ** 31 - 1
        off2 = off.copy()
        off2[0], off2[-1] = -7, 2 ** 31 - 1
        buf = torch.full(((T + 4) * N,), 7.0, device="cuda")
        y = q.qmoe_gemm_f8(to_dev(pool), P, xq, T, to_dev(bad), to_dev(off2), N, K, Y=buf[2 * N:(T + 2) * N].view(T, N))
        torch.cuda.synchronize()
        keep = [t for t in range(T) if t not in gone]
        assert torch.equal(y[keep], good[keep])
        assert (y[gone] == 7.0).all() and (buf[:2 * N] == 7.0).all() and (buf[(T + 2) * N:] == 7.0).all()


@pytest.mark.parametrize("P,T,k,N,K,only", [(1, 1, 1, 8, 128, None), (4, 33, 2, 40, 129, None),
                                            (3, 300, 2, 136, 257, None), (6, 64, 1, 33, 64, (0, 5))])
def test_moe_wgrad(P, T, k, N, K, only):
    q, torch = qg(), torch_cuda()
    flat, order, off = _slots(P, T, k, seed=4, only=only)
    x = fu.acts(T, K, seed=40)
    xr, _ = fu.quantize_rows(x)
    xq = q.qact_quantize_f8(to_dev(x))
    dy, dyv = _x(fu.acts(T * k, N, seed=41), "bfloat16")
    dw = q.qmoe_gemm_f8_wgrad(dy, xq, T, to_dev(order), to_dev(off), P, N, K)
    ref, s = np.zeros((P, N, K)), np.zeros((P, N, K))
    for e in range(P):
        at = np.flatnonzero(flat == e)
        ref[e], s[e] = dyv[at].T @ xr[at // k], np.abs(dyv[at]).T @ np.abs(xr[at // k])
    fu.assert_close(_np(dw), ref, fu.sum_bound(s, T), "moe wgrad")
    base = torch.randn(P, N, K, device="cuda")
    acc = q.qmoe_gemm_f8_wgrad(dy, xq, T, to_dev(order), to_dev(off), P, N, K, dW=base.clone(), accumulate=True)
    b0 = _np(base)
    b = fu.sum_bound(s, T)
    fu.assert_close(_np(acc), ref + b0, b + 2.0 ** -23 * (np.abs(ref) + np.abs(b0) + b), "moe wgrad accumulate")


# ------------------------------------------------------------------ binding
def test_binding_checks():
    q, torch = qg(), torch_cuda()
    W = to_dev(q.qquantize_f8(fu.weights(32, 256, seed=1)))
    x = torch.randn(4, 256, device="cuda")
    xq = q.qact_quantize_f8(x)
    for call in (lambda: q.qgemv_f8(W, x[:, :128], 32, 256), lambda: q.qgemv_f8(W[:100], x, 32, 256),
                 lambda: q.qgemm_f8(W, xq[:300], 4, 32, 256), lambda: q.qgemm_f8(W, xq, 4, 32, 256, Y=torch.empty(4, 31, device="cuda")),
                 lambda: q.qgemv_f8(W, x.t().contiguous().t(), 32, 256), lambda: q.qact_quantize_f8(x.t()),
                 lambda: q.qgemm_f8_wgrad(torch.zeros(4, 32, device="cuda", dtype=torch.bfloat16), xq, 4, 32, 256, accumulate=True),
                 lambda: q.qmoe_gemm_f8(W, 1, xq, 4, torch.zeros(7, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), 32, 256)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: q.qact_quantize_f8(x.double()), lambda: q.qgemm_f8(W, x, 4, 32, 256),
                 lambda: q.qgemm_f8(W, xq.cpu(), 4, 32, 256), lambda: q.qgemm_f8(W, xq, 4, 32, 256, dtype=torch.float64),
                 lambda: q.qgemm_f8_wgrad(torch.zeros(4, 32, device="cuda"), xq, 4, 32, 256)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: q.qgemv_f8(W, torch.zeros(9, 256, device="cuda"), 32, 256),
                 lambda: q.qact_quantize_f8(torch.zeros(0, 256, device="cuda")),
                 lambda: q.qact_quantize_f8(torch.zeros(1, 256, device="cuda").expand(4, 256)),
                 lambda: q.qgemm_f8(W, xq, 0, 32, 256)):
        with pytest.raises(q.QGError) as e:
            call()
        assert e.value.status == 2
