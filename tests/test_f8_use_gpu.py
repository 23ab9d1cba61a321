"""The f8 operators and the routing as programs use them: a layer of experts
forward and backward, captured graphs, other streams, several calls at once,
buffers beyond 32-bit offsets."""
import numpy as np
import pytest

import f8_util as fu
from gpu_util import qg, to_dev, torch_cuda

pytestmark = pytest.mark.gpu


def _np(t):
    torch_cuda().cuda.synchronize()
    return t.double().cpu().numpy()


def _pool(P, N, K, seed):
    q = qg()
    return np.concatenate([q.qquantize_f8(fu.weights(N, K, seed=seed + e)) for e in range(P)])


def _pool_values(pool, P, N, K):
    return [fu.unpack_weights(p, N, K)[0] for p in pool.reshape(P, -1)]


# ------------------------------------------------------- a layer of experts
@pytest.mark.parametrize("T,E,k,H,D", [(1, 4, 2, 128, 96), (37, 6, 2, 130, 257), (300, 5, 3, 256, 128)])
def test_layer_of_experts_forward_and_backward(T, E, k, H, D):
    """route -> quantize -> first product -> |.|^2 shape -> quantize -> second
    product -> weighted sum, and back: each step against its definition in
    binary64 on the inputs that the step had."""
    q, torch = qg(), torch_cuda()
    g = np.random.default_rng([T, E, 3])
    x = to_dev(fu.acts(T, D, seed=1)).to(torch.bfloat16)
    logits = to_dev(g.normal(size=(T, E)).astype(np.float32))
    mask = g.random(T) >= 0.2
    mask[0] = True                                       # the others: a padded batch
    up, down = _pool(E, H, D, seed=5), _pool(E, D, H, seed=60)
    up_v, down_v = _pool_values(up, E, H, D), _pool_values(down, E, D, H)
    up_d, down_d = to_dev(up), to_dev(down)
    S = T * k

    r = q.qmoe_route(logits, k, mask=to_dev(mask))
    ref = fu.route(_np(logits), k, mask)
    torch.cuda.synchronize()
    for name in ("idx", "counts", "offsets", "order"):
        assert np.array_equal(getattr(r, name).cpu().numpy(), ref[name]), name
    flat = ref["idx"].reshape(-1)
    xq = q.qact_quantize_f8(x)
    xv = _np(q.qact_dequant_f8(xq, T, D))
    assert np.array_equal(xv, fu.quantize_rows(_np(x))[0])
    h = q.qmoe_gemm_f8(up_d, E, xq, T, r.order, r.offsets, H, D)
    a = (h * h.abs()).to(torch.bfloat16)
    aq = q.qact_quantize_f8(a)
    av = _np(q.qact_dequant_f8(aq, S, H))
    y = q.qmoe_gemm_f8(down_d, E, aq, S, r.order, r.offsets, D, H)      # a row of its own for each slot
    out = (y.view(T, k, D) * r.weight.unsqueeze(2)).sum(1)

    def products(vals, rows, per):
        n = vals[0].shape[0]
        want, size = np.zeros((S, n)), np.zeros((S, n))
        for s, e in enumerate(flat):
            if e >= 0:
                want[s], size[s] = vals[e] @ rows[s // per], np.abs(vals[e]) @ np.abs(rows[s // per])
        return want, size

    for got, vals, rows, per, K, what in ((h, up_v, xv, k, D, "up"), (y, down_v, av, 1, H, "down")):
        want, size = products(vals, rows, per)
        fu.assert_close(_np(got), want, np.where((flat >= 0)[:, None], fu.sum_bound(size, K), 0.0), what)
    assert (_np(out)[~mask] == 0).all()

    # backward of sum(out * go) + 0.01 loss, products' gradients straight through the quantization
    go = to_dev(fu.acts(T, D, seed=9))
    gw = (y.view(T, k, D) * go.unsqueeze(1)).sum(2)
    dy = (go.unsqueeze(1) * r.weight.unsqueeze(2)).view(S, D).to(torch.bfloat16)
    dyv = _np(dy)
    d_down = q.qmoe_gemm_f8_wgrad(dy, aq, S, r.order, r.offsets, E, D, H)
    down_t = torch.cat([q.qtranspose_f8(w, D, H) for w in down_d.view(E, -1)])
    up_t = torch.cat([q.qtranspose_f8(w, H, D) for w in up_d.view(E, -1)])
    dyq = q.qact_quantize_f8(dy)
    da = q.qmoe_gemm_f8(down_t, E, dyq, S, r.order, r.offsets, H, D)
    dh = (da * 2 * h.abs()).to(torch.bfloat16)
    dhv = _np(dh)
    d_up = q.qmoe_gemm_f8_wgrad(dh, xq, T, r.order, r.offsets, E, H, D)
    dhq = q.qact_quantize_f8(dh)
    dx = q.qmoe_gemm_f8(up_t, E, dhq, S, r.order, r.offsets, D, H)
    one = torch.full((1,), 0.01, device="cuda")
    dl = q.qmoe_route_backward(logits, r, grad_weight=gw, grad_loss=one, mask=to_dev(mask))

    dyqv, dhqv = _np(q.qact_dequant_f8(dyq, S, D)), _np(q.qact_dequant_f8(dhq, S, H))
    for got, vals, rows, K, what in ((da, down_v, dyqv, D, "da"), (dx, up_v, dhqv, H, "dx")):
        want, size = products([v.T for v in vals], rows, 1)
        fu.assert_close(_np(got), want, np.where((flat >= 0)[:, None], fu.sum_bound(size, K), 0.0), what)
    for got, grad, rows, per, what in ((d_down, dyv, av, 1, "d_down"), (d_up, dhv, xv, k, "d_up")):
        got = _np(got)
        for e in range(E):
            at = np.flatnonzero(flat == e)
            rr = rows[at // per]
            fu.assert_close(got[e], grad[at].T @ rr, fu.sum_bound(np.abs(grad[at]).T @ np.abs(rr), max(len(at), 1)),
                            f"{what} of expert {e}")
    gwv = _np(gw)
    want = fu.route_gradient(ref, gwv, float(np.float32(0.01)))
    # weights and p to 2^-18 (see the routing's own tests), sums of k and E of them with magnitudes up to the
    # largest gradient
    size = np.abs(gwv).max(1, keepdims=True) + 0.01 * E
    fu.assert_close(_np(dl), want, 2.0 ** -15 * size + 0 * want, "dlogits")
    assert (_np(dl)[~mask] == 0).all()


# ------------------------------------------------------------------- graphs
def _everything(q, torch, s):
    """One call of each entry point on the buffers of s; the results."""
    T, k, E, N, K, M = s["T"], s["k"], s["E"], s["N"], s["K"], s["M"]
    r = q.qmoe_route(s["logits"], k, mask=s["mask"])
    dl = q.qmoe_route_backward(s["logits"], r, grad_weight=s["gw"], grad_loss=s["gl"], mask=s["mask"])
    xq = q.qact_quantize_f8(s["x"])
    tq = q.qact_quantize_f8(s["xt"])
    return [*r, dl, q.qact_dequant_f8(xq, M, K), q.qdequant_f8(s["W"], N, K), q.qtranspose_f8(s["W"], N, K),
            q.qgemv_f8(s["W"], s["x"][:5], N, K),
            q.qgemm_f8(s["W"], xq, M, N, K), q.qgemm_f8(s["W"], xq, M, N, K, dtype=torch.bfloat16),
            q.qgemm_f8_wgrad(s["dy"], xq, M, N, K),
            q.qmoe_gemm_f8(s["pool"], E, tq, T, r.order, r.offsets, N, K),
            q.qmoe_gemm_f8_wgrad(s["dyt"], tq, T, r.order, r.offsets, E, N, K)]


def _state(torch, M, T, seed):
    E, k, N, K = 6, 2, 136, 264
    dev = dict(device="cuda")
    s = dict(M=M, T=T, E=E, k=k, N=N, K=K,
             W=to_dev(qg().qquantize_f8(fu.weights(N, K, seed=seed))), pool=to_dev(_pool(E, N, K, seed=seed + 1)),
             logits=torch.empty(T, E, **dev), mask=torch.empty(T, dtype=torch.uint8, **dev),
             gw=torch.empty(T, k, **dev), gl=torch.empty(1, **dev),
             x=torch.empty(M, K, dtype=torch.bfloat16, **dev), xt=torch.empty(T, K, dtype=torch.float16, **dev),
             dy=torch.empty(M, N, dtype=torch.bfloat16, **dev), dyt=torch.empty(T * k, N, dtype=torch.bfloat16, **dev))
    return s


def _fill(torch, s, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for name in ("logits", "gw", "gl", "x", "xt", "dy", "dyt"):
        s[name].copy_(torch.randn(s[name].shape, generator=g, device="cuda"))
    s["mask"].copy_(torch.rand(s["mask"].shape, generator=g, device="cuda") > 0.1)


@pytest.mark.parametrize("M,T", [(9, 30), (40, 200), (2100, 700)])
def test_captured_graphs(M, T):
    """Two graphs of every entry point, replayed in turn on new inputs with eager calls between."""
    q, torch = qg(), torch_cuda()
    states = [_state(torch, M, T, seed=70), _state(torch, M, T, seed=90)]
    for i, s in enumerate(states):
        _fill(torch, s, i)
        _everything(q, torch, s)          # first calls outside of the capture
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_everything(q, torch, s))
        graphs.append(g)
    for turn in range(4):
        for i in (0, 1) if turn % 2 else (1, 0):
            _fill(torch, states[i], 10 * turn + i)
            graphs[i].replay()
            want = _everything(q, torch, states[i])
            torch.cuda.synchronize()
            for n, (a, b) in enumerate(zip(outs[i], want)):
                assert torch.equal(a, b), (turn, i, n)


def test_two_streams_at_once():
    q, torch = qg(), torch_cuda()
    states = [_state(torch, 2100, 700, seed=70), _state(torch, 33, 65, seed=90)]
    want = []
    for i, s in enumerate(states):
        _fill(torch, s, 5 + i)
        want.append(_everything(q, torch, s))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(states):
            with torch.cuda.stream(streams[i]):
                got[i].append(_everything(q, torch, s))
    torch.cuda.synchronize()
    for i in range(2):
        for rep in got[i]:
            for n, (a, b) in enumerate(zip(rep, want[i])):
                assert torch.equal(a, b), (i, n)


def test_calls_follow_the_current_stream():
    """Work queued before a call on the stream that is current is seen by it."""
    q, torch = qg(), torch_cuda()
    s = _state(torch, 300, 128, seed=70)
    _fill(torch, s, 1)
    first = _everything(q, torch, s)
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for _ in range(8):
            big = big @ big * 1e-3         # keeps the stream busy
        _fill(torch, s, 2)
        got = _everything(q, torch, s)
    torch.cuda.synchronize()
    want = _everything(q, torch, s)
    torch.cuda.synchronize()
    assert not torch.equal(got[0], first[0])
    for n, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), n


# ------------------------------------------------------------ weight gradient
@pytest.mark.parametrize("M,N,K", [(2500, 130, 129), (3100, 257, 131), (2048, 136, 132), (5000, 8, 1)])
def test_wgrad_in_parts(M, N, K):
    """Few tiles of many rows: parts in the workspace, joined; odd sizes on both sides, on top of dW too."""
    q, torch = qg(), torch_cuda()
    assert int(q.lib().qgemm_f8_wgrad_workspace(M, N, K)) > 0
    x = fu.acts(M, K, seed=14)
    xr, _ = fu.quantize_rows(x)
    dy = to_dev(fu.acts(M, N, seed=15)).to(torch.bfloat16)
    dyv = _np(dy)
    xq = q.qact_quantize_f8(to_dev(x))
    ref, b = dyv.T @ xr, fu.sum_bound(np.abs(dyv).T @ np.abs(xr), M)
    buf = torch.full((N * K + 7,), 3.0, device="cuda")
    for lead in (0, 1):                    # a dW that starts inside a vector, too
        dw = buf[lead:lead + N * K].view(N, K)
        dw.copy_(to_dev(np.arange(N * K, dtype=np.float32).reshape(N, K) % 64))
        base = _np(dw)
        q.qgemm_f8_wgrad(dy, xq, M, N, K, dW=dw, accumulate=True)
        fu.assert_close(_np(dw), ref + base, b + 2.0 ** -23 * (np.abs(ref) + np.abs(base) + b), "accumulate")
        q.qgemm_f8_wgrad(dy, xq, M, N, K, dW=dw)
        fu.assert_close(_np(dw), ref, b, "whole")
        assert (buf[lead + N * K:] == 3.0).all() and (buf[:lead] == 3.0).all()
        buf.fill_(3.0)


@pytest.mark.parametrize("M", [1, 5, 33])
def test_wgrad_nan_in_the_first_value_stays_in_its_column(M):
    """The rows that fill up a step take nothing from the first byte of the activations (0xff: a negative NaN)."""
    q, torch = qg(), torch_cuda()
    N, K = 40, 128
    x = fu.acts(M, K, seed=3)
    x[0, 0] = -np.float32(np.nan)
    assert np.signbit(x[0, 0])
    xq = q.qact_quantize_f8(to_dev(x))
    torch.cuda.synchronize()
    dy = to_dev(fu.acts(M, N, seed=4)).to(torch.bfloat16)
    dyv = _np(dy)
    for first in (None, 0xFF):
        if first is not None:
            xq[0] = first                  # whatever the sign that the conversion gave it
        dw = _np(q.qgemm_f8_wgrad(dy, xq, M, N, K))
        assert np.isnan(dw[:, 0]).all()
        xr, _ = fu.quantize_rows(x)
        xr = xr[:, 1:]
        fu.assert_close(dw[:, 1:], dyv.T @ xr, fu.sum_bound(np.abs(dyv).T @ np.abs(xr), M), "the other columns")
    order, off = torch.arange(M, dtype=torch.int32, device="cuda"), torch.tensor([0, M], dtype=torch.int32, device="cuda")
    dw = _np(q.qmoe_gemm_f8_wgrad(dy, xq, M, order, off, 1, N, K))[0]
    assert np.isnan(dw[:, 0]).all()
    fu.assert_close(dw[:, 1:], dyv.T @ xr, fu.sum_bound(np.abs(dyv).T @ np.abs(xr), M), "the other columns, experts")


# ------------------------------------------------------- beyond 32-bit offsets
def test_far_rows_of_weights():
    """Packed weights of 8.6 GB: the last rows' outputs are those of the last rows alone, bit for bit."""
    q, torch = qg(), torch_cuda()
    N, K, last = (1 << 21) + 40, 4096, 168           # whole 128-row blocks of scales before the last rows
    nb = q.qpacked_bytes_f8(N, K)
    s0 = 2048 * (-(-N // 16)) * (K // 128)
    W = torch.empty(nb, dtype=torch.uint8, device="cuda")
    W.fill_(0x31)
    tail = torch.randint(0, 0x7F, (2048 * (-(-last // 16)) * (K // 128),), dtype=torch.uint8, device="cuda")
    W[s0 - tail.numel():s0] = tail
    W[s0:] = 120
    assert (N - last) % 128 == 0
    small = torch.zeros(q.qpacked_bytes_f8(last, K), dtype=torch.uint8, device="cuda")
    small[:tail.numel()] = tail
    small[tail.numel():tail.numel() + 2 * (K // 128)] = 120
    x = to_dev(fu.acts(70, K, seed=1)).to(torch.bfloat16)
    for M in (1, 8):
        a, b = q.qgemv_f8(W, x[:M], N, K), q.qgemv_f8(small, x[:M], last, K)
        assert torch.equal(a[:, N - last:], b), M
    for M in (12, 30, 64, 70):
        xq = q.qact_quantize_f8(x[:M])
        a, b = q.qgemm_f8(W, xq, M, N, K), q.qgemm_f8(small, xq, M, last, K)
        if M <= 32:
            assert torch.equal(a[:, N - last:], b), M
        else:
            # other kernels for other N, so another order of the sums: each result is within the stated bound of
            # the exact sum, and two of them within twice that of each other
            d = (a[:, N - last:] - b).abs().double()
            xv = q.qact_dequant_f8(xq, M, K).abs().double()
            size = xv @ q.qdequant_f8(small, last, K).abs().double().t().contiguous()
            assert (d <= 2 * fu.sum_bound(1.0, K) * size).all()
    del W
    torch.cuda.empty_cache()


def test_far_rows_of_activations():
    """Activations of 8.6 GB, their products and weight gradient: the last rows count like any others."""
    q, torch = qg(), torch_cuda()
    M, N, K = (1 << 21) + 77, 24, 4096
    w = fu.weights(N, K, seed=4)
    W = to_dev(q.qquantize_f8(w))
    wv = fu.quantize_weights(w)[0]
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    last = 200
    tail = to_dev(fu.acts(last, K, seed=8)).to(torch.bfloat16)
    x[M - last:] = tail
    xr, _ = fu.quantize_rows(_np(tail))
    xq = q.qact_quantize_f8(x)
    del x
    y = q.qgemm_f8(W, xq, M, N, K)
    assert (y[:M - last] == 0).all()
    ref, size = xr @ wv.T, np.abs(xr) @ np.abs(wv).T
    fu.assert_close(_np(y[M - last:]), ref, fu.product_bound(ref, size, K, "float32"), "last rows")
    dy = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    dy[M - last:] = to_dev(fu.acts(last, N, seed=3)).to(torch.bfloat16)
    dyv = _np(dy[M - last:])
    dw = q.qgemm_f8_wgrad(dy, xq, M, N, K)
    # the rows before are zeros: their products add nothing, and rounding starts with the last rows
    fu.assert_close(_np(dw), dyv.T @ xr, fu.sum_bound(np.abs(dyv).T @ np.abs(xr), last), "weight gradient")
    back = q.qact_dequant_f8(xq, M, K, dtype=torch.bfloat16)
    assert np.array_equal(_np(back[M - last:]), xr)
    assert not back[:M - last].any()
    del back, xq, dy, y
    torch.cuda.empty_cache()


def test_far_outputs():
    """Y of 4.6e9 values: rows on both sides of 2^32 against the same rows alone."""
    q, torch = qg(), torch_cuda()
    M, N, K = 70001, 65700, 128
    W = to_dev(q.qquantize_f8(fu.weights(N, K, seed=2)))
    x = torch.randn(M, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
    y = q.qgemm_f8(W, q.qact_quantize_f8(x), M, N, K, dtype=torch.bfloat16)
    for at in (0, (1 << 32) // N - 100, M - 300):
        part = q.qgemm_f8(W, q.qact_quantize_f8(x[at:at + 300]), 300, N, K, dtype=torch.bfloat16)
        # one block of columns: two products of 64 a sum, in one order whatever the tile
        assert torch.equal(y[at:at + 300], part), at
    del y
    torch.cuda.empty_cache()


# ------------------------------------------------------- every choice of tiles
@pytest.mark.parametrize("M,N,K", [(1500, 1490, 300), (2210, 2100, 129), (3600, 3399, 257), (40, 8210, 200), (20, 12400, 384),
                                   (50, 20700, 130), (64, 300, 5000), (31, 4100, 1100)])
@pytest.mark.parametrize("dtype", fu.TYPES)
def test_gemm_shapes_of_tiles(M, N, K, dtype):
    """Sizes on both sides of each choice: 64 x 128, 128 x 128 (both depths), 256 x 256, streaming; ragged edges."""
    q, torch = qg(), torch_cuda()
    W, xq = to_dev(q.qquantize_f8(fu.weights(N, K, seed=31))), q.qact_quantize_f8(to_dev(fu.acts(M, K, seed=32)))
    wv, xv = q.qdequant_f8(W, N, K).double(), q.qact_dequant_f8(xq, M, K).double()
    ref, size = (xv @ wv.t().contiguous()).cpu().numpy(), (xv.abs() @ wv.abs().t().contiguous()).cpu().numpy()
    kind = getattr(torch, dtype)
    buf = torch.full((M * N + 8,), 5.0, dtype=kind, device="cuda")
    y = q.qgemm_f8(W, xq, M, N, K, Y=buf[:M * N].view(M, N))
    fu.assert_close(_np(y), ref, fu.product_bound(ref, size, K, dtype), f"{M}x{N}x{K} {dtype}")
    assert (buf[M * N:] == 5.0).all()


@pytest.mark.parametrize("M,N,K", [(70, 3601, 3500), (600, 3608, 3399), (2200, 3592, 3585), (33, 2055, 2050)])
def test_wgrad_large_tiles(M, N, K):
    q, torch = qg(), torch_cuda()
    xq = q.qact_quantize_f8(to_dev(fu.acts(M, K, seed=34)))
    dy = to_dev(fu.acts(M, N, seed=35)).to(torch.bfloat16)
    xv, dv = q.qact_dequant_f8(xq, M, K).double(), dy.double()
    ref, size = (dv.t().contiguous() @ xv).cpu().numpy(), (dv.abs().t().contiguous() @ xv.abs()).cpu().numpy()
    b = fu.sum_bound(size, M)
    dw = q.qgemm_f8_wgrad(dy, xq, M, N, K)
    fu.assert_close(_np(dw), ref, b, "dW")
    q.qgemm_f8_wgrad(dy, xq, M, N, K, dW=dw, accumulate=True)
    fu.assert_close(_np(dw), 2 * ref, 2 * b + 2.0 ** -23 * (2 * np.abs(ref) + b), "on top of itself")


@pytest.mark.parametrize("P,T,N,K", [(3, 400, 2055, 2050), (40, 700, 520, 1030), (2, 4300, 300, 260)])
@pytest.mark.parametrize("dtype", fu.TYPES)
def test_experts_with_uneven_slots(P, T, N, K, dtype):
    """One expert with most of the slots, some with none: products and weight gradients of wide matrices."""
    q, torch = qg(), torch_cuda()
    pool = to_dev(_pool(P, N, K, seed=41))
    g = np.random.default_rng(T)
    flat = np.where(g.random(T) < 0.6, 1, g.integers(0, P, T))
    flat[flat == 0] = -1
    key = np.where(flat >= 0, flat, P)
    order = np.argsort(key, kind="stable").astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=P + 1)[:P])]).astype(np.int32)
    xq = q.qact_quantize_f8(to_dev(fu.acts(T, K, seed=42)))
    xv = q.qact_dequant_f8(xq, T, K).double()
    dy = to_dev(fu.acts(T, N, seed=43)).to(torch.bfloat16)
    y = q.qmoe_gemm_f8(pool, P, xq, T, to_dev(order), to_dev(off), N, K, dtype=getattr(torch, dtype))
    dw = q.qmoe_gemm_f8_wgrad(dy, xq, T, to_dev(order), to_dev(off), P, N, K)
    yv, nb = _np(y), q.qpacked_bytes_f8(N, K)
    for e in range(P):
        at = np.flatnonzero(flat == e)
        if len(at) == 0:
            assert (dw[e] == 0).all()
            continue
        rows = xv[torch.from_numpy(at).cuda()]
        wv = q.qdequant_f8(pool[e * nb:(e + 1) * nb], N, K).double()
        ref, size = (rows @ wv.t().contiguous()).cpu().numpy(), (rows.abs() @ wv.abs().t().contiguous()).cpu().numpy()
        fu.assert_close(yv[at], ref, fu.product_bound(ref, size, K, dtype), f"expert {e}")
        d = dy[torch.from_numpy(at).cuda()].double()
        ref, size = (d.t().contiguous() @ rows).cpu().numpy(), (d.abs().t().contiguous() @ rows.abs()).cpu().numpy()
        fu.assert_close(_np(dw[e]), ref, fu.sum_bound(size, len(at)), f"gradient of expert {e}")
    assert (yv[flat < 0] == 0).all()
