"""GPU parity of the expert routing, its counts, sorted slots, balance loss
and gradient against the binary64 reference of f8_util."""
import numpy as np
import pytest

import f8_util as fu
from gpu_util import qg, to_dev, torch_cuda

pytestmark = pytest.mark.gpu


def _logits(T, E, dtype, seed, closed=0.0):
    torch = torch_cuda()
    g = np.random.default_rng([T, E, seed])
    x = g.normal(size=(T, E)) * 1.5 + g.normal(size=(1, E))
    x[g.random((T, E)) < closed] = -np.inf
    t = to_dev(x.astype(np.float32)).to(getattr(torch, dtype))
    return t, t.double().cpu().numpy()


def _check(r, ref, what):
    torch_cuda().cuda.synchronize()
    for name in ("idx", "counts", "offsets", "order"):
        assert np.array_equal(getattr(r, name).cpu().numpy(), ref[name]), (what, name)
    assert int(r.tokens.item()) == ref["tokens"]
    # exp, the sums of up to 512 of them and two divisions: a few units of 2^-24 each, and 2^-23 |x| from the
    # argument of exp, whose |x| here is below 32
    fu.assert_close(r.weight.cpu().numpy(), ref["weight"], 2.0 ** -18 * ref["weight"] + 1e-37, what)
    fu.assert_close(r.loss.cpu().numpy(), np.array([ref["loss"]]), 2.0 ** -18 * np.array([ref["loss"]]), what)


SHAPES = [(1, 1, 1), (1, 128, 10), (4, 128, 8), (63, 64, 2), (64, 65, 16), (65, 8, 8), (130, 256, 8), (1000, 60, 6),
          (300, 512, 16), (4097, 16, 2)]


@pytest.mark.parametrize("dtype", fu.TYPES)
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route(T, E, k, dtype):
    q, torch = qg(), torch_cuda()
    x, xv = _logits(T, E, dtype, seed=1, closed=0.05)
    mask = np.random.default_rng(T).random(T) >= 0.1
    for m in (None, mask):
        for renorm in (True, False):
            r = q.qmoe_route(x, k, mask=None if m is None else to_dev(m), renormalize=renorm)
            _check(r, fu.route(xv, k, m, renorm), f"{T}x{E} k={k} {dtype} renorm={renorm}")


@pytest.mark.parametrize("T", [3, 200])
def test_route_rows_that_leave_nothing(T):
    q, torch = qg(), torch_cuda()
    E, k = 24, 4
    x, _ = _logits(T, E, "float32", seed=2)
    x[0] = -float("inf")                                  # no expert is open
    x[1] = -float("inf")
    x[1, 5], x[1, 9] = 0.5, -2.0                          # fewer than k
    x[2] = torch.finfo(torch.float32).min                 # lowest finite value: all equal, not closed
    xv = x.double().cpu().numpy()
    for m in (np.ones(T, bool), np.zeros(T, bool), np.arange(T) % 2 == 1):
        r = q.qmoe_route(x, k, mask=to_dev(m))
        ref = fu.route(xv, k, m)
        _check(r, ref, "rows that leave nothing")
        gw, gl = torch.randn(T, k, device="cuda"), torch.full((1,), 3.0, device="cuda")
        d = q.qmoe_route_backward(x, r, grad_weight=gw, grad_loss=gl, mask=to_dev(m))
        want = fu.route_gradient(ref, gw.double().cpu().numpy(), 3.0)
        assert torch.isfinite(d).all()
        fu.assert_close(d.double().cpu().numpy(), want, np.full((T, E), 1e-4), "gradient")
        assert (d[~to_dev(m)] == 0).all() and (d[0] == 0).all()
        assert (d[1, [e for e in range(E) if e not in (5, 9)]] == 0).all()


def test_route_ties_go_to_the_lowest_index():
    q, torch = qg(), torch_cuda()
    for T, E, k in ((5, 200, 16), (150, 70, 7)):
        g = np.random.default_rng(4)
        xv = g.integers(-2, 3, size=(T, E)).astype(np.float64)
        xv[0] = 0.0
        xv[1, ::2] = -0.0
        xv[1, 1::2] = 0.0
        for dtype in fu.TYPES:
            x = to_dev(xv.astype(np.float32)).to(getattr(torch, dtype))
            _check(q.qmoe_route(x, k), fu.route(xv, k), f"ties {dtype}")


def test_route_nan_and_infinity_stay_in_their_token():
    q, torch = qg(), torch_cuda()
    for T in (6, 100):
        x, xv = _logits(T, 40, "float32", seed=5)
        clean = q.qmoe_route(x, 4)
        y = x.clone()
        y[1, 3], y[4, 7] = float("nan"), float("inf")
        r = q.qmoe_route(y, 4)
        assert torch.isnan(r.weight[[1, 4]]).all() and torch.isnan(r.loss).all()
        assert 3 not in r.idx[1].tolist() and r.idx[4, 0].item() == 7
        keep = [t for t in range(T) if t not in (1, 4)]
        assert torch.equal(r.idx[keep], clean.idx[keep]) and torch.equal(r.weight[keep], clean.weight[keep])
        assert int(r.offsets[-1]) == 4 * T and sorted(r.order.tolist()) == list(range(4 * T))


def test_route_strided_logits_and_repeats():
    q, torch = qg(), torch_cuda()
    wide = torch.randn(500, 131, device="cuda")
    for dtype in fu.TYPES:
        w = wide.to(getattr(torch, dtype))
        a, b = q.qmoe_route(w[:, 3:100], 5), q.qmoe_route(w[:, 3:100].contiguous(), 5)
        for u, v in zip(a, b):
            assert torch.equal(u, v)
        g = torch.randn(500, 5, device="cuda")
        one = torch.ones(1, device="cuda")
        da = q.qmoe_route_backward(w[:, 3:100], a, grad_weight=g, grad_loss=one)
        db = q.qmoe_route_backward(w[:, 3:100].contiguous(), b, grad_weight=g, grad_loss=one)
        assert torch.equal(da, db)


@pytest.mark.parametrize("dtype", fu.TYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (7, 128, 10), (200, 65, 3), (130, 300, 16)])
def test_route_gradient(T, E, k, renorm, dtype):
    q, torch = qg(), torch_cuda()
    x, xv = _logits(T, E, dtype, seed=6, closed=0.05)
    mask = np.random.default_rng(T + 1).random(T) >= 0.2
    r = q.qmoe_route(x, k, mask=to_dev(mask), renormalize=renorm)
    ref = fu.route(xv, k, mask, renorm)
    gw = torch.randn(T, k, device="cuda")
    gl = torch.full((1,), 0.7 * T, device="cuda")
    g64 = gw.double().cpu().numpy()
    for a, b in ((gw, gl), (gw, None), (None, gl), (None, None)):
        d = q.qmoe_route_backward(x, r, grad_weight=a, grad_loss=b, mask=to_dev(mask), renormalize=renorm)
        assert d.dtype == x.dtype
        want = fu.route_gradient(ref, None if a is None else g64, None if b is None else 0.7 * T, renorm)
        # each term of p (dp - sum p dp) and w (g - sum g w) carries 2^-18 of its size (as in _check)
        big = (np.abs(g64).max(1, keepdims=True) if a is not None else 0) * \
            (ref["p"] / np.maximum(1e-30, (ref["p"] * (ref["open"] & _chosen(ref))).sum(1, keepdims=True)) if renorm
             else ref["p"]) + \
            (0.7 * T * E * ref["p"] * ref["counts"].max() / (k * max(1, ref["tokens"]) ** 2) if b is not None else 0)
        bound = 2.0 ** -16 * big + fu.HALF_STEP[dtype] * np.abs(want) + 2 * fu.TINY[dtype] + 1e-37
        fu.assert_close(d.double().cpu().numpy(), want, bound, f"gradient {T}x{E}")


def _chosen(ref):
    c = np.zeros(ref["p"].shape, bool)
    for t, row in enumerate(ref["idx"]):
        c[t, row[row >= 0]] = True
    return c


def test_route_gradient_against_differences():
    """Central differences of the reference's own weight and loss (counts held): an error of the formula, not
    of rounding, would show."""
    q, torch = qg(), torch_cuda()
    T, E, k = 5, 9, 3
    x, xv = _logits(T, E, "float32", seed=9)
    g = np.random.default_rng(1).normal(size=(T, k))
    r = q.qmoe_route(x, k)
    d = q.qmoe_route_backward(x, r, grad_weight=to_dev(g.astype(np.float32)), grad_loss=torch.full((1,), 2.0, device="cuda"))
    base = fu.route(xv, k)

    def value(v):
        p = np.exp(v) / np.exp(v).sum(1, keepdims=True)
        w = np.take_along_axis(p, base["idx"], 1)
        w = w / w.sum(1, keepdims=True)
        f = base["counts"] / (k * T)
        return (g * w).sum() + 2.0 * E * (f * p.mean(0)).sum()

    h = 1e-5
    for t in range(T):
        for e in range(E):
            a, b = xv.copy(), xv.copy()
            a[t, e] += h
            b[t, e] -= h
            # differences: h^2 of the third derivative (about 1e-10) and 1e-16 / h of rounding; the kernel's fp32
            assert abs(float(d[t, e]) - (value(a) - value(b)) / (2 * h)) < 1e-5


def test_route_checks():
    q, torch = qg(), torch_cuda()
    x = torch.randn(4, 8, device="cuda")
    r = q.qmoe_route(x, 2)
    for call in (lambda: q.qmoe_route(x, 9), lambda: q.qmoe_route(x, 0), lambda: q.qmoe_route(torch.zeros(2, 513, device="cuda"), 2),
                 lambda: q.qmoe_route(torch.zeros(0, 8, device="cuda"), 2), lambda: q.qmoe_route(torch.zeros(4, 32, device="cuda"), 17)):
        with pytest.raises(q.QGError) as e:
            call()
        assert e.value.status == 2
    for call in (lambda: q.qmoe_route(x.t(), 2), lambda: q.qmoe_route(x, 2, mask=torch.ones(3, dtype=torch.bool, device="cuda")),
                 lambda: q.qmoe_route_backward(x[:3], r), lambda: q.qmoe_route_backward(x, r, grad_weight=torch.zeros(4, 3, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        q.qmoe_route(x.double(), 2)


@pytest.mark.parametrize("dtype", fu.TYPES)
@pytest.mark.parametrize("T,E,k", [(70, 200, 8), (33, 512, 16), (100, 257, 5), (2100, 64, 6)])
def test_route_gradient_of_many_experts(T, E, k, dtype):
    for renorm in (True, False):
        test_route_gradient(T, E, k, renorm, dtype)
