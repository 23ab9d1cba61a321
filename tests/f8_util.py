"""References of the f8 operators and of the routing, in binary64 numpy, from
the definitions in include/qgemv_f8.h alone (they share no code with the
library)."""
from __future__ import annotations

import numpy as np

TYPES = ("float32", "float16", "bfloat16")
HALF_STEP = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -149, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}   # half a subnormal step (fp32: one)


def code_values() -> np.ndarray:
    """The 256 e4m3 values."""
    c = np.arange(256)
    ex, ma = (c >> 3) & 15, c & 7
    v = np.where(ex > 0, (1 + ma / 8.0) * 2.0 ** (ex - 7.0), ma * 2.0 ** -9)
    v = np.where(c & 0x7F == 0x7F, np.nan, v)
    return np.where(c >= 128, -v, v)


def nearest_code_value(v: np.ndarray) -> np.ndarray:
    """v on the e4m3 grid: the nearest value, ties to the even code, by search over all codes."""
    grid = code_values()[:0x7F]                 # 0 .. 448, codes in order
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    return np.where(np.isfinite(v), np.copysign(grid[code], v), np.nan)


def block_exponent(amax: float) -> int:
    if amax == 0:
        return 0
    e = -127
    while amax > 448 * 2.0 ** e:
        e += 1
    return e


def exponents(amax: np.ndarray) -> np.ndarray:
    flat = amax.reshape(-1)
    out = np.zeros(flat.shape, np.int64)
    nz = flat > 0
    e = np.ceil(np.log2(flat[nz] / 448)).astype(np.int64) - 1
    for _ in range(3):
        e = np.where(flat[nz] > 448 * 2.0 ** e, e + 1, e)
    out[nz] = np.maximum(e, -127)
    return out.reshape(amax.shape)


def quantize_rows(x: np.ndarray):
    """(values fp64, exponents [M][cb]) of activations x[M][K]."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    cb = -(-K // 128)
    p = np.zeros((M, cb * 128))
    p[:, :K] = x
    b = p.reshape(M, cb, 128)
    e = exponents(np.where(np.isfinite(b), np.abs(b), 0).max(2))
    s = 2.0 ** e[:, :, None].astype(np.float64)
    q = nearest_code_value(b / s) * s
    return q.reshape(M, -1)[:, :K], e


def quantize_weights(w: np.ndarray):
    """(values fp64, exponents [rb][cb]) of weights w[N][K]."""
    w = np.asarray(w, np.float64)
    N, K = w.shape
    rb, cb = -(-N // 128), -(-K // 128)
    p = np.zeros((rb * 128, cb * 128))
    p[:N, :K] = w
    b = p.reshape(rb, 128, cb, 128)
    e = exponents(np.abs(b).max((1, 3)))
    s = 2.0 ** e[:, None, :, None].astype(np.float64)
    return (nearest_code_value(b / s) * s).reshape(rb * 128, cb * 128)[:N, :K], e


def unpack_weights(packed: np.ndarray, N: int, K: int):
    """(values fp64 [N][K], padding is zero) of one packed matrix."""
    cb, rt, rb = -(-K // 128), -(-N // 16), -(-N // 128)
    ls = (cb + 3) // 4 * 4
    s0 = 2048 * rt * cb
    n, k = np.arange(16 * rt)[:, None], np.arange(128 * cb)[None]
    at = 2048 * (n // 16 * cb + k // 128) + 256 * (k % 128 // 16) + 16 * (n % 16) + k % 16
    codes = packed[at]
    scales = packed[s0:s0 + rb * ls].reshape(rb, ls)
    v = code_values()[codes] * 2.0 ** (scales[n // 128, k // 128].astype(np.float64) - 127)
    clean = not codes[N:].any() and not codes[:, K:].any() and not scales[:, cb:].any() and \
        not packed[s0 + rb * ls:].any() and packed.size == (s0 + rb * ls + 255) // 256 * 256
    return v[:N, :K], clean


def unpack_acts(packed: np.ndarray, M: int, K: int) -> np.ndarray:
    cb = -(-K // 128)
    s0 = (128 * M * cb + 255) // 256 * 256
    ls = (cb + 3) // 4 * 4
    codes = packed[:128 * M * cb].reshape(M, 128 * cb)
    scales = packed[s0:s0 + M * ls].reshape(M, ls)[:, :cb]
    assert not codes[:, K:].any()
    v = code_values()[codes] * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 128, 1)
    return v[:, :K]


def sum_bound(s: np.ndarray, terms: int) -> np.ndarray:
    """Roundings of `terms` products summed in fp32 (s = sum of magnitudes): a
    matrix instruction rounds at least every eight products, a few more
    additions join waves and parts."""
    return (terms / 8 + 16) * 2.0 ** -24 * s + 1e-37


def product_bound(ref: np.ndarray, s: np.ndarray, terms: int, dtype: str) -> np.ndarray:
    """Of a product sum_k w x with outputs of `dtype`, as qgemv_f8.h states it."""
    if dtype == "float32":
        return sum_bound(s, terms)
    b = 1e-3 * s + sum_bound(s, terms)
    return b + HALF_STEP[dtype] * (np.abs(ref) + b) + TINY[dtype]


def assert_close(y: np.ndarray, ref: np.ndarray, bound: np.ndarray, what: str):
    y = np.asarray(y, np.float64)
    assert y.shape == ref.shape, (what, y.shape, ref.shape)
    bad = ~(np.abs(y - ref) <= bound)
    bad &= ~(np.isnan(y) & np.isnan(ref))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {i}: "
                             f"{y[i]!r} against {ref[i]!r}, bound {bound[i]!r}")


def weights(N, K, seed):
    g = np.random.default_rng([N, K, seed, 11])
    w = g.normal(size=(N, K)).astype(np.float32) * 0.02
    for b in range(0, N, 128):
        for c in range(0, K, 128):
            w[b:b + 128, c:c + 128] *= np.float32(np.exp(g.normal()))
    return w


def acts(M, K, seed):
    g = np.random.default_rng([M, K, seed, 13])
    return (g.normal(size=(M, K)) * np.exp(g.normal(size=(1, K))) * np.exp(0.5 * g.normal(size=(M, 1)))).astype(
        np.float32)


# ------------------------------------------------------------------- routing
def route(logits: np.ndarray, k: int, mask=None, renormalize=True):
    x = np.asarray(logits, np.float64).copy()
    T, E = x.shape
    if mask is not None:
        x[np.asarray(mask) == 0] = -np.inf
    open_ = x > -np.inf
    live = open_.any(1)
    p = np.zeros((T, E))
    for t in np.flatnonzero(live):
        with np.errstate(invalid="ignore"):
            z = np.exp(x[t] - x[t][open_[t]].max())
        p[t] = z / z.sum()
    idx = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        cand = sorted((e for e in range(E) if open_[t, e]), key=lambda e: (-x[t, e], e))[:k]
        idx[t, :len(cand)] = cand
        w[t, :len(cand)] = p[t, cand]
        if renormalize and len(cand):
            w[t, :len(cand)] /= p[t, cand].sum()
    n = int(live.sum())
    flat = idx.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(E)])
    order = sorted(range(T * k), key=lambda s: (flat[s] if flat[s] >= 0 else E, s))
    f = counts / (k * n) if n else np.zeros(E)
    loss = E * float((f * p.sum(0) / n).sum()) if n else 0.0
    return dict(idx=idx, weight=w, counts=counts, tokens=n, offsets=np.concatenate([[0], np.cumsum(counts)]),
                order=np.array(order), loss=loss, p=p, open=open_)


def route_gradient(r, grad_weight, grad_loss, renormalize=True):
    """dlogits from route()'s result, through the softmax's Jacobian."""
    p, idx = r["p"], r["idx"]
    T, E = p.shape
    k = idx.shape[1]
    out = np.zeros((T, E))
    n = r["tokens"]
    for t in range(T):
        dp = np.zeros(E)
        if n and grad_loss is not None:
            dp += grad_loss * E * r["counts"] / (k * n) / n
        sel = idx[t][idx[t] >= 0]
        if grad_weight is not None and len(sel):
            g = np.asarray(grad_weight[t], np.float64)[:len(sel)]
            if renormalize:
                total = p[t, sel].sum()
                dp[sel] += (g - (g * p[t, sel]).sum() / total) / total
            else:
                dp[sel] += g
        out[t] = p[t] * (dp - (p[t] * dp).sum())
    return np.where(r["open"], out, 0.0)
