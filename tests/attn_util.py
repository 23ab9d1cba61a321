"""References of the attention step in binary64 numpy, from the definitions in
include/qgemv_attn.h alone (they share no code with the library)."""
from __future__ import annotations

import numpy as np

import f8_util as fu

HALF_STEP, TINY = fu.HALF_STEP, fu.TINY


def axis_of_pairs(sections):
    return np.concatenate([np.full(n, a) for a, n in enumerate(sections)]) if sum(sections) else np.zeros(0, int)


def turns(positions, freq, sections):
    """cos, sin [T][1][rot / 2] of positions [axes][T]."""
    pos = np.atleast_2d(np.asarray(positions)).astype(np.float64)
    f = np.asarray(freq, np.float32).astype(np.float64)
    angle = pos[axis_of_pairs(sections)].T * f[None] if len(f) else np.zeros((pos.shape[1], 0))
    return np.cos(angle)[:, None], np.sin(angle)[:, None]


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(n, cos, sin, rot, interleaved):
    a, b = pairs(rot, interleaved)
    y = n.copy()
    y[..., a] = n[..., a] * cos - n[..., b] * sin
    y[..., b] = n[..., b] * cos + n[..., a] * sin
    return y


def spread(n, rot, interleaved):
    """|a| + |b| of an element's pair: what a rotation's roundings are relative to."""
    a, b = pairs(rot, interleaved)
    m = np.abs(n)
    m[..., a] = m[..., b] = np.abs(n[..., a]) + np.abs(n[..., b])
    return m


def norm(x, gain, eps):
    x = np.asarray(x, np.float64)
    if gain is None:
        return x.copy(), np.ones(x.shape[:-1] + (1,))
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))
    return x * r * np.asarray(gain, np.float64), r


def norm_rope(x, gain, eps, cos, sin, rot, interleaved):
    return rotate(norm(x, gain, eps)[0], cos, sin, rot, interleaved)


def norm_rope_gradient(x, dy, gain, eps, cos, sin, rot, interleaved):
    """(dx, dgain or None)."""
    h = rotate(np.asarray(dy, np.float64), cos, -sin, rot, interleaved)
    if gain is None:
        return h, None
    x, g = np.asarray(x, np.float64), np.asarray(gain, np.float64)
    r = norm(x, gain, eps)[1]
    n = x * r
    return r * (h * g - n * (h * g * n).mean(-1, keepdims=True)), (h * n).sum((0, 1))


# roundings of norm and rotation in fp32, relative to |a| + |b| of a pair: the sum of squares (16 additions at
# most, halved by the root), the root (2 steps), two products, cosine and sine (a step of 1: they and their angle
# are taken in 64 bits), a product and a sum: under 16 steps of 2^-24
HEADS = 16 * 2.0 ** -24


def heads_bound(n, y, rot, interleaved, dtype):
    b = HEADS * spread(n, rot, interleaved)
    return b + HALF_STEP[dtype] * (np.abs(y) + b) + TINY[dtype]


# ---------------------------------------------------------------------- cache
ITEM = {"f8": 1, "float16": 2, "bfloat16": 2}


def page_bytes(page, heads, dim, cache):
    n = 2 * heads * page * dim * ITEM[cache] + (2 * heads * page if cache == "f8" else 0)
    return -(-n // 256) * 256


def to16(v, cache):
    """fp64 -> what 16 bits hold, rounded to nearest even."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(v, np.float64))
    return t.to(getattr(torch, cache)).double().numpy()


def held(v, cache):
    """What the cache holds of vectors v [..., dim]: (values, exponents or None)."""
    v = np.asarray(v, np.float64)
    if cache != "f8":
        return to16(v, cache), None
    e = np.minimum(fu.exponents(np.where(np.isfinite(v), np.abs(v), 0).max(-1)), 120)[..., None]
    s = 2.0 ** e.astype(np.float64)
    q = fu.nearest_code_value(v / s)
    q = np.where(e == 120, np.clip(q, -240, 240), q)
    return q * s, e[..., 0]


def unpack(data, page, heads, dim, cache):
    """Raw pages uint8 [pages][bytes] -> (k, v) fp64 [pages * page][heads][dim]."""
    data = np.asarray(data)
    pages = data.shape[0]
    end = 2 * heads * page * dim * ITEM[cache]
    raw = np.ascontiguousarray(data[:, :end])
    if cache == "f8":
        v = fu.code_values()[raw].reshape(pages, heads, 2, page, dim)
        e = data[:, end:end + 2 * heads * page].astype(np.float64).reshape(pages, heads, 2, page, 1) - 127
        v = v * 2.0 ** e
    elif cache == "float16":
        v = raw.view(np.float16).astype(np.float64).reshape(pages, heads, 2, page, dim)
    else:
        v = (raw.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        v = v.reshape(pages, heads, 2, page, dim)
    v = v.transpose(2, 0, 3, 1, 4).reshape(2, pages * page, heads, dim)
    return v[0], v[1]


def pack(k, v, page, cache, rng=None):
    """Values [pages * page][heads][dim] as raw pages; the padding is `rng`'s bytes."""
    import torch
    slots, heads, dim = k.shape
    pages = slots // page
    nb = page_bytes(page, heads, dim, cache)
    data = np.zeros((pages, nb), np.uint8) if rng is None else rng.integers(0, 256, (pages, nb), dtype=np.uint8)
    both = np.stack([k, v]).reshape(2, pages, page, heads, dim).transpose(1, 3, 0, 2, 4)
    end = 2 * heads * page * dim * ITEM[cache]
    if cache == "f8":
        vals, e = held(both, cache)
        codes = torch.from_numpy(vals / 2.0 ** e[..., None].astype(np.float64)).float().to(torch.float8_e4m3fn)
        data[:, :end] = codes.view(torch.uint8).numpy().reshape(pages, -1)
        data[:, end:end + 2 * heads * page] = (e + 127).astype(np.uint8).reshape(pages, -1)
    else:
        t = torch.from_numpy(np.ascontiguousarray(both)).to(getattr(torch, cache))
        data[:, :end] = t.contiguous().view(torch.uint8).numpy().reshape(pages, -1)
    return data


# ------------------------------------------------------------------ attention
def attend(q, k, v, table, lens, page, pages, scale, window=0, softcap=0.0):
    """(out, bound of everything but the last rounding), q [B][M][heads][dim], k and v [pages * page][kv heads][dim].

    The bound: scores are sums of dim products in fp32, dim / 8 + 16 roundings of their magnitudes, and a few more
    of the score itself (scale, base 2, cap: 8); the exponential and the weights' two parts lose 2^-16 of a weight
    each at most; sums over n tokens round every 32 tokens, with the joining of parts n / 8 + 64 times."""
    B, M, H, D = q.shape
    share = H // k.shape[1]
    out, bound = np.zeros((B, M, H, D)), np.zeros((B, M, H, D))
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        for i in range(M):
            end = n - M + i + 1
            begin = max(0, end - window) if window else 0
            t = np.arange(begin, max(end, begin))
            p = table[b][t // page] if len(t) else t
            t = t[(p >= 0) & (p < pages)]
            if not len(t):
                continue
            at = table[b][t // page] * page + t % page
            for h in range(H):
                kk, vv = k[at, h // share], v[at, h // share]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = kk @ q[b, i, h] * scale
                    mag = np.abs(kk) @ np.abs(q[b, i, h]) * abs(scale)
                    step = (D / 8 + 16) * 2.0 ** -24 * mag + 8 * 2.0 ** -24 * np.abs(s)
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                        step = step + 8 * 2.0 ** -24 * softcap
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[b, i, h] = w @ vv
                    size = w @ np.abs(vv)
                    bound[b, i, h] = size * (2 * step.max() + 2.0 ** -15 + (len(t) / 8 + 64) * 2.0 ** -24)
    return out, bound


def assert_attend(y, ref, bound, dtype, what):
    fu.assert_close(y, ref, bound + HALF_STEP[dtype] * (np.abs(ref) + bound) + TINY[dtype], what)
