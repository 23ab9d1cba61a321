"""The attention step at the ends of the ranges that its calls accept, under bounds that follow from what a result
is, not from an option's size."""
import numpy as np
import pytest

import attn_util as au
import f8_util as fu
from gpu_util import qg, to_dev, torch_cuda
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


# -------------------------------------------------------------- far positions
FAR = (1 << 31) - 1, -(1 << 31), (1 << 30) + 7, -(1 << 29) - 3, (1 << 27) + 1, 1 << 24, 131071, -1


def _turns(pos, freq):
    """cos, sin [T][1][pairs] of the exact angles: position * freq has 55 bits, 64 are kept here."""
    assert np.finfo(np.longdouble).nmant >= 63
    angle = np.asarray(pos, np.longdouble)[:, None] * np.asarray(freq, np.float32).astype(np.longdouble)
    return np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]


def _freq(rng, n):
    """From 1, the first pair's of every usual rotation, down."""
    return np.concatenate([[1.0], rng.uniform(0.4, 1, n - 1)]).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_the_angle_of_a_far_position_is_as_good_as_of_a_near_one(interleaved, dtype):
    """Forward and backward without a norm: cosine and sine half a step off, two products and a sum rounded, at any
    position: 3 half steps of 2^-24 of |a| + |b|."""
    q, torch = qg(), torch_cuda()
    rng = np.random.default_rng(8)
    T, D = len(FAR), 128
    freq = _freq(rng, D // 2)
    x = to_dev(rng.normal(size=(T, 16, D)).astype(np.float32)).to(getattr(torch, dtype))
    pos = to_dev(np.array(FAR, np.int32))
    cos, sin = _turns(FAR, freq)
    how = dict(interleaved=interleaved)
    y, _ = q.qhead_norm_rope(x, None, pos, to_dev(freq), dtype=torch.float32, **how)
    bound = 3 * U * au.spread(_np(x), D, interleaved)
    fu.assert_close(_np(y), au.rotate(_np(x), cos, sin, D, interleaved), bound, "forward")
    d = q.qhead_norm_rope_backward(x, None, x.float(), None, pos, to_dev(freq), **how)[0]
    fu.assert_close(_np(d), au.rotate(_np(x), cos, -sin, D, interleaved), bound, "backward")


def test_keys_of_far_positions_have_the_codes_of_the_exact_values():
    q, torch = qg(), torch_cuda()
    rng = np.random.default_rng(9)
    T, H, D = 2048, 4, 128
    freq = _freq(rng, D // 2)
    pos = rng.integers(-(1 << 31), 1 << 31, T).astype(np.int32)
    x = to_dev(rng.normal(size=(T, 3 * H, D)).astype(np.float32))
    cache = q.qkv_cache(T // 64, 64, H, D)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    q.qkv_norm_rope_write(cache, x[:, :H], x[:, H:2 * H], x[:, 2 * H:], slots, to_dev(pos), to_dev(freq))
    want = au.rotate(_np(x[:, H:2 * H]), *_turns(pos, freq), D, False)
    assert np.array_equal(_np(q.qkv_read(cache, slots)[0]), au.held(want, "f8")[0])


# ------------------------------------------------------- rows of a key head
@pytest.mark.parametrize("cache", ["bfloat16", "float16", "f8"])
@pytest.mark.parametrize("M,share", [(1, 16), (1, 17), (5, 4), (8, 4), (3, 11), (12, 4), (16, 5), (4, 33)])
def test_rows_of_a_key_head_around_the_tiles_at_256_dimensions(cache, M, share):
    """One tile of 16 rows, two, groups of two, the last ones filled in part; runs over a long table and not."""
    q = "bfloat16" if cache == "f8" else cache
    for width in (None, 2500):
        _Batch([150, M, 37, 0], M, 2 * share, 2, 256, 16, cache, q, width=width).check()


# -------------------------------------------- more sequences than portions of work
FEW_RUNS = [  # sequences, longest, M, heads, key heads, D, cache, q
    (50, 200, 2, 8, 8, 256, "float16", "float16"),       # 32 portions, a wave a row in the join
    (60, 200, 1, 16, 16, 128, "f8", "bfloat16"),         # 48
    (36, 100, 3, 64, 32, 64, "bfloat16", "bfloat16"),    # 32
    (9, 300, 1, 96, 96, 256, "bfloat16", "bfloat16"),    # 2, four waves a row
    (9, 300, 1, 120, 60, 192, "f8", "float16"),          # 8
    (5, 200, 1, 300, 300, 64, "bfloat16", "bfloat16"),   # 3
    (5, 100, 1, 600, 600, 128, "bfloat16", "bfloat16"),  # 1: nothing to join
    (20, 130, 16, 32, 8, 128, "float16", "float16"),     # 64 rows a key head, 16
]


@pytest.mark.parametrize("case", FEW_RUNS)
@pytest.mark.parametrize("window", [0, 150])
def test_more_sequences_than_portions_of_work(case, window):
    """Portions that hold many sequences, sequences that take several portions, cuts between two and inside one."""
    count, longest, M, H, KV, D, cache, q = case
    rng = np.random.default_rng([count, D, KV])
    lens = [int(n) for n in rng.integers(0, longest, count)]
    lens[1], lens[2], lens[3], lens[-1] = 6 * longest, 0, 128, 256
    _Batch(lens, M, H, KV, D, 64, cache, q, width=40000 // 64).check(window=window)


def test_sequences_by_the_thousand_under_a_wide_table():
    b = _Batch([int(n) for n in np.random.default_rng(0).integers(0, 4, 3000)], 1, 2, 2, 64, 16, "f8", "bfloat16",
               width=3000)
    y = _np(b.check())
    assert all(y[i].any() for i, n in enumerate(b.lens) if n)


# --------------------------------------------------- values at the ends of the range
@pytest.mark.parametrize("cache,q", [("f8", "bfloat16"), ("bfloat16", "bfloat16")])
@pytest.mark.parametrize("exponent", [110, 60, -60, -100])
@pytest.mark.parametrize("M,D", [(1, 128), (3, 64), (2, 256)])
def test_values_of_every_size(cache, q, exponent, M, D):
    """300 values of about 2^110, at most 2^115, sum up to some 2^119 in magnitude, and 2^123 may be.  At 2^-100 an 8-bit
    value's scale is 2^-108 or so, and its weight a multiple of 2^-133: half of that is 2^-25 of the largest at most."""
    b = _Batch([300, 41, 0], M, 4, 2, D, 16, cache, q)
    b.v = au.held(b.v * 2.0 ** exponent, cache)[0]
    assert np.abs(b.v).max() < 2.0 ** (exponent + 5)
    b.data = au.pack(b.k, b.v, 16, cache)
    y = b.run()
    out, bound = b.reference()
    lost = 300 * 2.0 ** -25 * np.abs(b.v).max() if cache == "f8" and exponent == -100 else 0.0
    au.assert_attend(_np(y), out, bound + lost, q, f"values of 2^{exponent}")


@pytest.mark.parametrize("cache", ["bfloat16", "float16"])
@pytest.mark.parametrize("M", [1, 3])
def test_a_value_that_is_not_finite_reaches_who_sees_it(cache, M):
    """At the end of a sequence and in its middle, and no other element or sequence."""
    for place in (199, 70):
        b = _Batch([200, 180], M, 4, 2, 128, 16, cache, cache)
        ref, bound = b.reference()
        page, t = divmod(int(b.table[0, place // 16] * 16 + place % 16), 16)
        word = {"bfloat16": 0xFF80, "float16": 0xFC00}[cache]
        b.data[page, :2 * 2 * 16 * 128 * 2].view(np.uint16).reshape(2, 2, 16, 128)[1, 1, t, 77] = word   # -infinity
        got = _np(b.run())
        touched = np.zeros(ref.shape, bool)
        touched[0, M - 1 if place == 199 else slice(None), 2:, 77] = True
        assert np.array_equal(~np.isfinite(got), touched)
        au.assert_attend(np.where(touched, 0, got), np.where(touched, 0, ref), bound, cache, "others")
