"""The attention step's operators against their references in binary64."""
import numpy as np
import pytest

import attn_util as au
import f8_util as fu
from gpu_util import qg, to_dev, torch_cuda

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _np(t):
    torch_cuda().cuda.synchronize()
    return t.double().cpu().numpy()


def _dt(name):
    torch = torch_cuda()
    return torch.float8_e4m3fn if name == "f8" else getattr(torch, name)


def _rows(rng, T, H, D, dtype):
    """A projection's head vectors on the GPU: channels, heads and tokens of differing size."""
    x = rng.normal(size=(T, H, D)) * np.exp(0.7 * rng.normal(size=(1, H, D))) * np.exp(rng.normal(size=(T, 1, 1)))
    return to_dev(x.astype(np.float32)).to(_dt(dtype))


def _sections(rot, axes):
    n = rot // 2
    cut = [n // (axes + 1)] + [n // (axes + 1) + 1] * (axes - 2) if axes > 1 else []
    return cut + [n - sum(cut)]


# (T, query heads, key heads, D, rot, interleaved, axes, gains' type or None, inputs, outputs)
HEADS = [
    (1, 1, 1, 128, 128, False, 1, "float32", "bfloat16", "bfloat16"),
    (3, 32, 8, 128, 128, False, 1, "float32", "float32", "bfloat16"),
    (7, 4, 2, 128, 128, True, 1, "bfloat16", "float16", "float16"),
    (5, 3, 1, 64, 64, False, 1, "float16", "float32", "float32"),
    (33, 9, 3, 64, 32, True, 2, "float32", "bfloat16", "float32"),
    (6, 5, 5, 256, 256, False, 1, "float32", "float16", "bfloat16"),
    (9, 2, 1, 256, 64, False, 3, "bfloat16", "bfloat16", "bfloat16"),
    (4, 7, 1, 80, 40, False, 1, "float32", "float32", "float32"),
    (13, 3, 2, 96, 96, True, 3, "float32", "bfloat16", "bfloat16"),
    (2, 2, 2, 112, 16, False, 4, "float32", "float16", "float32"),
    (3, 1, 2, 8, 8, False, 1, "float32", "float32", "float32"),
    (3, 2, 1, 24, 8, True, 1, "float32", "float32", "float16"),
    (5, 40, 8, 128, 128, False, 1, None, "bfloat16", "bfloat16"),
    (5, 6, 2, 192, 128, True, 2, None, "float32", "float32"),
    (11, 4, 2, 128, 0, False, 1, "float32", "bfloat16", "bfloat16"),
    (4, 3, 0, 128, 128, False, 1, "float32", "bfloat16", "float32"),
    (4200, 2, 1, 64, 64, False, 1, "float32", "bfloat16", "bfloat16"),
    (2, 1000, 24, 64, 64, False, 1, "float32", "bfloat16", "bfloat16"),
]


class _Heads:
    def __init__(self, case, seed=0):
        self.T, self.nq, self.nk, self.D, self.rot, self.inter, axes, gain, self.x, self.y = case
        self.rng = rng = np.random.default_rng([seed] + [int(v) for v in case[:7]])
        self.sections = _sections(self.rot, axes)
        self.positions = rng.integers(0, 100000, (axes, self.T)).astype(np.int32)
        self.freq = np.exp(-np.arange(self.rot // 2) / max(self.rot // 2, 1) * 9).astype(np.float32)
        # q, k and v of one projection: views with a distance of tokens
        self.qkv = _rows(rng, self.T, self.nq + 2 * self.nk, self.D, self.x)
        self.q, self.k = self.qkv[:, :self.nq], self.qkv[:, self.nq:self.nq + self.nk]
        self.v = self.qkv[:, self.nq + self.nk:]
        self.gains = [None, None]
        if gain:
            self.gains = [to_dev((1 + 0.3 * rng.normal(size=self.D)).astype(np.float32)).to(_dt(gain)) for _ in "qk"]
        self.cos, self.sin = au.turns(self.positions, self.freq, self.sections)
        self.args = (to_dev(self.positions if axes > 1 else self.positions[0]), to_dev(self.freq), *self.gains)
        self.how = dict(eps=EPS, interleaved=self.inter, sections=self.sections if axes > 1 else None)

    def gain(self, i):
        return None if self.gains[i] is None else _np(self.gains[i])

    def reference(self, i):
        x = _np((self.q, self.k)[i])
        n = au.norm(x, self.gain(i), EPS)[0]
        return n, au.rotate(n, self.cos, self.sin, self.rot, self.inter)

    def check(self, got, i, dtype, what):
        n, y = self.reference(i)
        fu.assert_close(_np(got), y, au.heads_bound(n, y, self.rot, self.inter, dtype), what)


@pytest.mark.parametrize("case", HEADS)
def test_norm_rope(case):
    h, q = _Heads(case), qg()
    yq, yk = q.qhead_norm_rope(h.q, h.k if h.nk else None, *h.args, dtype=_dt(h.y), **h.how)
    assert yq.dtype == _dt(h.y) and yq.shape == (h.T, h.nq, h.D)
    h.check(yq, 0, h.y, "q")
    if h.nk:
        h.check(yk, 1, h.y, "k")
    else:
        assert yk is None


@pytest.mark.parametrize("case", [HEADS[1], HEADS[7], HEADS[9], HEADS[12]])
def test_norm_rope_in_place_and_into_views(case):
    h, q = _Heads(case), qg()
    torch = torch_cuda()
    yq, yk = q.qhead_norm_rope(h.q, h.k, *h.args, **h.how)
    wide = torch.full((h.T, h.nq + h.nk + 1, h.D), 7.0, dtype=h.qkv.dtype, device="cuda")
    out = (wide[:, :h.nq], wide[:, h.nq:h.nq + h.nk])
    a, b = q.qhead_norm_rope(h.q, h.k, *h.args, out=out, **h.how)
    assert a is out[0] and torch.equal(a, yq) and torch.equal(b, yk) and (wide[:, -1] == 7).all()
    v = h.v.clone()
    q.qhead_norm_rope(h.q, h.k, *h.args, out=(h.q, h.k), **h.how)
    assert torch.equal(h.q, yq) and torch.equal(h.k, yk) and torch.equal(h.v, v)


@pytest.mark.parametrize("far", [(1 << 31) - 1, -(1 << 31), 1 << 24, -12345])
@pytest.mark.parametrize("cache", ["f8", None])
def test_far_positions(far, cache):
    """The angle of a far position is taken in 64 bits; a 24-bit one would be off by whole turns."""
    h, q = _Heads((3, 2, 2, 128, 128, False, 1, "float32", "float32", "float32")), qg()
    pos = np.array([far, far - 1 if far > 0 else far + 1, 5], np.int32)
    h.cos, h.sin = au.turns(pos, h.freq, h.sections)
    if cache is None:
        yq, yk = q.qhead_norm_rope(h.q, h.k, to_dev(pos), *h.args[1:], **h.how)
        h.check(yq, 0, "float32", "q")
        h.check(yk, 1, "float32", "k")
    else:
        c = q.qkv_cache(1, 16, 2, 128)
        slots = to_dev(np.array([3, 0, 15], np.int32))
        yq = q.qkv_norm_rope_write(c, h.q, h.k, h.v, slots, to_dev(pos), *h.args[1:], **h.how)
        h.check(yq, 0, "float32", "q")
        assert np.array_equal(_np(q.qkv_read(c, slots)[0]), au.held(h.reference(1)[1], "f8")[0])


def test_what_is_not_turned_stays_with_its_infinities():
    q, torch = qg(), torch_cuda()
    x = torch.randn(2, 1, 128, device="cuda")
    x[0, 0, 100] = float("inf")
    x[1, 0, 101] = float("nan")
    pos = to_dev(np.array([5, 9], np.int32))
    y, _ = q.qhead_norm_rope(x, None, pos, torch.rand(32, device="cuda"))
    assert torch.equal(y[0, 0, 64:], x[0, 0, 64:]) and torch.isfinite(y[:, :, :64]).all()
    assert torch.isnan(y[1, 0, 101]) and torch.isfinite(y[1, 0, 102:]).all()


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_the_norm_is_the_same_however_many_pairs_turn(D, dtype):
    """The squares are summed in one order: what no pair turns has the bits that it has where none does."""
    torch = torch_cuda()
    rng = np.random.default_rng(D)
    q, k = (_rows(rng, 300, n, D, dtype) for n in (4, 2))
    gains = [to_dev((1 + 0.3 * rng.normal(size=D)).astype(np.float32)) for _ in "qk"]
    pos = to_dev(rng.integers(0, 5000, 300).astype(np.int32))
    still = qg().qhead_norm_rope(q, k, pos, None, *gains, EPS, dtype=torch.float32)
    rot = 8
    while rot < D:
        freq = to_dev(rng.uniform(0.001, 1, rot // 2).astype(np.float32))
        for y, z in zip(qg().qhead_norm_rope(q, k, pos, freq, *gains, EPS, dtype=torch.float32), still):
            assert torch.equal(y[..., rot:], z[..., rot:]), rot
        rot *= 2


@pytest.mark.parametrize("case", HEADS)
def test_norm_rope_backward(case):
    h, q = _Heads(case), qg()
    dy = [(_rows(h.rng, h.T, n, h.D, h.y) * 0.01) for n in (h.nq, h.nk)]
    got = q.qhead_norm_rope_backward(dy[0], dy[1] if h.nk else None, h.q, h.k if h.nk else None, *h.args, **h.how)
    for i in range(2 if h.nk else 1):
        x, g, d = _np((h.q, h.k)[i]), h.gain(i), _np(dy[i])
        want, want_g = au.norm_rope_gradient(x, d, g, EPS, h.cos, h.sin, h.rot, h.inter)
        size = au.spread(d, h.rot, h.inter)
        if g is None:
            b = au.HEADS * size
            assert got[2 + i] is None
        else:
            # both terms of dx, each off by the roundings of the forward pass twice over and of the mean's D terms
            r = au.norm(x, g, EPS)[1]
            n = np.abs(x * r)
            b = 4 * au.HEADS * r * (size * np.abs(g) + n * (size * np.abs(g) * n).mean(-1, keepdims=True))
            # a wave takes at most two tokens here: the sums of its heads, 32 of the workgroup, then in 64 bits
            assert h.T <= 8192
            terms = 2 * (h.nq + h.nk) + 32
            fu.assert_close(_np(got[2 + i]), want_g, (3 * au.HEADS + terms * 2.0 ** -24) * (size * n).sum((0, 1)),
                            f"gain {i}")
            assert got[2 + i].dtype == torch_cuda().float32
        fu.assert_close(_np(got[i]), want, b + au.HALF_STEP[h.x] * (np.abs(want) + b) + au.TINY[h.x], f"dx {i}")
    if not h.nk:
        assert got[1] is None and got[3] is None


def test_norm_rope_backward_against_differences():
    """fp32 gradients against differences of the reference's forward pass."""
    h, q = _Heads((2, 2, 1, 64, 48, False, 2, "float32", "float32", "float32")), qg()
    dy = [_rows(h.rng, h.T, n, h.D, "float32") for n in (h.nq, h.nk)]
    got = q.qhead_norm_rope_backward(dy[0], dy[1], h.q, h.k, *h.args, **h.how)
    for i in range(2):
        x, g, d = _np((h.q, h.k)[i]), h.gain(i), _np(dy[i])

        def f(x, g):
            return (au.norm_rope(x, g, EPS, h.cos, h.sin, h.rot, h.inter) * d).sum()

        for at in [(0, 0, 0), (1, 0, 5), (0, 0, 30), (1, 0, 47), (0, 0, 48), (1, 0, 63)]:
            step = 1e-6 * (1 + abs(x[at]))
            up, down = x.copy(), x.copy()
            up[at] += step
            down[at] -= step
            want = (f(up, g) - f(down, g)) / (2 * step)
            assert abs(_np(got[i])[at] - want) < 1e-4 * (1 + abs(want))
            up, down = g.copy(), g.copy()
            up[at[2]] += 1e-6
            down[at[2]] -= 1e-6
            want = (f(x, up) - f(x, down)) / 2e-6
            assert abs(_np(got[2 + i])[at[2]] - want) < 1e-4 * (1 + abs(want))


def test_backward_into_the_parts_of_one_gradient():
    h, q = _Heads(HEADS[1]), qg()
    torch = torch_cuda()
    dy = [_rows(h.rng, h.T, n, h.D, "bfloat16") for n in (h.nq, h.nk)]
    want = q.qhead_norm_rope_backward(dy[0], dy[1], h.q, h.k, *h.args, **h.how)
    d = torch.zeros_like(h.qkv)
    got = q.qhead_norm_rope_backward(dy[0], dy[1], h.q, h.k, *h.args,
                                     out=(d[:, :h.nq], d[:, h.nq:h.nq + h.nk]), **h.how)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not d[:, h.nq + h.nk:].any()


# ---------------------------------------------------------------------- cache
CACHES = [(1, 1, 64, 16, "f8", "bfloat16"), (37, 3, 64, 32, "f8", "float32"), (50, 8, 128, 64, "f8", "float16"),
          (21, 2, 192, 16, "f8", "bfloat16"), (9, 1, 256, 1024, "f8", "float32"), (30, 2, 64, 16, "float16", "float32"),
          (40, 3, 128, 128, "bfloat16", "bfloat16"), (13, 2, 192, 32, "float16", "float16"),
          (17, 5, 256, 64, "bfloat16", "float32"), (12, 1024, 64, 16, "f8", "bfloat16"),
          (11, 7, 256, 16, "f8", "float32")]


def _slots(rng, T, total):
    s = rng.permutation(total)[:T].astype(np.int32)
    bad = [-1, total, -(1 << 31), (1 << 31) - 1]
    for i, b in enumerate(bad):
        if T > 8:
            s[2 * i + 1] = b
    return s, (s >= 0) & (s < total)


@pytest.mark.parametrize("T,H,D,page,cache,x", CACHES)
def test_write_and_read(T, H, D, page, cache, x):
    """Bytes at their documented places, all others as they were, and the values back in every type."""
    q, torch = qg(), torch_cuda()
    rng = np.random.default_rng([T, H, D, page])
    pages = T // page + 2
    c = q.qkv_cache(pages, page, H, D, dtype=_dt(cache))
    before = rng.integers(0, 256, tuple(c.data.shape), dtype=np.uint8)
    c.data.copy_(to_dev(before))
    slots, there = _slots(rng, T, pages * page)
    kv = _rows(rng, T, 2 * H + 1, D, x)                       # a distance of tokens
    k, v = kv[:, :H], kv[:, H + 1:]
    k[0, 0] = 0
    q.qkv_write(c, k, v, to_dev(slots))
    after = c.data.cpu().numpy()
    want = [au.held(_np(t), cache)[0] for t in (k, v)]
    kk, vv = au.unpack(after, page, H, D, cache)
    assert np.array_equal(kk[slots[there]], want[0][there]) and np.array_equal(vv[slots[there]], want[1][there])
    # every byte of other slots, and the padding, is untouched
    keep = np.ones((pages, page), bool)
    keep.reshape(-1)[slots[there]] = False
    end = 2 * H * page * D * au.ITEM[cache]
    for a, b, width in ((0, end, D * au.ITEM[cache]), (end, end + (2 * H * page if cache == "f8" else 0), 1)):
        one, two = (t[:, a:b].reshape(pages, 2 * H, -1, width) for t in (before, after))
        if one.size:
            m = np.broadcast_to(keep[:, None], one.shape[:3])
            assert np.array_equal(one[m], two[m])
    tail = end + (2 * H * page if cache == "f8" else 0)
    assert np.array_equal(before[:, tail:], after[:, tail:])
    for name in fu.TYPES:
        if cache == "float16" and name == "bfloat16":
            continue
        got = q.qkv_read(c, to_dev(slots), dtype=_dt(name))
        for t, w in zip(got, want):
            exact = torch.from_numpy(np.where(there[:, None, None], w, 0)).to(_dt(name)).double().numpy()
            assert np.array_equal(_np(t), exact), name


def test_write_of_what_is_not_finite():
    """NaNs and infinities become the NaN code and do not enter the scale; 16-bit caches keep them."""
    q, torch = qg(), torch_cuda()
    x = torch.randn(5, 2, 64, device="cuda")
    x[0, 0, 3], x[1, 1, 60], x[2, 0, 7] = float("nan"), float("inf"), -float("inf")
    x[3] = float("inf")
    x[4, 0] = 3.4e38
    slots = to_dev(np.arange(5, dtype=np.int32))
    want = au.held(_np(x), "f8")[0]
    c = q.qkv_cache(1, 16, 2, 64)
    q.qkv_write(c, x, x, slots)
    for t in q.qkv_read(c, slots):
        got = _np(t)
        assert np.array_equal(np.isnan(got), ~np.isfinite(_np(x)))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))
    c = q.qkv_cache(1, 16, 2, 64, dtype=torch.bfloat16)
    q.qkv_write(c, x, x, slots)
    assert torch.equal(torch.nan_to_num(q.qkv_read(c, slots)[0]), torch.nan_to_num(x.to(torch.bfloat16).float()))


WRITES = [h + (cache, page) for h, cache, page in [
    (HEADS[0], "f8", 16), (HEADS[1], "f8", 64), (HEADS[2], "f8", 32), (HEADS[3], "float16", 16),
    (HEADS[4], "f8", 128), (HEADS[5], "bfloat16", 64), (HEADS[6], "f8", 16), (HEADS[12], "f8", 256),
    (HEADS[12], "bfloat16", 16), (HEADS[13], "f8", 32), (HEADS[14], "f8", 64), (HEADS[16], "f8", 64)]]


@pytest.mark.parametrize("case", WRITES)
def test_norm_rope_write(case):
    cache, page = case[10:]
    h, q = _Heads(case[:10]), qg()
    pages = h.T // page + 2
    c = q.qkv_cache(pages, page, h.nk, h.D, dtype=_dt(cache))
    slots, there = _slots(h.rng, h.T, pages * page)
    y = q.qkv_norm_rope_write(c, h.q, h.k, h.v, to_dev(slots), *h.args, dtype=_dt(h.y), **h.how)
    h.check(y, 0, h.y, "q")
    k, v = (_np(t) for t in q.qkv_read(c, to_dev(slots)))
    n, want = h.reference(1)
    if cache == "f8":
        assert np.array_equal(k[there], au.held(want, cache)[0][there])
    else:
        b = au.heads_bound(n, want, h.rot, h.inter, cache)
        fu.assert_close(k[there], want[there], b[there], "k")
    assert np.array_equal(v[there], au.held(_np(h.v), cache)[0][there])
    assert not k[~there].any() and not v[~there].any()


# ------------------------------------------------------------------ attention
class _Batch:
    """Sequences over a paged cache whose free places hold every byte there is."""

    def __init__(self, lens, M, H, KV, D, page, cache, q_type, seed=0, spare=2, width=None):
        rng = self.rng = np.random.default_rng([seed, M, H, D, page, len(lens)])
        used = [-(-max(n, 0) // page) for n in lens]
        self.width = width or max(1, max(used))
        self.pages = sum(used) + spare
        order = rng.permutation(self.pages)
        self.table = rng.choice([-1, self.pages, 1 << 30, -(1 << 31)], (len(lens), self.width)).astype(np.int64)
        total = self.pages * page
        self.k = rng.normal(size=(total, KV, D)) * np.exp(0.5 * rng.normal(size=(1, KV, D)))
        self.v = rng.normal(size=(total, KV, D)) * np.exp(0.5 * rng.normal(size=(total, KV, 1)))
        self.k, self.v = (au.held(t, cache)[0] for t in (self.k, self.v))
        data = au.pack(self.k, self.v, page, cache, rng)
        live = np.zeros(total, bool)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            for i in range(n):
                left = min(page, lens[b] - i * page)
                live[order[at + i] * page:order[at + i] * page + left] = True
            at += n
        # NaN codes, infinities, scales of 255 in every place without a token
        end = 2 * KV * page * D * au.ITEM[cache]
        free = ~live.reshape(self.pages, 1, page)
        codes = data[:, :end].reshape(self.pages, 2 * KV, page, -1)
        codes[np.broadcast_to(free, codes.shape[:3])] = 0xFF if cache == "f8" else 0x7F
        if cache == "f8":
            scales = data[:, end:end + 2 * KV * page].reshape(self.pages, 2 * KV, page)
            scales[np.broadcast_to(free, scales.shape)] = 255
        self.data, self.lens, self.page, self.cache_type, self.q_type = data, lens, page, cache, q_type
        self.kv, self.D = KV, D
        q = rng.normal(size=(len(lens), M, H, D)) * np.exp(0.5 * rng.normal(size=(len(lens), M, H, 1)))
        self.q = to_dev(q.astype(np.float32)).to(_dt(q_type))

    def cache(self):
        q = qg()
        return q.KVCache(to_dev(self.data), self.page, self.kv, self.D, _dt(self.cache_type))

    def run(self, q=None, **kw):
        t = to_dev(self.table.astype(np.int32))
        n = to_dev(np.array(self.lens, np.int32))
        return qg().qattn_decode(self.cache(), self.q if q is None else q, t, n, **kw)

    def reference(self, scale=None, window=0, softcap=0.0):
        scale = self.D ** -0.5 if scale is None else scale
        return au.attend(_np(self.q), self.k, self.v, self.table, self.lens, self.page, self.pages, scale, window,
                         softcap)

    def check(self, what="attention", **kw):
        y = self.run(**kw)
        ref, bound = self.reference(**kw)
        au.assert_attend(_np(y), ref, bound, self.q_type, what)
        for b, n in enumerate(self.lens):
            for i in range(self.q.shape[1]):
                if n - self.q.shape[1] + i < 0:
                    assert not _np(y)[b, i].any()
        return y


ATTEND = [  # lens, M, heads, key heads, D, page, cache, q
    ([1], 1, 1, 1, 128, 16, "f8", "bfloat16"),
    ([0], 1, 4, 2, 64, 16, "f8", "float16"),
    ([15, 16, 17, 31, 32, 33], 1, 8, 2, 128, 16, "f8", "bfloat16"),
    ([127, 128, 129, 0, 1, 255, 257], 1, 4, 1, 128, 64, "f8", "float16"),
    ([333], 1, 32, 8, 128, 64, "f8", "bfloat16"),
    ([700, 5], 1, 6, 3, 64, 128, "f8", "bfloat16"),
    ([401, 30], 1, 5, 1, 192, 32, "f8", "float16"),
    ([300, 0, 77], 1, 2, 2, 256, 16, "f8", "bfloat16"),
    ([333, 1, 0], 1, 8, 2, 128, 16, "bfloat16", "bfloat16"),
    ([260, 64], 1, 3, 3, 64, 64, "float16", "float16"),
    ([129, 47], 1, 4, 2, 192, 16, "bfloat16", "bfloat16"),
    ([200, 3], 1, 16, 1, 256, 32, "float16", "float16"),
    ([1000, 17, 64], 1, 24, 1, 128, 256, "f8", "bfloat16"),
    ([50, 2, 1, 0, 128], 2, 8, 4, 128, 16, "f8", "bfloat16"),
    ([130, 3, 40], 5, 6, 1, 128, 32, "f8", "float16"),
    ([70, 9, 300], 5, 12, 2, 64, 16, "float16", "float16"),
    ([290, 7], 8, 16, 2, 128, 64, "f8", "bfloat16"),
    ([140, 16, 20], 16, 4, 1, 256, 16, "bfloat16", "bfloat16"),
    ([90, 40], 16, 32, 2, 64, 32, "f8", "bfloat16"),
    ([60, 33], 16, 40, 1, 128, 16, "f8", "float16"),
    ([77, 12], 3, 64, 2, 192, 128, "float16", "float16"),
    ([1500], 4, 4, 4, 128, 1024, "bfloat16", "bfloat16"),
]


@pytest.mark.parametrize("case", ATTEND)
def test_attend(case):
    _Batch(*case).check()


@pytest.mark.parametrize("case", ATTEND)
def test_attend_under_a_wide_table(case):
    """A table for long sequences: work is cut into runs and joined, however short the sequences are."""
    _Batch(*case, width=40000 // case[5]).check()


@pytest.mark.parametrize("case", [ATTEND[3], ATTEND[9], ATTEND[14], ATTEND[18], ATTEND[20]])
@pytest.mark.parametrize("kw", [dict(window=2000), dict(window=70, softcap=9.0), dict(scale=0.0)])
def test_attend_options_under_a_wide_table(case, kw):
    _Batch(*case, width=40000 // case[5]).check(**kw)


@pytest.mark.parametrize("case", [ATTEND[3], ATTEND[6], ATTEND[14], ATTEND[15], ATTEND[17]])
@pytest.mark.parametrize("window", [1, 16, 33, 100, 100000])
def test_attend_in_a_window(case, window):
    _Batch(*case).check(window=window)


@pytest.mark.parametrize("window", [300, 1200, 1900, 100000])
@pytest.mark.parametrize("M,H,KV,D,cache,q,width", [
    (1, 8, 8, 128, "f8", "bfloat16", 32), (3, 8, 4, 64, "f8", "float16", 63),
    (1, 16, 16, 128, "bfloat16", "bfloat16", 32)])
def test_windows_of_many_sequences_under_a_table_of_middle_length(window, M, H, KV, D, cache, q, width):
    """Where the table alone gives a workgroup a sequence, and so asks for no workspace, a window does too."""
    from quantized_weight_gemv_amd import lib
    lens = [2048, 1999, 0, 1] + [int(n) for n in np.random.default_rng(window).integers(0, 150, 60)]
    assert lib().qattn_decode_workspace(len(lens), M, H, KV, D, {"f8": 3, "bfloat16": 2}[cache], 64, width) == 0
    _Batch(lens, M, H, KV, D, 64, cache, q, width=width).check(window=window)


@pytest.mark.parametrize("case", [ATTEND[2], ATTEND[9], ATTEND[14]])
@pytest.mark.parametrize("kw", [dict(softcap=5.0), dict(softcap=50.0, window=40), dict(scale=0.0), dict(scale=-0.3),
                                dict(scale=2.0)])
def test_attend_with_capped_and_scaled_scores(case, kw):
    _Batch(*case).check(**kw)


@pytest.mark.parametrize("cache,q", [("f8", "bfloat16"), ("bfloat16", "bfloat16")])
@pytest.mark.parametrize("lens,M,H,KV,window", [([9001], 1, 8, 2, 0), ([5000, 3, 2049, 700], 1, 4, 2, 0),
                                                ([3001, 900], 4, 4, 1, 0), ([6000, 1], 2, 4, 2, 1500)])
def test_attend_over_long_caches(cache, q, lens, M, H, KV, window):
    """Work that is split over the cache's length and joined."""
    _Batch(lens, M, H, KV, 128, 64, cache, q).check(window=window)


@pytest.mark.parametrize("width", [5, 4000])
@pytest.mark.parametrize("count,most", [(64, 70), (65, 70), (150, 70), (700, 20), (100, 400)])
def test_many_sequences(count, most, width):
    """More sequences than lanes, many of them empty, in portions of one and in runs over several."""
    rng = np.random.default_rng([count, most])
    lens = [int(n) if rng.random() > 0.2 else 0 for n in rng.integers(0, most, count)]
    _Batch(lens, 1, 2, 1, 64, 16, "f8", "bfloat16", width=max(width, most // 16 + 1)).check()


@pytest.mark.parametrize("D,cache,q", [(64, "f8", "float16"), (192, "bfloat16", "bfloat16"), (256, "f8", "bfloat16"),
                                       (256, "float16", "float16")])
def test_one_long_sequence_of_every_width(D, cache, q):
    _Batch([7001], 1, 4, 1, D, 128, cache, q).check()


def test_all_sequences_empty():
    for width in (2, 4000):
        b = _Batch([0] * 70, 2, 4, 2, 128, 16, "bfloat16", "bfloat16", width=width)
        assert not _np(b.check()).any()


def test_pages_that_are_not_there_hold_no_tokens():
    """Entries outside 0 .. pages - 1, inside a sequence's length: at its start, its middle, its end, everywhere."""
    b = _Batch([200, 200, 200, 200, 200], 2, 4, 2, 128, 16, "f8", "bfloat16")
    for row, col, page in ((0, 0, -1), (1, 5, b.pages), (2, 12, 1 << 30), (1, 6, -(1 << 31))):
        b.table[row, col] = page
    b.table[4, :] = -1
    y = b.check()
    assert not _np(y)[4].any()


def test_lengths_are_held_to_the_table():
    """Longer than the table: the table's; negative: none."""
    b = _Batch([64, 64, 64], 1, 4, 2, 128, 16, "f8", "bfloat16")
    full = _np(b.run())
    b.lens = [1 << 30, -5, (1 << 31) - 1]
    got = _np(b.run())
    assert np.array_equal(got[0], full[0]) and not got[1].any() and np.array_equal(got[2], full[2])


@pytest.mark.parametrize("cache,q", [("f8", "bfloat16"), ("bfloat16", "bfloat16"), ("float16", "float16")])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("heads", [4, 20])
def test_values_that_are_not_finite_reach_only_who_sees_them(cache, q, D, heads):
    """New tokens behind a query, and tokens in front of its window, may be NaN or infinite."""
    M, window, share = 4, 40, heads // 2
    b = _Batch([100, 37], M, heads, 2, D, 16, cache, q)
    ref, bound = b.reference(window=window)
    for place, value in ((99, np.nan), (98, np.inf if cache != "f8" else np.nan), (57, np.nan)):
        slot = b.table[0, place // 16] * 16 + place % 16
        raw = {"f8": 0x7F, "bfloat16": 0x7FC0, "float16": 0x7E00}[cache]
        inf = {"bfloat16": 0x7F80, "float16": 0x7C00}.get(cache, 0x7F)
        word = inf if value == np.inf else raw
        page, t = divmod(int(slot), 16)
        codes = b.data[page, :2 * 2 * 16 * D * au.ITEM[cache]].view(np.uint8 if cache == "f8" else np.uint16)
        codes.reshape(2, 2, 16, D)[0, 1, t, 5] = word      # head 0, values, element 5
    got = _np(b.run(window=window))
    # query i stands at 96 + i and sees 57 + i ..: place 57 only query 0, place 98 queries 2 and 3, place 99 query 3
    touched = np.zeros(ref.shape, bool)
    touched[0, 0, :share, 5] = touched[0, 2, :share, 5] = touched[0, 3, :share, 5] = True
    assert np.array_equal(~np.isfinite(got), touched)
    au.assert_attend(np.where(touched, 0, got), np.where(touched, 0, ref), bound, q, "others")


def test_a_key_that_is_not_finite():
    """NaN for who sees it; nothing for the others."""
    b = _Batch([50, 60], 2, 4, 2, 128, 16, "bfloat16", "bfloat16")
    ref, bound = b.reference()
    slot = b.table[1, 59 // 16] * 16 + 59 % 16
    page, t = divmod(int(slot), 16)
    b.data[page, :2 * 2 * 16 * 128 * 2].view(np.uint16).reshape(2, 2, 16, 128)[1, 0, t, 9] = 0x7FC0
    got = _np(b.run())
    touched = np.zeros(ref.shape, bool)
    touched[1, 1, 2:] = True
    assert np.array_equal(np.isnan(got), touched)
    au.assert_attend(np.where(touched, 0, got), np.where(touched, 0, ref), bound, "bfloat16", "others")


def test_queries_of_a_projection_and_a_given_output():
    q, torch = qg(), torch_cuda()
    b = _Batch([90, 33], 3, 4, 2, 128, 16, "f8", "bfloat16")
    y = b.check()
    wide = torch.randn(2, 3, 7, 128, device="cuda").to(torch.bfloat16)
    wide[:, :, 1:5] = b.q
    out = torch.empty_like(y)
    assert b.run(wide[:, :, 1:5], out=out) is out and torch.equal(out, y)
    one = _Batch([90, 33], 1, 4, 2, 128, 16, "f8", "bfloat16")
    assert torch.equal(one.run(one.q[:, 0]), one.run()[:, 0])


def test_a_query_that_is_not_finite():
    torch = torch_cuda()
    b = _Batch([50, 700], 2, 8, 2, 128, 16, "f8", "bfloat16")
    want = b.run()
    b.q[1, 0, 3, 7] = float("nan")
    got = b.run()
    assert torch.isnan(got[1, 0, 3]).all()
    got[1, 0, 3] = want[1, 0, 3]
    assert torch.equal(got, want)


def test_tensors_at_any_element():
    """Inputs and outputs that begin one element behind an aligned address."""
    q, torch = qg(), torch_cuda()

    def moved(t):
        out = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
        return out.copy_(t)

    for dtype in (torch.float32, torch.bfloat16):
        x, dy = (torch.randn(7, 6, 128, device="cuda").to(dtype) for _ in "xd")
        pos, f = torch.arange(7, dtype=torch.int32, device="cuda"), torch.rand(64, device="cuda")
        g = [torch.rand(128, device="cuda").to(dtype) for _ in "qk"]
        args = (moved(pos), moved(f), *(moved(t) for t in g))
        want = q.qhead_norm_rope(x[:, :4], x[:, 4:], pos, f, *g)
        y = moved(x)
        got = q.qhead_norm_rope(y[:, :4], y[:, 4:], *args, out=(y[:, :4], y[:, 4:]))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = q.qhead_norm_rope_backward(dy[:, :4], dy[:, 4:], x[:, :4], x[:, 4:], pos, f, *g)
        y, d = moved(x), moved(dy)
        got = q.qhead_norm_rope_backward(d[:, :4], d[:, 4:], y[:, :4], y[:, 4:], *args, out=(d[:, :4], d[:, 4:]))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        caches = [q.qkv_cache(2, 16, 2, 128) for _ in "ab"]
        slots = torch.arange(7, dtype=torch.int32, device="cuda")
        q.qkv_write(caches[0], x[:, :2], x[:, 2:4], slots)
        y = moved(x)
        q.qkv_write(caches[1], y[:, :2], y[:, 2:4], moved(slots))
        assert torch.equal(caches[0].data, caches[1].data)
    b = _Batch([50, 700], 2, 8, 2, 128, 16, "f8", "bfloat16")
    want = b.run()
    assert torch.equal(b.run(moved(b.q), out=moved(want)), want)


def test_results_repeat_bit_for_bit():
    torch = torch_cuda()
    b = _Batch([5000, 100, 1], 2, 8, 2, 128, 64, "f8", "bfloat16")
    first = b.run()
    for _ in range(3):
        assert torch.equal(b.run(), first)
    h = _Heads(HEADS[16])
    dy = [_rows(h.rng, h.T, n, h.D, "bfloat16") for n in (h.nq, h.nk)]
    first = qg().qhead_norm_rope_backward(dy[0], dy[1], h.q, h.k, *h.args, **h.how)
    for _ in range(3):
        again = qg().qhead_norm_rope_backward(dy[0], dy[1], h.q, h.k, *h.args, **h.how)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


# ------------------------------------------------------------------- refusals
def test_refusals_of_the_binding():
    q, torch = qg(), torch_cuda()
    bf = torch.bfloat16
    x = torch.zeros(4, 6, 128, device="cuda", dtype=bf)
    k = torch.zeros(4, 2, 128, device="cuda", dtype=bf)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(64, device="cuda")
    g = torch.ones(128, device="cuda")
    cache = q.qkv_cache(2, 16, 2, 128)
    table = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    wide = torch.zeros(4, 128, 6, device="cuda", dtype=bf).transpose(1, 2)
    bad = [
        lambda: q.qhead_norm_rope(x, k.float(), pos, f), lambda: q.qhead_norm_rope(x, k[:3], pos, f),
        lambda: q.qhead_norm_rope(x.int(), None, pos, f), lambda: q.qhead_norm_rope(wide, None, pos, f),
        lambda: q.qhead_norm_rope(x, k, pos.long(), f), lambda: q.qhead_norm_rope(x, k, pos[:3], f),
        lambda: q.qhead_norm_rope(x, k, pos, f.double()), lambda: q.qhead_norm_rope(x, k, pos, f, q_gain=g),
        lambda: q.qhead_norm_rope(x, k, pos, f, q_gain=g, k_gain=g[:64]),
        lambda: q.qhead_norm_rope(x, k, pos, f, q_gain=g, k_gain=g.to(bf)),
        lambda: q.qhead_norm_rope(x, k, torch.stack([pos, pos]), f),
        lambda: q.qhead_norm_rope(x, k, torch.stack([pos, pos]), f, sections=[32, 31]),
        lambda: q.qhead_norm_rope(x, k, pos, f, sections=[32, 32]),
        lambda: q.qhead_norm_rope(x, k, pos, torch.zeros(65, device="cuda")),
        lambda: q.qhead_norm_rope(x, k, pos, f, dtype=torch.int8),
        lambda: q.qhead_norm_rope(x, k, pos, f, out=(x, x)),
        lambda: q.qhead_norm_rope(x[:, :, :100], None, pos, None),
        lambda: q.qhead_norm_rope(x[:, 0], None, pos, f), lambda: q.qhead_norm_rope(x[:0], None, pos[:0], f),
        lambda: q.qhead_norm_rope_backward(x, k.float(), x, k, pos, f),
        lambda: q.qhead_norm_rope_backward(x[:, :5], k, x, k, pos, f),
        lambda: q.qkv_write(cache, x, x, pos), lambda: q.qkv_write(cache, k, k.float(), pos),
        lambda: q.qkv_write(cache, k, k, pos.long()), lambda: q.qkv_write(cache._replace(page=24), k, k, pos),
        lambda: q.qkv_write(cache._replace(heads=3), k, k, pos), lambda: q.qkv_write(cache, k, k, pos[:3]),
        lambda: q.qkv_write(cache._replace(data=cache.data[:, :-1].contiguous()), k, k, pos),
        lambda: q.qkv_write(cache._replace(data=cache.data.float()), k, k, pos),
        lambda: q.qkv_read(cache, pos, dtype=torch.float64), lambda: q.qkv_read(cache, pos[:0]),
        lambda: q.qkv_norm_rope_write(cache, x, x, k, pos, pos, f),
        lambda: q.qkv_norm_rope_write(cache, x, k, x, pos, pos, f),
        lambda: q.qkv_norm_rope_write(cache, x, k, k, pos[:2], pos, f),
        lambda: q.qattn_decode(cache, x.float(), table, pos), lambda: q.qattn_decode(cache, x[:, :5], table, pos),
        lambda: q.qattn_decode(cache, x, table[:3], pos), lambda: q.qattn_decode(cache, x, table, pos[:3]),
        lambda: q.qattn_decode(cache, x, table.long(), pos), lambda: q.qattn_decode(cache, x[:, :, :64], table, pos),
        lambda: q.qattn_decode(cache, wide, table, pos), lambda: q.qattn_decode(cache, x, table, pos, window=-1),
        lambda: q.qattn_decode(cache, x, table, pos, softcap=-1.0), lambda: q.qattn_decode(cache, x, table[:, :0], pos),
        lambda: q.qattn_decode(cache, x.view(1, 4, 6, 128).expand(17, 4, 6, 128), table, pos),
        lambda: q.qattn_decode(cache, x, table, pos, out=x.float()),
        lambda: q.qattn_decode(q.qkv_cache(2, 16, 2, 128, dtype=torch.float16), x, table, pos),
    ]
    for n, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, q.QGError)):
            call()
            pytest.fail(f"call {n} was not refused")
    torch.cuda.synchronize()


def test_a_rotation_without_positions_is_refused():
    q, torch = qg(), torch_cuda()
    x = torch.zeros(4, 6, 128, device="cuda", dtype=torch.bfloat16)
    f = torch.zeros(64, device="cuda")
    for call in (lambda: q.qhead_norm_rope(x, x, None, f), lambda: q.qhead_norm_rope_backward(x, x, x, x, None, f)):
        with pytest.raises(TypeError, match="positions"):
            call()
    assert torch.equal(q.qhead_norm_rope(x, x, None, None)[0], x)


def test_calls_that_would_lose_a_gradient_are_refused():
    q, torch = qg(), torch_cuda()
    x = torch.randn(2, 4, 128, device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    f, g = torch.rand(64, device="cuda"), torch.ones(128, device="cuda")
    cache = q.qkv_cache(2, 16, 4, 128)

    def leaf(t):
        return t.detach().clone().requires_grad_()

    calls = [lambda: q.qhead_norm_rope(leaf(x), x, pos, f), lambda: q.qhead_norm_rope(x, leaf(x), pos, f),
             lambda: q.qhead_norm_rope(x, x, pos, f, leaf(g), g), lambda: q.qhead_norm_rope(x, x, pos, leaf(f)),
             lambda: q.qhead_norm_rope_backward(leaf(x), x, x, x, pos, f), lambda: q.qkv_write(cache, leaf(x), x, pos),
             lambda: q.qkv_write(cache, x, leaf(x), pos),
             lambda: q.qkv_norm_rope_write(cache, x, x, leaf(x), pos, pos, f),
             lambda: q.qattn_decode(cache, leaf(x), table, pos)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()
    torch.cuda.synchronize()
