"""The attention step's entry points without a GPU: sizes, refusals (all
made on the host, before any launch), and the references against their own
definitions."""
import ctypes

import numpy as np
import pytest

import attn_util as au

P = 0x10000000           # an aligned address that no refused call touches


def _lib():
    import quantized_weight_gemv_amd as q
    return q.lib()


def test_page_bytes():
    L = _lib()
    for page in (16, 32, 64, 128, 256, 512, 1024):
        for heads in (1, 3, 8, 1024):
            for dim in (64, 128, 192, 256):
                for code, name in ((3, "f8"), (1, "float16"), (2, "bfloat16")):
                    assert L.qkv_page_bytes(page, heads, dim, code) == au.page_bytes(page, heads, dim, name)
    for bad in ((0, 8, 128, 3), (8, 8, 128, 3), (48, 8, 128, 3), (2048, 8, 128, 3), (-16, 8, 128, 3), (16, 0, 128, 3),
                (16, 1025, 128, 3), (16, 8, 0, 3), (16, 8, 96, 3), (16, 8, 512, 3), (16, 8, 128, 0),
                (16, 8, 128, 4)):
        assert L.qkv_page_bytes(*bad) == 0, bad


def _sections(*n):
    return (ctypes.c_int32 * len(n))(*n)


def _heads(**kw):
    a = dict(q=P, ldq=1024, nq=4, k=P, ldk=1024, nk=2, xt=2, gq=P, gk=P, gt=0, eps=1e-6, pos=P, axes=1, sec=None,
             freq=P, rot=128, inter=0, T=3, D=128, yq=P, ldyq=512, yk=P, ldyk=256, yt=2)
    a.update(kw)
    return tuple(a.values())


NULL, SHAPE, ALIGN = 1, 2, 3
HEAD_REFUSALS = [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(gq=None), NULL), (dict(gk=None), NULL), (dict(pos=None), NULL),
    (dict(freq=None), NULL), (dict(axes=2), NULL), (dict(yq=None), NULL), (dict(yk=None), NULL),
    (dict(ldq=511), SHAPE), (dict(ldk=255), SHAPE), (dict(ldyq=511), SHAPE), (dict(ldyk=255), SHAPE),
    (dict(nq=0), SHAPE), (dict(nk=-1), SHAPE), (dict(nq=1024, ldq=1 << 20, ldyq=1 << 20), SHAPE), (dict(xt=3), SHAPE),
    (dict(yt=3), SHAPE), (dict(gt=3), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(eps=float("inf")), SHAPE), (dict(axes=0), SHAPE), (dict(axes=5, sec=_sections(16, 16, 16, 8, 8)), SHAPE),
    (dict(axes=2, sec=_sections(16, 47)), SHAPE), (dict(axes=2, sec=_sections(16, 49)), SHAPE),
    (dict(axes=2, sec=_sections(-1, 65)), SHAPE), (dict(axes=2, sec=_sections(1 << 30, 1 << 30)), SHAPE),
    (dict(rot=136), SHAPE), (dict(rot=-8), SHAPE), (dict(rot=12), SHAPE), (dict(T=0), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=(1 << 30) + 1), SHAPE), (dict(D=12, rot=8), SHAPE), (dict(D=264), SHAPE), (dict(D=0, rot=0), SHAPE),
    (dict(ldq=1 << 62), SHAPE), (dict(q=P + 1), ALIGN), (dict(yk=P + 1), ALIGN), (dict(gq=P + 2), ALIGN),
    (dict(pos=P + 2), ALIGN), (dict(freq=P + 2), ALIGN),
]


@pytest.mark.parametrize("kw,status", HEAD_REFUSALS)
def test_norm_rope_refuses(kw, status):
    assert _lib().qhead_norm_rope(*_heads(**kw), None) == status


def _backward(**kw):
    a = dict(gyq=P, ldgq=512, gyk=P, ldgk=256, yt=2, q=P, ldq=1024, nq=4, k=P, ldk=1024, nk=2, xt=2, gq=P, gk=P, gt=0,
             eps=1e-6, pos=P, axes=1, sec=None, freq=P, rot=128, inter=0, T=3, D=128, dq=P, lddq=512, dk=P, lddk=256,
             g=P, ws=P)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [r for r in HEAD_REFUSALS if not {"yq", "yk", "ldyq", "ldyk"} & set(r[0])] + [
    (dict(gyq=None), NULL), (dict(gyk=None), NULL), (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(g=None), NULL),
    (dict(ws=None), NULL), (dict(ldgq=511), SHAPE), (dict(ldgk=255), SHAPE), (dict(lddq=511), SHAPE),
    (dict(lddk=255), SHAPE), (dict(ws=P + 8), ALIGN), (dict(g=P + 2), ALIGN), (dict(gyq=P + 1), ALIGN)])
def test_norm_rope_backward_refuses(kw, status):
    assert _lib().qhead_norm_rope_backward(*_backward(**kw), None) == status


CACHE_REFUSALS = [
    (dict(cache=None), NULL), (dict(cache=P + 128), ALIGN), (dict(pages=0), SHAPE), (dict(pages=-1), SHAPE),
    (dict(pages=(1 << 31) // 64), SHAPE), (dict(page=8), SHAPE), (dict(page=24), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=1025), SHAPE), (dict(dim=96), SHAPE), (dict(type=0), SHAPE), (dict(type=4), SHAPE)]


def _cache(**kw):
    a = dict(cache=P, pages=10, page=64, heads=2, dim=128, type=3)
    a.update({n: v for n, v in kw.items() if n in a})
    return tuple(a.values()), {n: v for n, v in kw.items() if n not in a}


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(ldk=255), SHAPE),
    (dict(ldv=255), SHAPE), (dict(xt=3), SHAPE), (dict(T=0), SHAPE), (dict(k=P + 1), ALIGN),
    (dict(slots=P + 2), ALIGN)])
def test_write_refuses(kw, status):
    cache, kw = _cache(**kw)
    a = dict(k=P, ldk=256, v=P, ldv=256, xt=2, slots=P, T=5)
    a.update(kw)
    assert _lib().qkv_write(*a.values(), *cache, None) == status


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(yt=3), SHAPE), (dict(T=0), SHAPE),
    (dict(v=P + 1), ALIGN)])
def test_read_refuses(kw, status):
    cache, kw = _cache(**kw)
    a = dict(slots=P, T=5, k=P, v=P, yt=2)
    a.update(kw)
    assert _lib().qkv_read(*cache, *a.values(), None) == status


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(yq=None), NULL),
    (dict(gk=None), NULL), (dict(ldv=255), SHAPE), (dict(ldyq=511), SHAPE), (dict(yt=3), SHAPE), (dict(rot=136), SHAPE),
    (dict(v=P + 1), ALIGN), (dict(yq=P + 1), ALIGN)])
def test_norm_rope_write_refuses(kw, status):
    cache, kw = _cache(**kw)
    a = dict(q=P, ldq=1024, nq=4, k=P, ldk=1024, v=P, ldv=1024, xt=2, gq=P, gk=P, gt=0, eps=1e-6, pos=P, axes=1,
             sec=None, freq=P, rot=128, inter=0, T=3, slots=P, yq=P, ldyq=512, yt=2)
    a.update(kw)
    assert _lib().qkv_norm_rope_write(*a.values(), *cache, None) == status


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    (dict(q=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
    (dict(qt=0), SHAPE), (dict(qt=3), SHAPE), (dict(type=2, qt=1), SHAPE), (dict(ldq=511), SHAPE), (dict(B=0), SHAPE),
    (dict(B=65537), SHAPE), (dict(M=0), SHAPE), (dict(M=17), SHAPE), (dict(nq=3), SHAPE), (dict(nq=1), SHAPE),
    (dict(nq=1026, ldq=1 << 20), SHAPE), (dict(B=65536, M=16, nq=16, ldq=2048), SHAPE),
    (dict(width=(1 << 30) // 64 + 1), SHAPE), (dict(B=65, width=(1 << 30) // 64), SHAPE), (dict(width=0), SHAPE),
    (dict(width=(1 << 31) // 64), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(window=-1), SHAPE),
    (dict(window=1 << 31), SHAPE), (dict(cap=-1.0), SHAPE), (dict(cap=float("inf")), SHAPE), (dict(cap=1e-40), SHAPE),
    (dict(q=P + 1), ALIGN),
    (dict(table=P + 2), ALIGN), (dict(lens=P + 2), ALIGN), (dict(out=P + 1), ALIGN), (dict(ws=P + 8), ALIGN)])
def test_attend_refuses(kw, status):
    cache, kw = _cache(**kw)
    a = dict(q=P, qt=2, ldq=512, B=3, M=1, nq=4, table=P, width=7, lens=P, scale=0.1, window=0, cap=0.0, out=P, ws=P)
    a.update(kw)
    assert _lib().qattn_decode(*cache, *a.values(), None) == status


def test_workspaces_of_sizes_out_of_range():
    L = _lib()
    assert L.qhead_norm_rope_backward_workspace(5, 4, 2, 128, 0) == 0
    assert L.qhead_norm_rope_backward_workspace(0, 4, 2, 128, 1) == 0
    assert L.qhead_norm_rope_backward_workspace(5, 4, 2, 130, 1) == 0
    assert L.qhead_norm_rope_backward_workspace(5, 4, 2, 128, 1) > 0
    assert L.qattn_decode_workspace(1, 17, 4, 2, 128, 3, 64, 7) == 0
    assert L.qattn_decode_workspace(1, 1, 3, 2, 128, 3, 64, 7) == 0


def test_the_binding_refuses_host_tensors():
    import torch

    import quantized_weight_gemv_amd as q
    x = torch.zeros(2, 4, 128)
    pos = torch.zeros(2, dtype=torch.int32)
    cache = q.qkv_cache(2, 16, 4, 128, device="cpu")
    for call in (lambda: q.qhead_norm_rope(x, x, pos, None), lambda: q.qkv_write(cache, x, x, pos),
                 lambda: q.qkv_read(cache, pos), lambda: q.qattn_decode(cache, x, pos.view(2, 1), pos),
                 lambda: q.qhead_norm_rope_backward(x, x, x, x, pos, None),
                 lambda: q.qkv_norm_rope_write(cache, x, x, x, pos, pos, None)):
        with pytest.raises(TypeError, match="device"):
            call()
    with pytest.raises(TypeError):
        q.qkv_cache(2, 16, 4, 128, dtype=torch.float32, device="cpu")
    with pytest.raises(q.QGError):
        q.qkv_cache(2, 16, 4, 100, device="cpu")


# ------------------------------------------------------------- the references
@pytest.mark.parametrize("D,rot,interleaved,sections", [(16, 16, False, [8]), (24, 16, True, [3, 5]),
                                                        (8, 0, False, [0]), (32, 24, False, [2, 4, 6])])
@pytest.mark.parametrize("normed", [False, True])
def test_reference_gradient_against_differences(D, rot, interleaved, sections, normed):
    g = np.random.default_rng([D, rot, normed])
    T, H, eps = 3, 2, 1e-6
    x, dy = g.normal(size=(T, H, D)), g.normal(size=(T, H, D))
    gain = g.normal(size=D) if normed else None
    pos = g.integers(-50, 50, (len(sections), T))
    cos, sin = au.turns(pos, g.random(rot // 2), sections)

    def f(x, gain):
        return (au.norm_rope(x, gain, eps, cos, sin, rot, interleaved) * dy).sum()

    dx, dg = au.norm_rope_gradient(x, dy, gain, eps, cos, sin, rot, interleaved)
    step = 1e-5
    for at in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[at] += step
        down[at] -= step
        assert abs((f(up, gain) - f(down, gain)) / (2 * step) - dx[at]) < 1e-7
    if normed:
        for i in range(D):
            up, down = gain.copy(), gain.copy()
            up[i] += step
            down[i] -= step
            assert abs((f(x, up) - f(x, down)) / (2 * step) - dg[i]) < 1e-7


def test_reference_rotation_is_a_turn():
    """Lengths of pairs stay, and turning by p then by q is turning by p + q."""
    g = np.random.default_rng(3)
    x, f = g.normal(size=(4, 2, 16)), g.random(8).astype(np.float32)
    p, q = g.integers(0, 99, 4), g.integers(0, 99, 4)
    for inter in (False, True):
        one = au.rotate(x, *au.turns(p, f, [8]), 16, inter)
        a, b = au.pairs(16, inter)
        assert np.allclose(one[..., a] ** 2 + one[..., b] ** 2, x[..., a] ** 2 + x[..., b] ** 2)
        two = au.rotate(one, *au.turns(q, f, [8]), 16, inter)
        assert np.allclose(two, au.rotate(x, *au.turns(p + q, f, [8]), 16, inter))


@pytest.mark.parametrize("cache", ["f8", "float16", "bfloat16"])
def test_reference_pages_there_and_back(cache):
    g = np.random.default_rng(5)
    k, v = g.normal(size=(64, 3, 64)), g.normal(size=(64, 3, 64)) * 1e-3
    kk, vv = au.unpack(au.pack(k, v, 32, cache), 32, 3, 64, cache)
    assert np.array_equal(kk, au.held(k, cache)[0]) and np.array_equal(vv, au.held(v, cache)[0])


def test_reference_attention_worked_example():
    """Two places, equal scores; one place; a page that is not there; nothing."""
    k, v = np.zeros((32, 1, 64)), np.zeros((32, 1, 64))
    v[16:18, 0, 0] = [1.0, 3.0]
    q = np.ones((4, 1, 2, 64))
    table = np.array([[1], [1], [7], [1]])
    out, _ = au.attend(q, k, v, table, [2, 1, 2, 0], 16, 2, 1.0)
    assert np.array_equal(out[:, 0, 0, 0], [2.0, 1.0, 0.0, 0.0]) and not out[..., 1:].any()
    out, _ = au.attend(np.ones((1, 3, 2, 64)), k, v, table[:1], [2], 16, 2, 1.0, window=1)
    assert np.array_equal(out[0, :, 1, 0], [0.0, 1.0, 3.0])
