"""The attention step as programs use it: a decode step from projection to
projection, a training layer as an autograd function, captured graphs, other
streams, several calls at once, buffers beyond 32-bit offsets."""
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


def _freq(rot):
    return np.exp(-np.arange(rot // 2) / (rot // 2) * 9).astype(np.float32)


# ------------------------------------------------------------- a decode step
@pytest.mark.parametrize("cache_type,page", [("float8_e4m3fn", 16), ("bfloat16", 32)])
@pytest.mark.parametrize("M", [1, 3])
def test_decode_steps_from_projection_to_projection(cache_type, page, M):
    """A prompt written with qkv_write, then steps of M tokens a sequence: f8 projection -> norm, rotation and
    write -> attention -> f8 projection, each against its definition on the inputs that the step had."""
    q, torch = qg(), torch_cuda()
    rng = np.random.default_rng([M, page])
    B, H, KV, D, W = 3, 4, 2, 64, 96
    heads = H + 2 * KV
    dtype = getattr(torch, cache_type)
    name = "f8" if cache_type.startswith("float8") else cache_type
    lens = np.array([0, 5, 40], np.int64)
    pages = 20
    table = rng.permutation(pages)[:B * 6].reshape(B, 6)
    cache = q.qkv_cache(pages, page, KV, D, dtype=dtype)
    # prompts
    places = [(b, t) for b in range(B) for t in range(lens[b])]
    slots = np.array([table[b, t // page] * page + t % page for b, t in places], np.int32)
    k0, v0 = (to_dev(rng.normal(size=(len(places), KV, D)).astype(np.float32)) for _ in "kv")
    q.qkv_write(cache, k0, v0, to_dev(slots))
    held_k, held_v = np.zeros((pages * page, KV, D)), np.zeros((pages * page, KV, D))
    held_k[slots], held_v[slots] = au.held(_np(k0), name)[0], au.held(_np(v0), name)[0]
    w_in, w_out = fu.weights(heads * D, W, seed=1), fu.weights(W, H * D, seed=2)
    wi, wo = to_dev(q.qquantize_f8(w_in)), to_dev(q.qquantize_f8(w_out))
    gq, gk = (to_dev((1 + 0.2 * rng.normal(size=D)).astype(np.float32)) for _ in "qk")
    freq = _freq(D)
    d_table = to_dev(table.astype(np.int32))
    for _ in range(3):
        x = to_dev(rng.normal(size=(B * M, W)).astype(np.float32))
        lens = lens + M
        pos = np.array([lens[b] - M + i for b in range(B) for i in range(M)])
        of = np.repeat(np.arange(B), M)
        at = (table[of, pos // page] * page + pos % page).astype(np.int32)
        qkv = q.qgemm_f8(wi, q.qact_quantize_f8(x), B * M, heads * D, W).view(B * M, heads, D)
        a, b = fu.quantize_rows(_np(x))[0], fu.quantize_weights(w_in)[0]
        fu.assert_close(_np(qkv).reshape(B * M, -1), a @ b.T, fu.sum_bound(np.abs(a) @ np.abs(b).T, W), "qkv")
        qh, kh, vh = qkv.split((H, KV, KV), 1)
        y = q.qkv_norm_rope_write(cache, qh, kh, vh, to_dev(at), to_dev(pos.astype(np.int32)), to_dev(freq), gq, gk,
                                  dtype=torch.bfloat16)
        cos, sin = au.turns(pos, freq, [D // 2])
        n, ref = au.norm(_np(qh), _np(gq), EPS)[0], au.norm_rope(_np(qh), _np(gq), EPS, cos, sin, D, False)
        fu.assert_close(_np(y), ref, au.heads_bound(n, ref, D, False, "bfloat16"), "q")
        kk, vv = (_np(t) for t in q.qkv_read(cache, to_dev(at)))
        ref = au.norm_rope(_np(kh), _np(gk), EPS, cos, sin, D, False)
        if name == "f8":
            assert np.array_equal(kk, au.held(ref, name)[0])
        else:
            n = au.norm(_np(kh), _np(gk), EPS)[0]
            fu.assert_close(kk, ref, au.heads_bound(n, ref, D, False, name), "k")
        assert np.array_equal(vv, au.held(_np(vh), name)[0])
        held_k[at], held_v[at] = kk, vv
        o = q.qattn_decode(cache, y.view(B, M, H, D), d_table, to_dev(lens.astype(np.int32)))
        ref, bound = au.attend(_np(y).reshape(B, M, H, D), held_k, held_v, table, lens, page, pages, D ** -0.5)
        au.assert_attend(_np(o), ref, bound, "bfloat16", "attention")
        out = q.qgemm_f8(wo, q.qact_quantize_f8(o.view(B * M, H * D)), B * M, W, H * D)
        a, b = fu.quantize_rows(_np(o).reshape(B * M, -1))[0], fu.quantize_weights(w_out)[0]
        fu.assert_close(_np(out), a @ b.T, fu.sum_bound(np.abs(a) @ np.abs(b).T, H * D), "out")
    kk, vv = au.unpack(cache.data.cpu().numpy(), page, KV, D, name)
    written = np.unique(np.concatenate([slots, at]))
    assert np.array_equal(kk[written], held_k[written]) and np.array_equal(vv[written], held_v[written])


@pytest.mark.parametrize("axes", [1, 3])
def test_norm_rope_as_an_autograd_function(axes):
    """Shared by a loss on both results, with the gradients of one packed projection, against torch in binary64."""
    q, torch = qg(), torch_cuda()
    T, H, KV, D, rot = 50, 3, 1, 96, 64
    rng = np.random.default_rng(axes)
    pos = to_dev(rng.integers(0, 5000, (axes, T)).astype(np.int32))
    sections = [8, 12, 12] if axes == 3 else [32]
    freq = to_dev(_freq(rot))
    how = dict(sections=sections if axes == 3 else None, interleaved=True)
    p = pos if axes == 3 else pos[0]

    class NormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, qkv, gq, gk):
            ctx.save_for_backward(qkv, gq, gk)
            return q.qhead_norm_rope(qkv[:, :H], qkv[:, H:], p, freq, gq, gk, **how)

        @staticmethod
        def backward(ctx, dq, dk):
            qkv, gq, gk = ctx.saved_tensors
            d = torch.empty_like(qkv)
            grads = q.qhead_norm_rope_backward(dq.contiguous(), dk.contiguous(), qkv[:, :H], qkv[:, H:], p, freq, gq,
                                               gk, out=(d[:, :H], d[:, H:]), **how)
            return d, grads[2], grads[3]

    leaves = [to_dev(rng.normal(size=s).astype(np.float32)).requires_grad_() for s in ((T, H + KV, D), (D,), (D,))]
    w = to_dev(rng.normal(size=(T, H + KV, D)).astype(np.float32))

    def loss(yq, yk, w):
        return (torch.cat([yq, yk], 1) * w).sum()

    loss(*NormRope.apply(*leaves), w).backward()
    refs = [t.detach().double().cpu().requires_grad_() for t in leaves]
    cos, sin = (torch.from_numpy(t) for t in au.turns(_np(pos), _np(freq), sections))
    x = refs[0] * torch.rsqrt((refs[0] ** 2).mean(-1, keepdim=True) + float(np.float32(EPS)))
    gains = torch.cat([refs[1].expand(H, D), refs[2].expand(KV, D)])
    x = x * gains
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)
    loss(y[:, :H], y[:, H:], w.detach().double().cpu()).backward()
    for got, ref in zip(leaves, refs):
        err = (got.grad.double().cpu() - ref.grad).abs().max()
        # every term carries under 64 roundings of 2^-24 (the forward's 16, four times over); gains sum T heads of them
        assert err <= 64 * 2.0 ** -24 * 50 * float(ref.grad.abs().max()), float(err)


# ------------------------------------------------------------ captured graphs
def _capture(torch, run):
    run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            out = run()
    torch.cuda.current_stream().wait_stream(side)
    return g, out


@pytest.mark.parametrize("longest", [60, 4000])
def test_a_captured_step_follows_its_inputs(longest):
    """One graph of a whole step, replayed with other projections, slots, positions and lengths, the program's own
    eager work and synchronizations in between; a second graph of the same cache runs between the replays."""
    q, torch = qg(), torch_cuda()
    rng = np.random.default_rng(longest)
    B, H, KV, D, page = 3, 8, 2, 128, 64
    W = -(-longest // page)
    pages = B * W
    cache = q.qkv_cache(pages, page, KV, D)
    n = pages * page
    fill = torch.randn(n, KV, D, device="cuda", dtype=torch.bfloat16)
    q.qkv_write(cache, fill, fill.flip(0), torch.arange(n, dtype=torch.int32, device="cuda"))
    table = to_dev(rng.permutation(pages).reshape(B, W).astype(np.int32))
    gains = [torch.rand(D, device="cuda") + 0.5 for _ in "qk"]
    freq = to_dev(_freq(D))
    qkv = torch.empty(B, H + 2 * KV, D, device="cuda")
    pos, slots, lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))

    def step():
        a, b, c = qkv.split((H, KV, KV), 1)
        y = q.qkv_norm_rope_write(cache, a, b, c, slots, pos, freq, *gains, dtype=torch.bfloat16)
        return y, q.qattn_decode(cache, y, table, lens)

    def feed(seed):
        g = np.random.default_rng(seed)
        ln = g.integers(1, longest + 1, B)
        ln[seed % B] = longest if seed % 2 else 1
        qkv.copy_(torch.randn(qkv.shape, device="cuda"))
        p = ln - 1
        pos.copy_(to_dev(p.astype(np.int32)))
        lens.copy_(to_dev(ln.astype(np.int32)))
        t = table.cpu().numpy()
        slots.copy_(to_dev(np.array([t[b, p[b] // page] * page + p[b] % page for b in range(B)], np.int32)))

    feed(0)
    graph, out = _capture(torch, step)
    ones = torch.ones(B, H, D, device="cuda", dtype=torch.bfloat16)
    other, _ = _capture(torch, lambda: q.qattn_decode(cache, ones, table, lens, window=7))
    for seed in range(1, 6):
        feed(seed)
        before = cache.data.clone()
        want = [t.clone() for t in step()]
        after = cache.data.clone()
        cache.data.copy_(before)
        for t in out:
            t.fill_(float("nan"))
        other.replay()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), seed
        assert torch.equal(cache.data, after)


def test_captured_training_calls():
    q, torch = qg(), torch_cuda()
    T, H, KV, D = 300, 4, 2, 128
    x = torch.randn(T, H + KV, D, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(T, H + KV, D, device="cuda", dtype=torch.bfloat16)
    g = [torch.rand(D, device="cuda") for _ in "qk"]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freq = to_dev(_freq(D))

    def run():
        y = q.qhead_norm_rope(x[:, :H], x[:, H:], pos, freq, *g)
        d = q.qhead_norm_rope_backward(dy[:, :H], dy[:, H:], x[:, :H], x[:, H:], pos, freq, *g)
        return list(y) + list(d)

    graph, out = _capture(torch, run)
    for _ in range(4):
        x.copy_(torch.randn(x.shape, device="cuda"))
        want = [t.clone() for t in run()]
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


# ---------------------------------------------------------- streams and sizes
def test_calls_on_two_streams_at_once():
    q, torch = qg(), torch_cuda()
    rng = np.random.default_rng(3)
    B, H, KV, D, page, W = 4, 8, 2, 128, 16, 300
    sets = []
    for s in range(2):
        cache = q.qkv_cache(B * W, page, KV, D)
        kv = torch.randn(B * W * page, KV, D, device="cuda", dtype=torch.bfloat16)
        q.qkv_write(cache, kv, kv.flip(0), torch.arange(B * W * page, dtype=torch.int32, device="cuda"))
        table = to_dev(rng.permutation(B * W).reshape(B, W).astype(np.int32))
        lens = to_dev(rng.integers(1, W * page, B).astype(np.int32))
        x = torch.randn(B, H, D, device="cuda", dtype=torch.bfloat16)
        sets.append((cache, x, table, lens, q.qattn_decode(cache, x, table, lens)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, (st, (cache, x, table, lens, _)) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(st):
                got[i].append(q.qattn_decode(cache, x, table, lens))
    torch.cuda.synchronize()
    for g, s in zip(got, sets):
        assert all(torch.equal(t, s[4]) for t in g)


def test_cache_beyond_four_gib():
    """Pages far behind 2^32 bytes, written, read back and attended to."""
    q, torch = qg(), torch_cuda()
    KV, D, page = 8, 256, 1024
    nb = q.qkv_page_bytes(page, KV, D, torch.bfloat16)
    pages = (5 << 30) // nb
    cache = q.KVCache(torch.zeros(pages, nb, dtype=torch.uint8, device="cuda"), page, KV, D, torch.bfloat16)
    n = 1500
    table = np.array([[pages - 1, 0], [pages // 2, pages - 2]])
    slots = np.concatenate([[t[p // page] * page + p % page for p in range(n)] for t in table]).astype(np.int32)
    k, v = (torch.randn(2 * n, KV, D, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    q.qkv_write(cache, k, v, to_dev(slots))
    kk, vv = q.qkv_read(cache, to_dev(slots), dtype=torch.bfloat16)
    assert torch.equal(kk, k) and torch.equal(vv, v)
    x = torch.randn(2, KV * 2, D, device="cuda", dtype=torch.bfloat16)
    got = q.qattn_decode(cache, x, to_dev(table.astype(np.int32)), to_dev(np.array([n, n - 1], np.int32)))
    places = np.arange(2 * n).reshape(2, n)          # the same tokens in pages of one
    ref, bound = au.attend(_np(x)[:, None], _np(k), _np(v), places, [n, n - 1], 1, 2 * n, D ** -0.5)
    au.assert_attend(_np(got)[:, None], ref, bound, "bfloat16", "far pages")


def test_heads_beyond_two_gib_of_elements():
    """Tokens far apart: offsets of elements beyond 2^31, in and out, forward and backward."""
    q, torch = qg(), torch_cuda()
    T, H, D = 5, 2, 64
    gap = 600_000_000
    wide = torch.zeros(gap * (T - 1) + H * D, device="cuda", dtype=torch.bfloat16)
    x = wide.as_strided((T, H, D), (gap, D, 1))
    x.copy_(torch.randn(T, H, D, device="cuda"))
    small = x.contiguous()
    pos, freq, g = torch.arange(T, dtype=torch.int32, device="cuda"), to_dev(_freq(D)), torch.rand(D, device="cuda")
    want = q.qhead_norm_rope(small, None, pos, freq, g)[0]
    dwant = q.qhead_norm_rope_backward(small, None, small, None, pos, freq, g)
    assert torch.equal(q.qhead_norm_rope(x, None, pos, freq, g)[0], want)
    dgot = q.qhead_norm_rope_backward(x, None, x, None, pos, freq, g)
    assert torch.equal(dgot[0], dwant[0]) and torch.equal(dgot[2], dwant[2])
    q.qhead_norm_rope(x, None, pos, freq, g, out=(x, None))
    assert torch.equal(x, want)


def test_large_outputs_are_the_small_ones():
    """The stores that go past the caches (outputs from 64 MiB on) against portions of the same call."""
    q, torch = qg(), torch_cuda()
    T, H, KV, D = 4200, 48, 16, 128
    x = torch.randn(T, H + KV, D, device="cuda", dtype=torch.bfloat16)
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), to_dev(_freq(D))
    g = [torch.rand(D, device="cuda") for _ in "qk"]
    for dtype in (torch.bfloat16, torch.float32):
        y = q.qhead_norm_rope(x[:, :H], x[:, H:], pos, freq, *g, dtype=dtype)
        d = q.qhead_norm_rope_backward(*y, x[:, :H], x[:, H:], pos, freq, *g)
        for a in range(0, T, 1000):
            part = slice(a, a + 1000)
            z = q.qhead_norm_rope(x[part, :H], x[part, H:], pos[part], freq, *g, dtype=dtype)
            e = q.qhead_norm_rope_backward(*z, x[part, :H], x[part, H:], pos[part], freq, *g)
            assert all(torch.equal(s[part], t) for s, t in zip(y, z))
            assert all(torch.equal(s[part], t) for s, t in zip(d[:2], e[:2]))
    cache = q.qkv_cache(T // 16 + 1, 16, KV, D)
    slots = torch.randperm(T, device="cuda").to(torch.int32)
    q.qkv_write(cache, x[:, :KV], x[:, KV:2 * KV], slots)
    k, v = q.qkv_read(cache, slots)
    for a in range(0, T, 1000):
        part = slice(a, a + 1000)
        kk, vv = q.qkv_read(cache, slots[part])
        assert torch.equal(k[part], kk) and torch.equal(v[part], vv)


def test_another_device_than_the_current_one():
    torch = torch_cuda()
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    q = qg()
    with torch.cuda.device(0):
        cache = q.qkv_cache(4, 16, 2, 64, device="cuda:1")
        x = torch.randn(3, 2, 64, device="cuda:1", dtype=torch.bfloat16)
        slots = torch.arange(3, dtype=torch.int32, device="cuda:1")
        q.qkv_write(cache, x, x, slots)
        k, _ = q.qkv_read(cache, slots)
        with pytest.raises(ValueError):
            q.qkv_write(cache, x.to("cuda:0"), x, slots)
        assert k.device == x.device and (k - x.float()).abs().max() < 0.5
