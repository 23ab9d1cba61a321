"""Norms of head vectors: heads of 192 elements, whose lanes are not all in use, against the binary64 references, and
the bits that separate operations give."""
import numpy as np
import pytest

import test_attn_gpu as base
from gpu_util import qg, to_dev, torch_cuda

pytestmark = pytest.mark.gpu

# (T, query heads, key heads, D, rot, interleaved, axes, gains' type, inputs, outputs)
WIDE = [
    (5, 3, 1, 192, 192, False, 1, "float32", "bfloat16", "bfloat16"),
    (7, 5, 3, 192, 128, False, 1, "bfloat16", "float32", "float32"),
    (3, 1, 2, 192, 192, True, 3, "float32", "float16", "float16"),
    (9, 7, 1, 192, 64, True, 1, "float16", "bfloat16", "float32"),
    (4, 3, 5, 192, 0, False, 1, "float32", "float32", "bfloat16"),
    (300, 2, 1, 192, 96, False, 2, "float32", "bfloat16", "bfloat16"),
    (6, 3, 1, 200, 200, False, 1, "float32", "float32", "float32"),
    (6, 3, 3, 248, 240, True, 1, "bfloat16", "bfloat16", "float32"),
]


@pytest.mark.parametrize("case", WIDE)
def test_norm_rope(case):
    base.test_norm_rope(case)


@pytest.mark.parametrize("case", WIDE)
def test_norm_rope_backward(case):
    base.test_norm_rope_backward(case)


@pytest.mark.parametrize("case,cache,page", [
    (WIDE[0], "f8", 16), (WIDE[1], "f8", 64), (WIDE[2], "f8", 32), (WIDE[3], "f8", 16), (WIDE[4], "f8", 16),
    (WIDE[5], "f8", 128), (WIDE[0], "bfloat16", 16), (WIDE[2], "float16", 32), (WIDE[4], "bfloat16", 16)])
def test_norm_rope_write(case, cache, page):
    base.test_norm_rope_write(case + (cache, page))


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_zeros_between_others(eps):
    """Zeros stay zeros with an eps, as formulas have it NaNs without one; neither reaches another head, and an 8-bit
    cache holds the exact values' codes of the others."""
    q, torch = qg(), torch_cuda()
    rng = np.random.default_rng(4)
    T, D = 5, 192
    x = to_dev(rng.normal(size=(T, 9, D)).astype(np.float32))
    x[2, :, :] = 0
    x[:, 4, :] = 0
    g = to_dev((1 + 0.3 * rng.normal(size=D)).astype(np.float32))
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    cache = q.qkv_cache(1, 16, 3, D)
    y = q.qkv_norm_rope_write(cache, x[:, :3], x[:, 3:6], x[:, 6:], slots, None, None, g, g, eps)
    k = q.qkv_read(cache, slots)[0]
    r = 1 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + float(np.float32(eps)))
    want = (x.double() * r * g.double()).cpu().numpy()
    got = np.concatenate([base._np(y), base._np(k)], 1)
    zero = (x[:, :6] == 0).all(-1).cpu().numpy()
    assert np.isnan(got[zero]).all() if eps == 0 else not got[zero].any()
    want, heads = want[:, :6], np.arange(6)[None] < 3
    n = want[~zero & heads]
    base.fu.assert_close(got[~zero & heads], n, base.au.HEADS * np.abs(n), "q")
    assert np.array_equal(got[~zero & ~heads], base.au.held(want[~zero & ~heads], "f8")[0])


def _separate(x, gain, cos, sin, rot, interleaved):
    """The norm and the rotation by one operation after the other, in fp32."""
    torch = torch_cuda()
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + base.EPS) * gain
    if not rot:
        return x
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_the_bits_of_separate_operations(D, dtype):
    """Squares are summed in the order that a mean over these row lengths takes, the root is the nearest, every
    product rounds by itself, and cosine and sine are the nearest: no bit differs (another order of that mean, in
    another release, shows here)."""
    q, torch = qg(), torch_cuda()
    rng = np.random.default_rng(D)
    for T, H in ((1, 1), (1, 7), (5, 32), (300, 3), (5000, 8)):
        x = rng.normal(size=(T, H, D)) * np.exp(rng.normal(size=(T, H, 1)))
        x = to_dev(x.astype(np.float32)).to(getattr(torch, dtype))
        gain = to_dev((1 + 0.2 * rng.normal(size=D)).astype(np.float32))
        pos = to_dev(rng.integers(0, 1 << 17, T).astype(np.int32))
        for rot, interleaved in ((0, False), (D, False), (D, True), (D // 16 * 8, True), (32, False)):
            freq = to_dev(np.exp(-np.arange(rot // 2) / max(rot // 2, 1) * 13).astype(np.float32))
            angle = pos.double()[:, None, None] * freq.double()
            want = _separate(x, gain, torch.cos(angle).float(), torch.sin(angle).float(), rot, interleaved)
            got = q.qhead_norm_rope(x, None, pos, freq if rot else None, gain, interleaved=interleaved,
                                    dtype=torch.float32)[0]
            assert torch.equal(got, want), (T, H, rot, interleaved)
