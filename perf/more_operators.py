"""The attention step's operators of the library, with their plain forms.

Between a layer's qkv projection and its output projection: norms of the query
and key heads with the rotation of positions, a paged cache that is quantised
as it is written, and attention of new tokens over it.

Operators (``case["op"]``):
  norm_rope  each head's RMS norm with a gain and the rotation of its first
             `rot` dimensions (halves or neighbours; one to three position
             axes) in one pass; with "train" the gradient as well
  write      the same for a projection's output, with the keys and values
             quantised into the paged cache in the same launch; the new
             tokens are read back
  cache      keys and values written into the paged cache and read back
  attend     one to 16 new tokens of each sequence over the paged cache,
             with a window and a tanh cap of the scores where the case has them

Cache: uint8 [pages][bytes of a page].  A page holds `page` tokens of every
head: codes [head][K, V][token][dim], then for f8 the scale bytes (e + 127)
[head][K, V][token], rounded up to 256 bytes.  f8: OCP e4m3 codes with one
power of two a token and head, the smallest 2^e with |v| <= 448 * 2^e.
"""
import math
import random

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2, "f8": 1}
EPS = 1e-6


# --------------------------------------------------------------------- cases
def listed():
    return [
        # decode of five sequences, straight from the projection's 32-bit output: latency
        dict(name="norm_rope decode", op="norm_rope", t=5, hq=32, hk=8, d=128, rot=128, neighbours=False, axes=1,
             norm=True, x="fp32", y="bf16", train=False),
        # a training batch, forward and backward
        dict(name="norm_rope batch", op="norm_rope", t=16384, hq=32, hk=8, d=128, rot=128, neighbours=False, axes=1,
             norm=True, x="bf16", y="bf16", train=True),
        # ragged image and video tokens with time, height and width, part of a head rotated
        dict(name="norm_rope video", op="norm_rope", t=2731, hq=14, hk=2, d=96, rot=64, neighbours=True, axes=3,
             norm=True, x="fp16", y="fp16", train=True),
        # a decode step of 64 sequences into an 8-bit cache
        dict(name="write decode", op="write", t=64, hq=32, hk=8, d=128, rot=128, neighbours=False, axes=1, norm=True,
             x="fp32", y="bf16", cache="f8", page=64),
        # a prompt without norms into a 16-bit cache of small pages
        dict(name="write prompt", op="write", t=8192, hq=40, hk=8, d=128, rot=128, neighbours=False, axes=1,
             norm=False, x="bf16", y="bf16", cache="bf16", page=16),
        # a long prompt's keys and values, and a later prompt reading them back
        dict(name="cache prompt", op="cache", t=16384, hk=8, d=128, x="bf16", cache="f8", page=64, y="bf16"),
        # odd head counts and dimension, padding among the tokens
        dict(name="cache odd", op="cache", t=777, hk=3, d=192, x="fp32", cache="f8", page=32, y="fp32"),
        # one short sequence: latency
        dict(name="attend short", op="attend", b=1, m=1, hq=32, hk=8, d=128, longest=333, cache="f8", page=64,
             q="bf16", window=0, cap=0.0),
        # one sequence with a long context
        dict(name="attend long", op="attend", b=1, m=1, hq=32, hk=8, d=128, longest=262143, cache="f8", page=64,
             q="bf16", window=0, cap=0.0),
        # a ragged batch over a 16-bit cache of small pages
        dict(name="attend batch", op="attend", b=64, m=1, hq=32, hk=8, d=128, longest=8190, cache="bf16", page=16,
             q="bf16", window=0, cap=0.0),
        # drafted tokens verified: five new tokens a sequence, six query heads a key head
        dict(name="attend verify", op="attend", b=16, m=5, hq=48, hk=8, d=128, longest=16001, cache="f8", page=128,
             q="fp16", window=0, cap=0.0),
        # a layer with a window and capped scores, wide heads of their own
        dict(name="attend window", op="attend", b=33, m=1, hq=16, hk=16, d=256, longest=5003, cache="fp16", page=32,
             q="fp16", window=1000, cap=50.0),
    ]


def _log(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def _heads(rng, most):
    hk = rng.choice([h for h in (1, 2, 3, 4, 5, 8, 12, 16) if h <= most])
    return hk * rng.choice([g for g in (1, 2, 3, 4, 5, 6, 8, 12, 16) if hk * g <= most]), hk


def draw(rng):
    op = rng.choice(["norm_rope", "write", "cache", "attend", "attend"])
    if op in ("norm_rope", "write"):
        hq, hk = _heads(rng, 40)
        d = rng.choice([64, 80, 96, 128, 256] if op == "norm_rope" else [64, 128, 192, 256])
        x = rng.choice(["fp32", "bf16", "fp16"])
        axes = rng.choice([1, 1, 2, 3])
        case = dict(op=op, t=_log(rng, 1, (1 << 24) // (hq * d)), hq=hq, hk=hk, d=d,
                    rot=rng.choice([d, d, d // 16 * 8, 32, 0]), neighbours=rng.random() < 0.4, axes=axes,
                    norm=rng.random() < 0.7, x=x, y=rng.choice([x, "bf16", "fp16"]))
        if case["rot"] == 0:
            case["axes"] = 1
        if op == "norm_rope":
            return dict(case, train=rng.random() < 0.6)
        case["y"] = rng.choice(["bf16", "fp16"])
        return dict(case, cache=rng.choice(["f8", "f8", "bf16", "fp16"]), page=rng.choice([16, 32, 64, 128, 256]))
    if op == "cache":
        hk, d = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128, 192, 256])
        return dict(op=op, t=_log(rng, 1, (1 << 24) // (hk * d)), hk=hk, d=d, x=rng.choice(["fp32", "bf16", "fp16"]),
                    cache=rng.choice(["f8", "f8", "bf16", "fp16"]), page=rng.choice([16, 32, 64, 128, 256]),
                    y=rng.choice(["fp32", "bf16", "fp16"]))
    hq, hk = _heads(rng, 64)
    d, cache = rng.choice([64, 128, 192, 256]), rng.choice(["f8", "f8", "bf16", "fp16"])
    b, m = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 4, 5, 8, 16])
    longest = _log(rng, 1, max(1, min(200000, (400 << 20) // (b * hk * d * SIZE[cache]), (64 << 20) // (b * hq * m))))
    window = 0 if rng.random() < 0.7 else _log(rng, 1, 4096)
    return dict(op=op, b=b, m=m, hq=hq, hk=hk, d=d, longest=longest, cache=cache, page=rng.choice([16, 32, 64, 128, 256]),
                q=cache if cache != "f8" else rng.choice(["bf16", "fp16"]), window=window,
                cap=0.0 if rng.random() < 0.7 else rng.choice([15.0, 30.0, 50.0]))


def _lengths(case):
    """Tokens in the cache of each sequence, the new ones among them: short ones more often than long ones, an empty
    place of the batch among many."""
    b, longest = case["b"], case["longest"]
    lens = [max(1, round(longest * ((i + 1) / b) ** 1.5)) for i in range(b)]
    if b >= 8:
        lens[0] = 0
    return lens


def work(case):
    """Each input read and each output written once; two operations for a product and its sum."""
    op, d = case["op"], case["d"]
    if op == "attend":
        m, hq, hk, window = case["m"], case["hq"], case["hk"], case["window"]
        seen = [min(n, window + m - 1) if window else n for n in _lengths(case)]
        pairs = sum(min(max(0, n - m + 1 + i), window or n) for n in _lengths(case) for i in range(m))
        token = 2 * hk * (d * SIZE[case["cache"]] + (case["cache"] == "f8"))
        return {"bytes": sum(seen) * token + 2 * case["b"] * m * hq * d * SIZE[case["q"]], "flops": 4 * pairs * hq * d}
    t, hk = case["t"], case["hk"]
    kv = 2 * t * hk * d
    if op == "cache":
        return {"bytes": kv * (SIZE[case["x"]] + 2 * SIZE[case["cache"]] + SIZE[case["y"]]), "flops": 4 * kv}
    q = t * case["hq"] * d
    if op == "write":
        return {"bytes": q * (SIZE[case["x"]] + SIZE[case["y"]]) + kv * (SIZE[case["x"]] + 2 * SIZE[case["cache"]] + 4),
                "flops": 10 * q + 10 * kv}
    x, y, n = SIZE[case["x"]], SIZE[case["y"]], q + t * hk * d
    return {"bytes": n * (x + y) + (n * (2 * x + y) if case["train"] else 0), "flops": n * (30 if case["train"] else 10)}


# -------------------------------------------------------------------- inputs
def _two(e):
    """2^e as fp32, -126 <= e <= 127, by its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scaled(v, e):
    """v 2^e in two exact steps."""
    half = e.to(torch.int32) // 2
    return v * _two(half).to(v.dtype) * _two(e.to(torch.int32) - half).to(v.dtype)


def _exponent(v):
    """Of each last-axis vector: the smallest e with |v| <= 448 * 2^e, 0 for zeros."""
    fr, e = torch.frexp(v.abs().amax(-1, keepdim=True))
    return torch.where(fr > 0, e - 9 + (fr > 0.875), 0).clamp(-127, 120)


def _page_bytes(page, heads, d, cache):
    n = 2 * heads * page * d * SIZE[cache] + (2 * heads * page if cache == "f8" else 0)
    return (n + 255) // 256 * 256


def _pages(kv, page, cache):
    """Values [pages][K, V][page][heads][d] as cache pages."""
    pages, _, _, heads, d = kv.shape
    out = torch.zeros(pages, _page_bytes(page, heads, d, cache), dtype=torch.uint8, device="cuda")
    v = kv.permute(0, 3, 1, 2, 4)
    end = 2 * heads * page * d * SIZE[cache]
    if cache == "f8":
        e = _exponent(v)
        out[:, :end] = _scaled(v, -e).to(torch.float8_e4m3fn).reshape(pages, -1).view(torch.uint8)
        out[:, end:end + 2 * heads * page] = (e + 127).to(torch.uint8).reshape(pages, -1)
    else:
        out[:, :end] = v.to(TYPES[cache]).reshape(pages, -1).view(torch.uint8)
    return out


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 31) + 29)


def _projection(g, t, heads, d, dtype):
    """What a projection gives: some channels wider than others, heads and tokens of differing size."""
    x = torch.randn(t, heads, d, generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn(1, heads, d, generator=g, device="cuda"))
    x *= torch.exp(0.3 * torch.randn(t, 1, 1, generator=g, device="cuda"))
    return x.to(TYPES[dtype])


def _sections(case):
    """Pairs of dimensions of each position axis: time has the fewest."""
    n, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return [n]
    first = n // (axes + 1)
    rest = n - first
    return [first] + [rest // (axes - 1) + (i < rest % (axes - 1)) for i in range(axes - 1)]


def _slots(g, t, slots):
    """Places of t new tokens in the cache, some of them padding (-1)."""
    s = torch.randperm(slots, generator=g, device="cuda")[:t].to(torch.int32)
    if t > 4:
        s[torch.rand(t, generator=g, device="cuda") < 0.02] = -1
    return s


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op, d, hk = case["op"], case["d"], case["hk"]
    if op == "attend":
        b, page = case["b"], case["page"]
        lens = _lengths(case)
        random.Random(seed).shuffle(lens)
        width = max(1, (max(lens) + page - 1) // page)
        used = [(n + page - 1) // page for n in lens]
        pages = sum(used) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(used):
            table[i, :n] = order[at:at + n]
            at += n
        step = max(1, (1 << 26) // (2 * page * hk * d))
        wide = torch.exp(0.5 * torch.randn(2, 1, hk, d, generator=g, device="cuda"))
        parts = []
        for a in range(0, pages, step):
            kv = torch.randn(min(step, pages - a), 2, page, hk, d, generator=g, device="cuda") * wide
            kv[:, 1] *= torch.exp(0.5 * torch.randn(kv.shape[0], page, hk, 1, generator=g, device="cuda"))
            parts.append(_pages(kv, page, case["cache"]))
        s["data"] = torch.cat(parts)
        s["table"] = table
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = torch.randn(b, case["m"], case["hq"], d, generator=g, device="cuda")
        q *= torch.exp(0.5 * torch.randn(b, case["m"], case["hq"], 1, generator=g, device="cuda"))
        s["q_in"] = q.to(TYPES[case["q"]])
        return s
    t = case["t"]
    if op in ("cache", "write"):
        pages = (t + t // 8) // case["page"] + 2
        s["data"] = torch.zeros(pages, _page_bytes(case["page"], hk, d, case["cache"]), dtype=torch.uint8,
                                device="cuda")
        s["slots"] = _slots(g, t, pages * case["page"])
    if op == "cache":
        s["k_in"] = _projection(g, t, hk, d, case["x"])
        s["v_in"] = _projection(g, t, hk, d, case["x"])
        return s
    hq, rot = case["hq"], case["rot"]
    s["qkv"] = _projection(g, t, hq + 2 * hk, d, case["x"])
    if case["axes"] == 1:
        s["pos"] = torch.randint(0, 1 << 17, (t,), generator=g, device="cuda", dtype=torch.int32)
    else:
        s["pos"] = torch.randint(0, 4096, (case["axes"], t), generator=g, device="cuda", dtype=torch.int32)
    s["freq"] = torch.exp(-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / max(rot, 1) *
                          math.log(500000.0)).float()
    s["gq"] = s["gk"] = None
    if case["norm"]:
        s["gq"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["gk"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    if case.get("train"):
        s["dq"] = (torch.randn(t, hq, d, generator=g, device="cuda") * 1e-2).to(TYPES[case["y"]])
        s["dk"] = (torch.randn(t, hk, d, generator=g, device="cuda") * 1e-2).to(TYPES[case["y"]])
    return s


# --------------------------------------------------------------- plain forms
def _turn(s, dtype):
    """cos and sin [t][1][rot / 2]; angles of far positions in 64 bits."""
    pos = s["pos"].view(s["axes"], s["t"]).double()
    axis = torch.repeat_interleave(torch.arange(s["axes"], device="cuda"),
                                   torch.tensor(_sections(s), device="cuda"))
    angle = pos[axis].T * s["freq"].double()
    return torch.cos(angle).to(dtype)[:, None], torch.sin(angle).to(dtype)[:, None]


def _rotate(y, cos, sin, rot, neighbours):
    out = y.clone()
    if rot:
        at = (slice(0, rot, 2), slice(1, rot, 2)) if neighbours else (slice(0, rot // 2), slice(rot // 2, rot))
        a, b = y[..., at[0]], y[..., at[1]]
        out[..., at[0]] = a * cos - b * sin
        out[..., at[1]] = b * cos + a * sin
    return out


def _heads_forward(s, x, gain, dtype=torch.float32):
    x = x.to(dtype)
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.to(dtype)
    cos, sin = _turn(s, dtype)
    return _rotate(x, cos, sin, s["rot"], s["neighbours"])


def _heads_backward(s, x, dy, gain):
    cos, sin = _turn(s, torch.float32)
    h = _rotate(dy.float(), cos, -sin, s["rot"], s["neighbours"])
    if gain is None:
        return h.to(x.dtype), None
    r = torch.rsqrt((x.float() * x.float()).mean(-1, keepdim=True) + EPS)
    n = x.float() * r
    dg = (h * n).sum((0, 1), dtype=torch.float64).float()
    h = h * gain
    return (r * (h - n * (h * n).mean(-1, keepdim=True))).to(x.dtype), dg


def _held(v, cache):
    """What the cache holds of vectors v, fp32."""
    if cache != "f8":
        return v.to(TYPES[cache]).float()
    e = _exponent(v)
    v = _scaled(v, -e)
    step = torch.frexp(v)[1].clamp(min=-5) - 4         # a code's last place: four bits of significand, from 2^-6 up
    return _scaled(_scaled(torch.round(_scaled(v, -step)), step), e).float()


def _back(held, s, dtype):
    """Written to the cache's slots and read from them again; nothing at -1."""
    return torch.where((s["slots"] >= 0)[:, None, None], held, 0.0).to(dtype)


def _table_values():
    c = torch.arange(256, device="cuda")
    ex, ma = (c >> 3) & 15, c & 7
    v = torch.where(ex > 0, (1 + ma / 8) * _two(ex - 7), ma / 512)
    return torch.where(c >= 128, -v, v)


def _tokens(s, pages):
    """Cache pages [...] as fp32 values [..., K or V, page, heads, d]."""
    page, hk, d, cache = s["page"], s["hk"], s["d"], s["cache"]
    raw = s["data"][pages]
    lead, end = raw.shape[:-1], 2 * hk * page * d * SIZE[cache]
    if cache == "f8":
        v = _table_values()[raw[..., :end].int()].view(*lead, hk, 2, page, d)
        e = raw[..., end:end + 2 * hk * page].view(*lead, hk, 2, page, 1).int() - 127
        v = _scaled(v, e)
    else:
        v = raw[..., :end].contiguous().view(TYPES[cache]).view(*lead, hk, 2, page, d).float()
    return v.movedim(-4, -2)


def _plain_attend(s):
    b, m, hq, hk, d = s["b"], s["m"], s["hq"], s["hk"], s["d"]
    out = torch.empty(b, m, hq, d, dtype=s["q_in"].dtype, device="cuda")
    n = s["table"].shape[1] * s["page"]
    step = max(1, (1 << 29) // (n * max(hk * d, hq * m)))
    for a in range(0, b, step):
        kv = _tokens(s, s["table"][a:a + step].clamp(min=0).long())       # [b][width][2][page][hk][d]
        c = kv.shape[0]
        kv = kv.permute(2, 0, 4, 1, 3, 5).reshape(2, c, hk, n, d)
        q = s["q_in"][a:a + step].float().view(c, m, hk, hq // hk, d).transpose(1, 2).reshape(c, hk, -1, d)
        x = torch.matmul(q, kv[0].transpose(2, 3)).view(c, hk, m, hq // hk, n) / math.sqrt(d)
        if s["cap"]:
            x = s["cap"] * torch.tanh(x / s["cap"])
        last = s["lens"][a:a + step, None] - m + torch.arange(m, device="cuda")          # the query's own position
        at = torch.arange(n, device="cuda")
        seen = at <= last[..., None]
        if s["window"]:
            seen &= at > last[..., None] - s["window"]
        seen = seen[:, None, :, None]
        x = torch.where(seen, x, -math.inf)
        big = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(big > -math.inf, big, 0.0))
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
        y = torch.matmul(p.view(c, hk, -1, n), kv[1]).view(c, hk, m, hq // hk, d)
        out[a:a + step] = y.transpose(1, 2).reshape(c, m, hq, d)
    return out


def _plain(s):
    op, hk = s["op"], s["hk"]
    if op == "attend":
        return _plain_attend(s)
    if op == "cache":
        y = TYPES[s["y"]]
        return _back(_held(s["k_in"].float(), s["cache"]), s, y), _back(_held(s["v_in"].float(), s["cache"]), s, y)
    hq, y = s["hq"], TYPES[s["y"]]
    q, k = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hk]
    if op == "write":
        # codes are cut at borders: the keys in 64 bits
        k = _heads_forward(s, k, s["gk"], torch.float64 if s["cache"] == "f8" else torch.float32)
        v = s["qkv"][:, hq + hk:].float()
        return (_heads_forward(s, q, s["gq"]).to(y), _back(_held(k, s["cache"]), s, torch.float32),
                _back(_held(v, s["cache"]), s, torch.float32))
    out = (_heads_forward(s, q, s["gq"]).to(y), _heads_forward(s, k, s["gk"]).to(y))
    if s["train"]:
        dq, dgq = _heads_backward(s, q, s["dq"], s["gq"])
        dk, dgk = _heads_backward(s, k, s["dk"], s["gk"])
        out += (dq, dk) + ((dgq, dgk) if s["norm"] else ())
    return out


# ----------------------------------------------------------- the own kernels
def _own(s):
    import quantized_weight_gemv_amd as qg
    op, hk = s["op"], s["hk"]
    cache = qg.KVCache(s["data"], s["page"], hk, s["d"], TYPES[s["cache"]]) if op != "norm_rope" else None
    if op == "attend":
        return qg.qattn_decode(cache, s["q_in"], s["table"], s["lens"], window=s["window"], softcap=s["cap"])
    if op == "cache":
        qg.qkv_write(cache, s["k_in"], s["v_in"], s["slots"])
        return qg.qkv_read(cache, s["slots"], dtype=TYPES[s["y"]])
    hq = s["hq"]
    q, k, v = s["qkv"].split((hq, hk, hk), 1)
    how = dict(q_gain=s["gq"], k_gain=s["gk"], eps=EPS, interleaved=s["neighbours"],
               sections=_sections(s) if s["axes"] > 1 else None)
    if op == "write":
        y = qg.qkv_norm_rope_write(cache, q, k, v, s["slots"], s["pos"], s["freq"], dtype=TYPES[s["y"]], **how)
        return (y,) + tuple(qg.qkv_read(cache, s["slots"], dtype=torch.float32))
    out = qg.qhead_norm_rope(q, k, s["pos"], s["freq"], dtype=TYPES[s["y"]], **how)
    if s["train"]:
        dq, dk, dgq, dgk = qg.qhead_norm_rope_backward(s["dq"], s["dk"], q, k, s["pos"], s["freq"], **how)
        out = tuple(out) + (dq, dk) + ((dgq, dgk) if s["norm"] else ())
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ in 64 bits
def _pow2(e):
    """2^e in 64 bits, exact where a power function need not be."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_heads(s, x, gain):
    """Through complex numbers: a pair is a point of the plane, turned by its angle."""
    t, rot, d = s["t"], s["rot"], s["d"]
    y = x
    if gain is not None:
        y = x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt() * gain.double()
    if rot == 0:
        return y
    pos = s["pos"].view(s["axes"], t).double()
    parts, at = [], 0
    for a, n in enumerate(_sections(s)):
        parts.append(pos[a][:, None] * s["freq"][at:at + n].double()[None])
        at += n
    angle = torch.cat(parts, 1)[:, None]
    turn = torch.polar(torch.ones_like(angle), angle)
    if s["neighbours"]:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
        z = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        z = torch.cat((z.real, z.imag), -1)
    return torch.cat((z, y[..., rot:]), -1)


def _exact_held(v, cache):
    """64-bit values as the cache holds them; to 8 bits by the nearest of all codes, ties to the even one."""
    if cache != "f8":
        return v.to(TYPES[cache]).double()
    grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    a = v.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 448))
    e = e - (a <= 448 * _pow2(e - 1)).double()                         # log2 may be off by an ulp
    e = e + (a > 448 * _pow2(e)).double()
    e = torch.where(a > 0, e, 0.0).clamp(-127, 120)
    m = v.abs() * _pow2(-e)
    up = torch.searchsorted(grid, m.contiguous()).clamp(1, 126)
    over, under = grid[up] - m, m - grid[up - 1]
    code = torch.where(over < under, up, torch.where(over > under, up - 1, up + up % 2 * -1))
    return torch.copysign(grid[code], v) * _pow2(e)


def _exact_attend(s):
    b, m, hq, hk, d, page, cache = (s[n] for n in ("b", "m", "hq", "hk", "d", "page", "cache"))
    out = torch.zeros(b, m, hq, d, dtype=torch.float64, device="cuda")
    end = 2 * hk * page * d * SIZE[cache]
    for i, n in enumerate(s["lens"].tolist()):
        first = max(0, n - m + 1 - s["window"]) // page if s["window"] else 0     # pages that nobody sees are left out
        ids = s["table"][i, first:(n + page - 1) // page].long()
        if len(ids) == 0:
            continue
        for h in range(hk):
            at = h * 2 * page * d * SIZE[cache]
            raw = s["data"][ids, at:at + 2 * page * d * SIZE[cache]].view(TYPES[cache]).view(-1, 2, page, d).double()
            if cache == "f8":
                at = end + h * 2 * page
                raw = raw * _pow2(s["data"][ids, at:at + 2 * page].view(-1, 2, page, 1).long() - 127)
            k, v = raw[:, 0].reshape(-1, d), raw[:, 1].reshape(-1, d)
            where = torch.arange(first * page, first * page + len(k), device="cuda")
            g = hq // hk
            for j in range(m):
                own_place = n - m + j
                take = (where <= own_place) & ((where > own_place - s["window"]) if s["window"] else True)
                if not bool(take.any()):
                    continue
                x = k[take] @ s["q_in"][i, j, h * g:(h + 1) * g].double().T.contiguous() * d ** -0.5
                if s["cap"]:
                    x = s["cap"] * torch.tanh(x / s["cap"])
                out[i, j, h * g:(h + 1) * g] = torch.softmax(x, 0).T.contiguous() @ v[take]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, hk = case["op"], case["hk"]
    if op == "attend":
        return _exact_attend(s)
    if op in ("cache", "write"):
        there = (s["slots"] >= 0).double()[:, None, None]
    if op == "cache":
        return tuple(_exact_held(s[n].double(), case["cache"]) * there for n in ("k_in", "v_in"))
    hq = case["hq"]
    q, k, v = (p.double().contiguous() for p in s["qkv"].split((hq, hk, hk), 1))
    if op == "write":
        return (_exact_heads(s, q, s["gq"]), _exact_held(_exact_heads(s, k, s["gk"]), case["cache"]) * there,
                _exact_held(v, case["cache"]) * there)
    if not case["train"]:
        return _exact_heads(s, q, s["gq"]), _exact_heads(s, k, s["gk"])
    gains = [g.double().requires_grad_() for g in (s["gq"], s["gk"])] if case["norm"] else [None, None]
    leaves = [q.requires_grad_(), k.requires_grad_()]
    ys = [_exact_heads(s, x, g) for x, g in zip(leaves, gains)]
    wanted = leaves + [g for g in gains if g is not None]
    grads = torch.autograd.grad(ys, wanted, [s["dq"].double(), s["dk"].double()])
    return tuple(y.detach() for y in ys) + grads
