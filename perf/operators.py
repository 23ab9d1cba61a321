"""The 8-bit floating point operators of the library, with their plain forms.

f8 values: OCP e4m3 codes (448 the largest) and a power-of-two scale for each
block of 128: 128 x 128 for weights, 128 elements of a row for activations.
The scale of a block is the smallest 2^e with |v| <= 448 * 2^e for all of it
(e = 0 where the block is zero), a code is v / 2^e rounded to nearest, ties to
even.

Operators (``case["op"]``):
  gemv        y = f8(x) W^T, 1 to 8 tokens, x in 16 or 32 bits, y in 32
  gemm        y = f8(x) W^T for a prompt or a training batch, any y type
  moe         the same for tokens sorted by expert: y[slot] = W_e f8(x[slot / k])
  checkpoint  x held as f8 between the passes, and read back
  backward    of y = f8(x) W^T: dx = f8(dy) W, dw = dy^T f8(x) from the 8-bit x
  route       top-k softmax routing with per-expert counts, the slots sorted by
              expert and the balance loss; with "train" the gradient as well
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # decode of one sequence: the latency of one projection
        dict(name="gemv one token", op="gemv", m=1, n=4096, k=4096, x="fp16"),
        # eight sequences decoded together, the stacked gate and up projection
        dict(name="gemv eight tokens", op="gemv", m=8, n=28672, k=4096, x="bf16"),
        # a verification or a small batch of decodes on a projection back to the model width
        dict(name="gemm small batch", op="gemm", m=61, n=4096, k=14336, x="fp16", y="fp32"),
        # a ragged prompt on odd sizes, neither side a multiple of a tile or of a block
        dict(name="gemm odd prompt", op="gemm", m=733, n=2053, k=5011, x="fp32", y="fp16"),
        # a training batch, or a long prompt
        dict(name="gemm batch", op="gemm", m=8192, n=14336, k=4096, x="bf16", y="bf16"),
        # decode of four tokens over a pool of many small experts
        dict(name="moe decode", op="moe", m=4, experts=128, top=10, n=640, k=2560, x="bf16", y="fp32"),
        # a prompt over the same kind of pool; its last tokens are padding
        dict(name="moe prompt", op="moe", m=4001, experts=64, top=6, n=2048, k=2048, x="bf16", y="bf16"),
        # one layer's activations put away for the backward pass and read back
        dict(name="checkpoint", op="checkpoint", m=8192, k=4096, x="bf16"),
        # gradients of a small odd layer
        dict(name="backward odd", op="backward", m=519, n=1288, k=2056),
        # gradients of an attention projection in a training batch
        dict(name="backward batch", op="backward", m=8192, n=6144, k=4096),
        # routing of a few decoded tokens: latency
        dict(name="route decode", op="route", m=4, experts=128, top=10, x="fp32", train=False),
        # routing of a training batch, forward and backward
        dict(name="route train", op="route", m=16384, experts=256, top=8, x="bf16", train=True),
    ]


def _log(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def _size(rng, low, high):
    """A size of the range: one in three odd or ragged, else a multiple of 64."""
    v = _log(rng, low, high)
    return v if rng.random() < 1 / 3 or v < 128 else v // 64 * 64


def draw(rng):
    op = rng.choice(["gemv", "gemm", "moe", "checkpoint", "backward", "route"])
    if op == "gemv":
        return dict(op=op, m=rng.randint(1, 8), n=_size(rng, 256, 28672), k=_size(rng, 256, 8192),
                    x=rng.choice(["fp16", "bf16", "fp32"]))
    if op == "gemm":
        return dict(op=op, m=_size(rng, 1, 8192), n=_size(rng, 256, 7168), k=_size(rng, 128, 7168),
                    x=rng.choice(["fp16", "bf16", "fp32"]), y=rng.choice(["fp32", "fp16", "bf16"]))
    if op == "moe":
        experts = rng.choice([8, 16, 32, 60, 64, 128])
        return dict(op=op, m=_size(rng, 1, 4096), experts=experts, top=rng.randint(1, min(8, experts)),
                    n=_size(rng, 256, 1536), k=_size(rng, 256, 2048), x=rng.choice(["fp16", "bf16"]),
                    y=rng.choice(["fp32", "bf16"]))
    if op == "checkpoint":
        return dict(op=op, m=_size(rng, 1, 8192), k=_size(rng, 100, 8192), x=rng.choice(["fp16", "bf16", "fp32"]))
    if op == "backward":
        return dict(op=op, m=_size(rng, 1, 8192), n=_size(rng, 128, 6144), k=_size(rng, 128, 4096))
    return dict(op=op, m=_log(rng, 1, 16384), experts=_log(rng, 4, 384), top=rng.randint(1, 4),
                x=rng.choice(["fp32", "bf16", "fp16"]), train=rng.random() < 0.5)


def _up(v, to):
    return (v + to - 1) // to * to


def work(case):
    """Each input read and each output written once; two operations for a product and its sum."""
    op, m = case["op"], case["m"]
    size = {"fp32": 4, "fp16": 2, "bf16": 2}
    if op in ("gemv", "gemm"):
        n, k = case["n"], case["k"]
        return {"bytes": n * k + m * k * size[case["x"]] + m * n * size[case.get("y", "fp32")], "flops": 2 * m * n * k}
    if op == "moe":
        n, k, slots = case["n"], case["k"], m * case["top"]
        used = case["experts"] * (1 - (1 - 1 / case["experts"]) ** slots)
        return {"bytes": int(used * n * k) + m * k * size[case["x"]] + slots * n * size[case["y"]],
                "flops": 2 * slots * n * k}
    if op == "checkpoint":
        b = m * case["k"] * size[case["x"]]
        return {"bytes": 2 * b + 2 * m * case["k"], "flops": 6 * m * case["k"]}
    if op == "backward":
        n, k = case["n"], case["k"]
        return {"bytes": n * k + 2 * m * (n + k) + 2 * m * k + 4 * n * k, "flops": 4 * m * n * k}
    b = m * case["experts"] * size[case["x"]]
    return {"bytes": b * (3 if case["train"] else 1) + 12 * m * case["top"], "flops": 8 * m * case["experts"]}


# -------------------------------------------------------------------- inputs
def _two(e):
    """2^e as fp32, -126 <= e <= 127, by its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scaled(v, e):
    """v 2^e, -252 <= e <= 254, in two exact steps."""
    e = e.to(torch.int32)
    half = e // 2
    return v * _two(half) * _two(e - half)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 31) + 17)


def _weights(g, n, k, count=1):
    """`count` packed n x k f8 matrices: values of a normal distribution whose width changes from block to block.

    One matrix: the codes in tiles of 16 rows x 128 columns, tiles of a row block one after the other, a tile as
    [half of 64 columns][16 columns][16 rows][16 columns] bytes; then the scale bytes (e + 127), [row block][column
    block] with rows of a multiple of four bytes; rows, columns and the end (256 bytes) padded with zeros."""
    rb, cb = (n + 127) // 128, (k + 127) // 128
    np_, kp, ls = _up(n, 16), 128 * cb, _up(cb, 4)
    total = _up(np_ * kp + rb * ls, 256)
    packed = torch.zeros(count, total, dtype=torch.uint8, device="cuda")
    for c in range(count):
        w = torch.zeros(128 * rb, kp, device="cuda")
        w[:n, :k] = torch.randn(n, k, generator=g, device="cuda") * 0.02
        blocks = w.view(rb, 128, cb, 128)
        blocks *= torch.exp(0.7 * torch.randn(rb, 1, cb, 1, generator=g, device="cuda"))
        amax = blocks.abs().amax((1, 3))
        m, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - 9 + (m > 0.875), 0)
        codes = _scaled(blocks, -e[:, None, :, None]).view(128 * rb, kp)[:np_].to(torch.float8_e4m3fn)
        tiles = codes.view(torch.uint8).view(np_ // 16, 16, cb, 2, 4, 16).permute(0, 2, 3, 4, 1, 5)
        packed[c, :np_ * kp] = tiles.reshape(-1)
        scales = torch.zeros(rb, ls, dtype=torch.uint8, device="cuda")
        scales[:, :cb] = (e + 127).to(torch.uint8)
        packed[c, np_ * kp:np_ * kp + rb * ls] = scales.view(-1)
    return packed.view(-1) if count == 1 else packed


def _acts(g, m, k, dtype):
    """Activations: some channels are far wider than the others, tokens differ in size."""
    x = torch.randn(m, k, generator=g, device="cuda")
    x *= torch.exp(torch.randn(1, k, generator=g, device="cuda"))
    x *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device="cuda"))
    return x.to(TYPES[dtype])


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op, m = case["op"], case["m"]
    if op == "route":
        logits = torch.randn(m, case["experts"], generator=g, device="cuda") * 1.5
        logits += torch.randn(1, case["experts"], generator=g, device="cuda")
        masked = torch.rand(m, case["experts"], generator=g, device="cuda") < 0.05     # experts closed to a token
        s["logits"] = logits.masked_fill(masked, -math.inf).to(TYPES[case["x"]])
        s["mask"] = (torch.rand(m, generator=g, device="cuda") >= 0.03).to(torch.uint8)   # padding of the batch
        if m > 2:
            s["logits"][m // 2] = -math.inf
        s["grad_weight"] = torch.randn(m, case["top"], generator=g, device="cuda")
        s["grad_loss"] = torch.full((1,), 0.01 * m, device="cuda")
        return s
    k = case["k"]
    s["x_in"] = _acts(g, m, k, case.get("x", "bf16"))
    if op == "moe":
        P, top, n = case["experts"], case["top"], case["n"]
        s["w"] = _weights(g, n, k, P)
        # a skewed choice of `top` different experts for each token; one token in 50 is padding
        score = torch.randn(m, P, generator=g, device="cuda") + 0.5 * torch.randn(1, P, generator=g, device="cuda")
        idx = torch.argsort(score, 1, descending=True)[:, :top].to(torch.int32)
        idx[torch.rand(m, generator=g, device="cuda") < 0.02] = -1
        key = torch.where(idx >= 0, idx, P).view(-1)
        s["order"] = torch.argsort(key, stable=True).to(torch.int32)
        counts = torch.bincount(key, minlength=P + 1)[:P]
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)]).to(torch.int32)
        s["most"] = max(1, int(counts.max()))
    elif op == "backward":
        n = case["n"]
        s["w_t"] = _weights(g, k, n)          # W^T packed: the matrix of dx = f8(dy) W
        s["dy"] = (torch.randn(m, n, generator=g, device="cuda") * 1e-3 *
                   torch.exp(torch.randn(m, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    elif op != "checkpoint":
        s["w"] = _weights(g, case["n"], k)
    return s


# --------------------------------------------------------------- plain forms
def _unpack(packed, n, k):
    """The values of packed matrices [..., bytes] -> fp32 [..., n, k], by the definition of e4m3."""
    rb, cb = (n + 127) // 128, (k + 127) // 128
    np_, kp, ls = _up(n, 16), 128 * cb, _up(cb, 4)
    lead = packed.shape[:-1]
    codes = packed[..., :np_ * kp].reshape(*lead, np_ // 16, cb, 2, 4, 16, 16)
    codes = codes.movedim(-2, -5).reshape(*lead, np_, kp)[..., :n, :k]
    e = packed[..., np_ * kp:np_ * kp + rb * ls].reshape(*lead, rb, ls)[..., :cb].int() - 127
    c = torch.arange(256, device=packed.device)
    ex, ma = (c >> 3) & 15, c & 7
    table = torch.where(ex > 0, (1 + ma / 8) * _two(ex - 7), ma / 512)
    table = torch.where(c >= 128, -table, table)
    v = table[codes.int()]
    return _scaled(v, e.repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k])


def _f8(x):
    """The values of x's f8 form, fp32."""
    m, k = x.shape
    cb = (k + 127) // 128
    v = torch.nn.functional.pad(x.float(), (0, 128 * cb - k)).view(m, cb, 128)
    fr, e = torch.frexp(v.abs().amax(2, keepdim=True))
    e = torch.where(fr > 0, e - 9 + (fr > 0.875), 0).clamp(-127, 127)
    v = _scaled(v, -e)
    step = torch.frexp(v)[1].clamp(min=-5) - 4         # a code's last place: four bits of significand, from 2^-6 up
    q = _scaled(torch.round(_scaled(v, -step)), step)
    return _scaled(q, e).view(m, 128 * cb)[:, :k]


def _plain_moe(s):
    n, k, P, top = s["n"], s["k"], s["experts"], s["top"]
    x, order, offsets = _f8(s["x_in"]), s["order"].long(), s["offsets"].long()
    slots, most = order.numel(), s["most"]
    row = torch.arange(slots, device="cuda")
    e = (row[:, None] >= offsets[None, 1:]).sum(1)                  # P: no expert
    y = torch.zeros(slots, n, device="cuda")
    live = (e < P)[:, None]
    if slots * 2 <= P:
        w = _unpack(s["w"][e.clamp(max=P - 1)], n, k)
        rows = torch.bmm(w, x[order // top][:, :, None])[:, :, 0]
    else:
        at = e.clamp(max=P - 1) * most + torch.where(e < P, row - offsets[e.clamp(max=P - 1)], 0)
        xs = torch.zeros(P * most, k, device="cuda")
        xs.index_add_(0, at, torch.where(live, x[order // top], 0.0))
        w = _unpack(s["w"], n, k).transpose(1, 2).contiguous()
        rows = torch.bmm(xs.view(P, most, k), w).view(P * most, n)[at]
    y[order] = torch.where(live, rows, 0.0)
    return y.to(TYPES[s["y"]])


def _plain_route(s):
    E, top, m = s["experts"], s["top"], s["m"]
    x = s["logits"].float()
    open_ = (x > -math.inf) & (s["mask"] != 0)[:, None]
    live = open_.any(1, keepdim=True)
    x = torch.where(open_, x, -math.inf)
    big = torch.where(live, x.amax(1, keepdim=True), 0.0)
    p = torch.exp(x - big)
    p = torch.where(live, p / p.sum(1, keepdim=True), 0.0)
    idx = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :top]
    chosen = open_.gather(1, idx)
    raw = torch.where(chosen, p.gather(1, idx), 0.0)
    total = raw.sum(1, keepdim=True)
    weight = torch.where(chosen, raw / torch.where(total > 0, total, 1.0), 0.0)
    idx = torch.where(chosen, idx, -1).to(torch.int32)
    key = torch.where(idx >= 0, idx, E).view(-1)
    order = torch.sort(key, stable=True)[1].to(torch.int32)
    hits = (key[:, None] == torch.arange(E, device="cuda")[None]) if key.numel() * E <= 1 << 26 else None
    counts = hits.sum(0) if hits is not None else torch.zeros(E + 1, dtype=torch.int64, device="cuda").index_add_(
        0, key, torch.ones_like(key, dtype=torch.int64))[:E]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)]).to(torch.int32)
    tokens = live.sum().clamp(min=1).float()
    f = counts.float() / (tokens * top)
    loss = E * (f.double() * p.sum(0, dtype=torch.float64) / tokens.double()).sum()
    out = dict(idx=idx, weight=weight, counts=counts.to(torch.int32), offsets=offsets, order=order,
               loss=loss.float().view(1))
    if s["train"]:
        c = (s["grad_weight"] * weight).sum(1, keepdim=True)
        d = torch.zeros(m, E, device="cuda")
        d.scatter_add_(1, idx.clamp(min=0).long(), torch.where(chosen, weight * (s["grad_weight"] - c), 0.0))
        dp = (s["grad_loss"] * E * f / tokens)[None]
        out["dlogits"] = (d + p * (dp - (p * dp).sum(1, keepdim=True))).to(s["logits"].dtype)
    return out


def _plain(s):
    op = s["op"]
    if op in ("gemv", "gemm"):
        return (_f8(s["x_in"]) @ _unpack(s["w"], s["n"], s["k"]).T).to(TYPES[s.get("y", "fp32")])
    if op == "moe":
        return _plain_moe(s)
    if op == "checkpoint":
        return _f8(s["x_in"]).to(s["x_in"].dtype)
    if op == "backward":
        dx = _f8(s["dy"]) @ _unpack(s["w_t"], s["k"], s["n"]).T
        return dx.to(torch.bfloat16), s["dy"].float().T.contiguous() @ _f8(s["x_in"])
    return _plain_route(s)


# ----------------------------------------------------------- the own kernels
def _own(s):
    import quantized_weight_gemv_amd as qg
    op = s["op"]
    if op == "gemv":
        return qg.qgemv_f8(s["w"], s["x_in"], s["n"], s["k"])
    if op == "gemm":
        xq = qg.qact_quantize_f8(s["x_in"])
        return qg.qgemm_f8(s["w"], xq, s["m"], s["n"], s["k"], dtype=TYPES[s["y"]])
    if op == "moe":
        xq = qg.qact_quantize_f8(s["x_in"])
        return qg.qmoe_gemm_f8(s["w"], s["experts"], xq, s["m"], s["order"], s["offsets"], s["n"], s["k"],
                               dtype=TYPES[s["y"]])
    if op == "checkpoint":
        xq = qg.qact_quantize_f8(s["x_in"])
        return qg.qact_dequant_f8(xq, s["m"], s["k"], dtype=s["x_in"].dtype)
    if op == "backward":
        xq = qg.qact_quantize_f8(s["x_in"])
        dyq = qg.qact_quantize_f8(s["dy"])
        dx = qg.qgemm_f8(s["w_t"], dyq, s["m"], s["k"], s["n"], dtype=torch.bfloat16)
        return dx, qg.qgemm_f8_wgrad(s["dy"], xq, s["m"], s["n"], s["k"])
    r = qg.qmoe_route(s["logits"], s["top"], mask=s["mask"])
    out = dict(idx=r.idx, weight=r.weight, counts=r.counts, offsets=r.offsets, order=r.order, loss=r.loss)
    if s["train"]:
        out["dlogits"] = qg.qmoe_route_backward(s["logits"], r, grad_weight=s["grad_weight"],
                                                grad_loss=s["grad_loss"], mask=s["mask"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ in 64 bits
def _pow2(e):
    """2^e in 64 bits, exact where a power function need not be."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(packed, n, k):
    """One packed matrix's values in 64 bits, through torch's own reading of e4m3."""
    rb, cb = (n + 127) // 128, (k + 127) // 128
    rows, cols, ls = _up(n, 16), 128 * cb, _up(cb, 4)
    r, c = torch.arange(n, device="cuda")[:, None], torch.arange(k, device="cuda")[None]
    at = ((r // 16 * cb + c // 128) * 2048 + c % 128 // 16 * 256 + r % 16 * 16 + c % 16)
    e = packed[rows * cols + r // 128 * ls + c // 128].long() - 127
    return packed[at].view(torch.float8_e4m3fn).double() * _pow2(e)


def _exact_f8(x):
    m, k = x.shape
    out = torch.empty(m, k, dtype=torch.float64, device="cuda")
    for c in range(0, k, 128):
        v = x[:, c:c + 128].double()
        a = v.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 448))
        e = e - ((e > -127) & (a <= 448 * _pow2(e - 1))).double()      # log2 may be off by an ulp
        e = e + (a > 448 * _pow2(e)).double()
        e = torch.where(a > 0, e, 0.0).clamp(min=-127)
        q = (v * _pow2(-e)).float().to(torch.float8_e4m3fn)
        out[:, c:c + 128] = q.double() * _pow2(e)
    return out


def _exact_route(s):
    E, top, m = s["experts"], s["top"], s["m"]
    x = s["logits"].double()
    x[s["mask"] == 0] = -math.inf
    p = torch.softmax(x, 1)
    live = ~torch.isnan(p[:, 0])
    p[~live] = 0
    some = x > -math.inf
    # rank of an expert: those above it, and the equal ones before it
    rank = torch.empty(m, E, dtype=torch.int64, device="cuda")
    before = torch.tril(torch.ones(E, E, dtype=torch.bool, device="cuda"), -1)
    for a in range(0, m, 1024):
        v = x[a:a + 1024]
        rank[a:a + 1024] = (v[:, None, :] > v[:, :, None]).sum(2)
        rank[a:a + 1024] += ((v[:, None, :] == v[:, :, None]) & before[None]).sum(2)
    taken = (rank < top) & some
    w = torch.where(taken, p, 0.0)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total.clamp(min=1e-300), 0.0)
    idx = torch.full((m, top), -1, dtype=torch.int64, device="cuda")
    weight = torch.zeros(m, top, dtype=torch.float64, device="cuda")
    t, e = taken.nonzero(as_tuple=True)
    idx[t, rank[t, e]] = e
    weight[t, rank[t, e]] = w[t, e]
    tokens = max(1, int(live.sum()))
    counts = taken.sum(0)
    f = counts.double() / (tokens * top)
    loss = E * (f * p.sum(0) / tokens).sum()
    # slots by expert: the pair (expert, slot), sorted
    flat = idx.view(-1)
    key = torch.where(flat >= 0, flat, E) * flat.numel() + torch.arange(flat.numel(), device="cuda")
    out = dict(idx=idx.int(), weight=weight, counts=counts.int(),
               offsets=torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int(),
               order=(torch.sort(key)[0] % flat.numel()).int(), loss=loss.view(1))
    if s["train"]:
        gw, gl = s["grad_weight"].double(), s["grad_loss"].double()
        dp = (gl * E * f / tokens)[None].expand(m, E)
        gs = torch.zeros(m, E, dtype=torch.float64, device="cuda")
        gs[t, e] = gw[t, rank[t, e]]
        d_w = torch.where(taken, gs - (gs * w).sum(1, keepdim=True), 0.0) / torch.where(total > 0, total, 1.0)
        d = d_w + dp
        out["dlogits"] = p * (d - (p * d).sum(1, keepdim=True))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    x = _exact_f8(s["x_in"])
    if op == "checkpoint":
        return x
    if op == "backward":
        dx = _exact_f8(s["dy"]) @ _exact_values(s["w_t"], case["k"], case["n"]).T.contiguous()
        return dx, s["dy"].double().T.contiguous() @ x
    if op == "moe":
        y = torch.zeros(case["m"] * case["top"], case["n"], dtype=torch.float64, device="cuda")
        at = s["offsets"].tolist()
        for e in range(case["experts"]):
            slots = s["order"][at[e]:at[e + 1]].long()
            if len(slots):
                y[slots] = x[slots // case["top"]] @ _exact_values(s["w"][e], case["n"], case["k"]).T.contiguous()
        return y
    return x @ _exact_values(s["w"], case["n"], case["k"]).T.contiguous()
