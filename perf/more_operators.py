"""The operators of an expert layer in a training step, as measured cases.

Four operators, each with its plain form (elementary torch operations in 32
bits, rounded once at the end), its call into this package, and its definition
in 64 bits:

  route    the router: top-k experts of every token with their weights, counts
           per expert and the slots in the experts' order, a balance loss; and
           the gradient of the logits
  blocks   matrices held in 8-bit floating point with a power-of-two scale for
           each block of 128 (rows: 1 x 128, weights: 128 x 128), and their
           product, dense or over a stack of experts, in both directions
  norm     the norms after and before a block, fused with the block's gate and
           the residual scale, and their backward pass
  dropout  dropout from a counter-based generator: the mask is drawn again in
           the backward pass instead of being kept

The 8-bit form. A block of values is held as e4m3 numbers q and one byte s:
the value is q * 2^(s - 127). s is the smallest exponent, at least 1, with
(largest magnitude) <= 448 * 2^(s - 127); q = x * 2^(127 - s) rounded half to
even. A block with an infinity or NaN has s = 255 and reads back as NaN. Rows
of q are padded to a multiple of 16 bytes, rows of s to a multiple of 4, with
zeros.

The generator. Eight consecutive columns of a row share a counter n = offset +
row * ceil(cols / 8) + column / 8. Philox4x32-10 with the key `seed` and the
counter words (n mod 2^32, n / 2^32, 0, 0) gives eight 16-bit numbers h (a word's
low half first), with (n mod 2^32, n / 2^32, 1, 0) eight more, l. An element is
dropped when h * 65536 + l < round(p * 2^32), the others are scaled by the
inverse of the exact share that stays.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DT = {"bf16": BF16, "f32": F32}
SIZE = {"bf16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the router of a layer of 256 experts over a packed batch, forward and backward
        dict(name="route-long", op="route", tokens=32768, experts=256, top_k=8, dtype="bf16", dead=0.05,
             renormalise=True),
        # fp32 logits, odd sizes, weights as they come out of the softmax
        dict(name="route-odd-f32", op="route", tokens=1021, experts=76, top_k=3, dtype="f32", dead=0.1,
             renormalise=False),
        # a layer's weights held in 8 bits after an optimizer step, and read back
        dict(name="blocks-weights", op="hold", tiles=True, groups=8, rows=8192, cols=6144, dtype="bf16"),
        # the input of a dense layer quantised and multiplied, a full batch
        dict(name="product-dense", op="product", rows=8192, n=8192, k=6144, groups=1, top_k=1, back=False,
             dtype="bf16", out="bf16"),
        # 76 experts of 2048 x 6144: the tokens' rows gathered in the experts' order, quantised, multiplied
        dict(name="product-experts", op="product", rows=38912, n=2048, k=6144, groups=76, top_k=4, back=False,
             dtype="bf16", out="bf16"),
        # one decoding step of a few sequences through a dense layer: the weights' bytes are what counts
        dict(name="product-tokens", op="product", rows=7, n=8192, k=6144, groups=1, top_k=1, back=False,
             dtype="bf16", out="bf16"),
        # the gradient of the input of a stack of experts, odd sizes, fp32 in and out
        dict(name="product-back-odd", op="product", rows=1531, n=1000, k=2303, groups=5, top_k=1, back=True,
             dtype="f32", out="f32"),
        # norms and gate around a block over a full batch, forward and backward
        dict(name="norm-long", op="norm", rows=16384, cols=8192, dtype="bf16", residual="bf16", weights="bf16",
             gate="cols", backward=True),
        # a short odd batch, the residual stream in fp32, one gate for each token
        dict(name="norm-odd", op="norm", rows=331, cols=2303, dtype="bf16", residual="f32", weights="f32",
             gate="rows", backward=True),
        # the same block in a decoding step
        dict(name="norm-tokens", op="norm", rows=7, cols=6144, dtype="bf16", residual="bf16", weights="bf16",
             gate="none", backward=False),
        # dropout of a block's output added to the residual stream, and the gradient's dropout
        dict(name="dropout-long", op="dropout", rows=16384, cols=8192, dtype="bf16", p=0.1),
        # a short odd batch in fp32
        dict(name="dropout-odd-f32", op="dropout", rows=331, cols=2303, dtype="f32", p=0.25),
    ]


def _between(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm, odd half of the time."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v |= 1
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["route", "hold", "product", "product", "product", "norm", "norm", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    while True:
        if op == "route":
            experts = _between(rng, 8, 512)
            c = dict(op=op, tokens=_between(rng, 1, 32768), experts=experts, top_k=min(experts, rng.choice([1, 2, 4, 6, 8])),
                     dtype=dtype, dead=rng.choice([0.0, 0.1]), renormalise=rng.random() < 0.7)
            if c["tokens"] < 64:
                c["dead"] = 0.0
        elif op == "hold":
            tiles = rng.random() < 0.5
            c = dict(op=op, tiles=tiles, groups=rng.choice([1, 3]) if tiles else 1, rows=_between(rng, 1, 16384),
                     cols=_between(rng, 64, 14336), dtype=dtype)
        elif op == "product":
            c = dict(op=op, rows=_between(rng, 1, 32768), n=_between(rng, 64, 8192), k=_between(rng, 64, 8192),
                     groups=rng.choice([1, 1, 4, 16]), top_k=rng.choice([1, 1, 2]), back=rng.random() < 0.4, dtype=dtype,
                     out=rng.choice(["bf16", "f32"]))
            c["rows"] -= c["rows"] % c["top_k"] if c["rows"] > c["top_k"] else c["rows"] - c["top_k"]
        elif op == "norm":
            c = dict(op=op, rows=_between(rng, 1, 16384), cols=_between(rng, 64, 12288), dtype=dtype,
                     residual="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]), weights=rng.choice(["bf16", "f32"]),
                     gate=rng.choice(["none", "cols", "rows", "full"]), backward=rng.random() < 0.7)
        else:
            c = dict(op=op, rows=_between(rng, 1, 16384), cols=_between(rng, 64, 14336), dtype=dtype,
                     p=rng.choice([0.05, 0.1, 0.5]))
        w = work(c)
        if op == "product":
            heavy = w["flops"] > 8e11 or c["groups"] * c["n"] * c["k"] > 1 << 29
        else:
            heavy = w["bytes"] > 1.8e9
        if not heavy:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, dtype, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g, dtype=F32) * std).to(dtype)


def _activations(rows, cols, g, dtype):
    """Values as a layer's activations are spread: each row with its own size, and a few columns much larger."""
    x = torch.randn((rows, cols), device="cuda", generator=g, dtype=F32)
    x *= torch.exp(0.5 * torch.randn((rows, 1), device="cuda", generator=g))
    x *= torch.exp(0.7 * torch.randn((1, cols), device="cuda", generator=g))
    return x.to(dtype)


def prepare(case, seed):
    c, g, s = case, _gen(seed), dict(case=case)
    op, dt = c["op"], DT[c["dtype"]]
    if op == "route":
        n, e = c["tokens"], c["experts"]
        x = torch.randn((n, e), device="cuda", generator=g) + 0.7 * torch.randn((1, e), device="cuda", generator=g)
        live = torch.rand(n, device="cuda", generator=g) >= c["dead"]
        x[~live] = math.nan  # rows of padding hold anything
        s.update(logits=x.to(dt), live=live if c["dead"] > 0 else None,
                 dweights=_normal((n, c["top_k"]), g, F32, 1e-2))
    elif op == "hold":
        if c["tiles"]:
            s["x"] = _normal((c["groups"], c["rows"], c["cols"]), g, dt, 0.02)
        else:
            s["x"] = _activations(c["rows"], c["cols"], g, dt)
    elif op == "product":
        m, n, k, e = c["rows"], c["n"], c["k"], c["groups"]
        s["x"] = _activations(m // c["top_k"], n if c["back"] else k, g, dt)
        w = torch.empty((e, n, -(-k // 16) * 16), device="cuda", dtype=torch.uint8)
        t = torch.empty((e, -(-n // 128), _scale_pitch(k)), device="cuda", dtype=torch.uint8)
        for i in range(0, e, 8):
            w[i:i + 8], t[i:i + 8] = _hold_tiles(_normal((min(8, e - i), n, k), g, F32, 0.02))
        s["w"], s["ws"] = w, t
        if e > 1:  # the slots of the rows, expert by expert; the first expert has none
            r = np.random.RandomState(int(seed) % (1 << 31))
            share = np.exp(0.5 * r.randn(e))
            share[0] = 0.0
            s["ends"] = [0] + [int(v) for v in np.rint(np.cumsum(share) / share.sum() * m)]
            s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda")
        else:
            s["ends"], s["offsets"] = [0, m], None
        s["order"] = torch.randperm(m, device="cuda", generator=g).int() if e > 1 or c["top_k"] > 1 else None
    elif op == "norm":
        m, n, wt = c["rows"], c["cols"], DT[c["weights"]]
        s["x"] = _activations(m, n, g, DT[c["residual"]])
        s["y"] = _activations(m, n, g, dt)
        s["post"], s["pre"] = (1 + _normal((n,), g, F32, 0.2)).to(wt), (1 + _normal((n,), g, F32, 0.2)).to(wt)
        shape = dict(none=None, cols=(n,), rows=(m, 1), full=(m, n))[c["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(_normal(shape, g, F32)).to(wt if c["gate"] == "cols" else dt)
        s["alpha"], s["beta"], s["eps"] = 0.9, 0.6, 1e-6
        if c["backward"]:
            s["dres"], s["dnormed"] = _normal((m, n), g, DT[c["residual"]], 1e-2), _normal((m, n), g, dt, 1e-2)
    else:
        s["x"], s["residual"] = _activations(c["rows"], c["cols"], g, dt), _normal((c["rows"], c["cols"]), g, dt)
        s["dy"] = _normal((c["rows"], c["cols"]), g, dt, 1e-2)
        s["seed"] = int(torch.randint(0, 1 << 62, (1,), device="cuda", generator=g))
        s["offset"] = (1 << 32) - c["rows"]  # counters of a long run pass 32 bits
    return s


# ------------------------------------------------------------------ plain forms
def _plain_route(s, c):
    n, e, k = c["tokens"], c["experts"], c["top_k"]
    z = s["logits"].float()
    live = torch.ones(n, dtype=torch.bool, device=z.device) if s["live"] is None else s["live"]
    live = live & (z > -math.inf).any(-1)
    z = torch.where(live[:, None], z, torch.zeros_like(z))
    top = z.amax(-1, keepdim=True)
    p = (z - top).exp()
    total = p.sum(-1, keepdim=True)
    p = p / total
    logz = torch.where(live, (top + total.log())[:, 0], torch.zeros_like(top[:, 0]))
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :k]
    chosen = live[:, None] & (z.gather(1, order) > -math.inf)
    experts = torch.where(chosen, order, torch.full_like(order, -1)).int()
    w = torch.where(chosen, p.gather(1, order), torch.zeros_like(p[:, :k]))
    if c["renormalise"]:
        w = w / torch.where(live[:, None], w.sum(-1, keepdim=True), torch.ones_like(w[:, :1]))
    flat = experts.reshape(-1).long()
    flat = torch.where(flat < 0, torch.full_like(flat, e), flat)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=z.device)
    counts.index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts[:e].cumsum(0)]).int()
    slots = torch.sort(flat, stable=True).indices
    slots = torch.where(torch.arange(n * k, device=z.device) < offsets[e], slots, torch.full_like(slots, -1)).int()
    t = live.sum().float().clamp(min=1)
    mean = torch.where(live[:, None], p, torch.zeros_like(p)).sum(0) / t
    share = counts[:e].float() * (e / k) / t
    loss = 0.01 * (share * mean).sum() + 0.001 * (logz * logz).sum() / t
    # the gradient of the logits
    dw = torch.where(chosen, s["dweights"], torch.zeros_like(s["dweights"]))
    slope = (0.01 / t) * share[None].expand(n, e)
    if c["renormalise"]:
        direct = w * (dw - (w * dw).sum(-1, keepdim=True))
        d = p * (slope - (p * slope).sum(-1, keepdim=True) + (0.002 / t) * logz[:, None])
        d = d.scatter_add(1, order, torch.where(chosen, direct, torch.zeros_like(direct)))
    else:
        slope = slope.scatter_add(1, order, dw)
        d = p * (slope - (p * slope).sum(-1, keepdim=True) + (0.002 / t) * logz[:, None])
    d = torch.where(live[:, None], d, torch.zeros_like(d))
    return experts, w, counts[:e].int(), offsets, slots, loss, logz, d.to(s["logits"].dtype)


def _scale_pitch(cols):
    return -(-(-(-cols // 128)) // 4) * 4


def _e4m3(b, top):
    """(bytes of b in units of its block's scale, the scale bytes), the blocks' largest magnitudes in `top`."""
    bits = top.view(torch.int32)
    s = torch.where(bits >= 0x7F800000, torch.full_like(bits, 255), (((bits + 0x1FFFFF) >> 23) - 8).clamp(min=1))
    up = ((254 - s.clamp(max=253)) << 23).view(F32)
    q = (b * up).to(E4M3).view(torch.uint8)
    return torch.where(s == 255, torch.full_like(q, 0x7F), q), s.to(torch.uint8)


def _pad(x, cols, value=0):
    return torch.nn.functional.pad(x, (0, cols - x.shape[-1]), value=value)


def _hold_rows(x):
    """(q, s) of a float32 matrix, a scale for each 128 values of a row."""
    rows, cols = x.shape
    n = -(-cols // 128)
    b = _pad(x, n * 128).view(rows, n, 128)
    q, s = _e4m3(b, b.abs().amax(-1, keepdim=True))
    return _pad(q.view(rows, -1)[:, :cols], -(-cols // 16) * 16), _pad(s[..., 0], _scale_pitch(cols))


def _hold_tiles(x):
    """(q, s) of a float32 stack of matrices, a scale for each 128 x 128 values."""
    e, rows, cols = x.shape
    m, n = -(-rows // 128), -(-cols // 128)
    b = torch.nn.functional.pad(x, (0, n * 128 - cols, 0, m * 128 - rows)).view(e, m, 128, n, 128)
    q, s = _e4m3(b, b.abs().amax((2, 4), keepdim=True))
    q = q.view(e, m * 128, n * 128)[:, :rows, :cols]
    return _pad(q, -(-cols // 16) * 16), _pad(s.view(e, m, n), _scale_pitch(cols))


def _unit(s):
    s = s.int()
    return torch.where(s == 255, torch.full_like(s, 0x7FC00000), s.clamp(min=1) << 23).view(F32)


def _rows_held(q, s, cols):
    unit = _unit(s[:, : -(-cols // 128)]).repeat_interleave(128, 1)[:, :cols]
    return q[:, :cols].view(E4M3).float() * unit


def _tiles_held(q, s, cols):
    rows = q.shape[1]
    unit = _unit(s[:, :, : -(-cols // 128)]).repeat_interleave(128, 1)[:, :rows].repeat_interleave(128, 2)[:, :, :cols]
    return q[:, :, :cols].contiguous().view(E4M3).float() * unit


def _plain_product(s, c):
    x = s["x"].float()
    if s["order"] is not None:
        x = x[s["order"].long() // c["top_k"]]
    a = _rows_held(*_hold_rows(x), x.shape[1])
    ends, out = s["ends"], []
    for i in range(c["groups"]):
        w = _tiles_held(s["w"][i:i + 1], s["ws"][i:i + 1], c["k"])[0]
        rows = a[ends[i]:ends[i + 1]]
        out.append(torch.matmul(rows, w if c["back"] else w.t()))
    return torch.cat(out).to(DT[c["out"]])


def _plain_norm(s, c):
    x, y, n = s["x"].float(), s["y"].float(), c["cols"]
    post, pre = s["post"].float(), s["pre"].float()
    gate = torch.ones((), device=x.device) if s["gate"] is None else s["gate"].float()
    ry = torch.rsqrt((y * y).sum(-1, keepdim=True) / n + s["eps"])
    yh = y * ry
    u = yh * post
    r = s["alpha"] * x + s["beta"] * gate * u
    rr = torch.rsqrt((r * r).sum(-1, keepdim=True) / n + s["eps"])
    rh = r * rr
    forward = r.to(s["x"].dtype), (rh * pre).to(s["y"].dtype)
    if not c["backward"]:
        return forward
    dz, dr = s["dnormed"].float(), s["dres"].float()
    g = dz * pre
    dr = dr + rr * (g - rh * ((g * rh).sum(-1, keepdim=True) / n))
    dpre = (dz * rh).sum(0)
    dgate = s["beta"] * dr * u
    du = s["beta"] * gate * dr
    dpost = (du * yh).sum(0)
    g = du * post
    dy = ry * (g - yh * ((g * yh).sum(-1, keepdim=True) / n))
    if c["gate"] == "cols":
        dgate = dgate.sum(0)
    elif c["gate"] == "rows":
        dgate = dgate.sum(-1, keepdim=True)
    grads = [(s["alpha"] * dr).to(s["x"].dtype), dy.to(s["y"].dtype), dpost.to(s["post"].dtype), dpre.to(s["pre"].dtype)]
    if c["gate"] != "none":
        grads.append(dgate.to(s["gate"].dtype))
    return (*forward, *grads)


def _philox(n, seed, third):
    """Four 32-bit words for each 64-bit counter, in int64."""
    low = 0xFFFFFFFF

    def mul(a, b):  # high and low word of a * b
        p0, p1 = (a & 0xFFFF) * b, (a >> 16) * b
        return (p1 + (p0 >> 16)) >> 16, ((p1 << 16) + p0) & low

    a, b, c, d = n & low, (n >> 32) & low, torch.full_like(n, third), torch.zeros_like(n)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        (h0, l0), (h1, l1) = mul(a, 0xD2511F53), mul(c, 0xCD9E8D57)
        a, b, c, d = h1 ^ b ^ k0, l1, h0 ^ d ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([a, b, c, d], -1)


def _kept(s, c):
    rows, cols = c["rows"], c["cols"]
    packs = -(-cols // 8)
    limit = round(c["p"] * 2 ** 32)
    keep = torch.empty((rows, cols), dtype=torch.bool, device=s["x"].device)
    for a in range(0, rows, 2048):
        b = min(rows, a + 2048)
        n = s["offset"] + torch.arange(a * packs, b * packs, device=keep.device)
        high, low = _philox(n, s["seed"], 0), _philox(n, s["seed"], 1)
        v = torch.stack([((high & 0xFFFF) << 16) | (low & 0xFFFF), (high & 0xFFFF0000) | (low >> 16)], -1)
        keep[a:b] = (v >= limit).view(b - a, packs * 8)[:, :cols]
    return keep, float(torch.tensor(2.0 ** 32 / (2 ** 32 - limit), dtype=F32))


def _plain_dropout(s, c):
    keep, scale = _kept(s, c)
    dt = s["x"].dtype
    zero = torch.zeros((), device=s["x"].device)
    out = s["residual"].float() + torch.where(keep, s["x"].float() * scale, zero)
    return out.to(dt), torch.where(keep, s["dy"].float() * scale, zero).to(dt)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        return _own(s, c, op)
    if op == "route":
        return _plain_route(s, c)
    if op == "hold":
        if c["tiles"]:
            return _tiles_held(*_hold_tiles(s["x"].float()), c["cols"]).to(s["x"].dtype)
        return _rows_held(*_hold_rows(s["x"].float()), c["cols"]).to(s["x"].dtype)
    if op == "product":
        return _plain_product(s, c)
    if op == "norm":
        return _plain_norm(s, c)
    return _plain_dropout(s, c)


# ------------------------------------------------------------------ this package's calls
def _own(s, c, op):
    from newton_schulz_quintic_gb300 import api
    if op == "route":
        coefs = dict(live=s["live"], renormalise=c["renormalise"], balance_coef=0.01, z_coef=0.001)
        r = api.route(s["logits"], c["top_k"], **coefs)
        d = api.route_backward(s["logits"], r, s["dweights"], renormalise=c["renormalise"], balance_coef=0.01, z_coef=0.001)
        return r.experts, r.weights, r.counts, r.offsets, r.order, r.loss, r.logz, d
    if op == "hold":
        return api.blocks_load(api.blocks_store(s["x"], tiles=c["tiles"]), dtype=s["x"].dtype)
    if op == "product":
        w = api.Blocks8(s["w"], s["ws"], c["k"], tiles=True)
        a = api.blocks_store(s["x"], rows=s["order"], per=c["top_k"])
        return api.blocks_matmul(a, w, transpose=c["back"], offsets=s["offsets"], dtype=DT[c["out"]])
    if op == "norm":
        kw = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"], residual_scale=s["alpha"],
                  block_scale=s["beta"])
        f = api.block_norm(s["x"], s["y"], eps=s["eps"], **kw)
        if not c["backward"]:
            return f.residual, f.normed
        b = api.block_norm_backward(s["dres"], s["dnormed"], s["x"], s["y"], f, **kw)
        grads = (b.dx, b.dy, b.dpost_weight, b.dpre_weight)
        return (f.residual, f.normed, *grads) if s["gate"] is None else (f.residual, f.normed, *grads, b.dgate)
    out = api.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"])
    return out, api.dropout(s["dy"], c["p"], s["seed"], s["offset"])


# ------------------------------------------------------------------ least work
def work(case):
    c = case
    op, z = c["op"], SIZE[c["dtype"]]
    if op == "route":  # logits in twice, their gradient out; the chosen ones' numbers
        n, slots = c["tokens"] * c["experts"], c["tokens"] * c["top_k"]
        return dict(bytes=3 * n * z + slots * (4 + 4 + 4 + 4) + 8 * c["tokens"], flops=12 * n)
    if op == "hold":  # written and read back
        n = c["groups"] * c["rows"] * c["cols"]
        return dict(bytes=n * (2 * z + 2), flops=3 * n)
    if op == "product":
        m, n, k = c["rows"], c["n"], c["k"]
        inner, outer = (n, k) if c["back"] else (k, n)
        used = min(c["groups"], m)  # experts that can have a row
        return dict(bytes=m // c["top_k"] * inner * z + used * n * k + m * outer * SIZE[c["out"]], flops=2.0 * m * n * k)
    n = c["rows"] * c["cols"]
    if op == "norm":
        r, full = SIZE[c["residual"]], c["gate"] == "full"
        if not c["backward"]:
            return dict(bytes=n * (2 * r + 2 * z + full * z), flops=9 * n)
        return dict(bytes=n * (5 * r + 5 * z + full * 3 * z), flops=30 * n)
    return dict(bytes=5 * n * z, flops=30 * n)


# ------------------------------------------------------------------ 64 bits
def _exact_route(s, c):
    n, e, k = c["tokens"], c["experts"], c["top_k"]
    x = s["logits"].double()
    ok = torch.ones(n, dtype=torch.bool, device="cuda") if s["live"] is None else s["live"]
    x[~ok] = 0
    x.requires_grad_(True)
    p = torch.softmax(x, -1)
    lse = torch.logsumexp(x, -1)
    # distinct whole numbers in the order of (value, lower index first)
    values, rank = torch.unique(x.detach(), return_inverse=True)
    experts = torch.topk(rank * (2 * e) + (e - 1 - torch.arange(e, device="cuda")), k, dim=-1).indices
    w = torch.gather(torch.softmax(torch.gather(x, 1, experts), -1) if c["renormalise"] else p, 1,
                     torch.arange(k, device="cuda").expand(n, k) if c["renormalise"] else experts)
    counts = torch.bincount(experts[ok].reshape(-1), minlength=e)
    t = int(ok.sum())
    balance = e / (k * t * t) * (counts.double() * p[ok].sum(0)).sum() if t else 0 * p.sum()
    z = (lse[ok] ** 2).sum() / t if t else 0 * p.sum()
    loss = 0.01 * balance + 0.001 * z
    (loss + (w * s["dweights"].double())[ok].sum()).backward()
    experts = torch.where(ok[:, None], experts, torch.full_like(experts, -1))
    slot = torch.full((n * k,), -1, dtype=torch.int32, device="cuda")
    flat = experts.reshape(-1)
    where = torch.nonzero(flat >= 0)[:, 0]
    slot[: where.numel()] = where[torch.argsort(flat[where] * (n * k) + where)].int()
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0).int()
    zero = torch.zeros((), dtype=F64, device="cuda")
    return (experts.int(), torch.where(ok[:, None], w.detach(), zero), counts.int(), offsets, slot, loss.detach(),
            torch.where(ok, lse.detach(), zero), x.grad)


def _pow2(e):
    """2^e of whole numbers, exactly (a library power may be off by a unit in the last place)."""
    return ((e.long() + 1023) << 52).view(F64)


def _nearest_e4m3(v):
    """v (float64, at most 448 in magnitude) to the nearest number of 4 significant bits, 2^-9 apart near zero, ties to even."""
    step = _pow2(torch.clamp(torch.frexp(v).exponent - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _exact_unit(top):
    """Smallest power of two, at least 2^-126, that brings `top` to 448 or less."""
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448))
    e = torch.where(top > 448 * _pow2(e), e + 1, e)
    e = torch.where(top <= 448 * _pow2(e - 1), e - 1, e)
    return _pow2(e.clamp(min=-126))


def _exact_rows(x):
    rows, cols = x.shape
    out = torch.empty((rows, cols), dtype=F64, device="cuda")
    for a in range(0, cols, 128):
        b = x[:, a:a + 128].double()
        unit = _exact_unit(b.abs().max(-1, keepdim=True).values)
        out[:, a:a + 128] = _nearest_e4m3(b / unit) * unit
    return out


def _from_bytes(q, s, cols):
    """The matrix that bytes stand for, digit by digit (no NaN among them)."""
    q = q[:, :cols].int()
    expo, frac = (q >> 3) & 15, (q & 7).double()
    v = torch.where(expo == 0, frac * 2.0 ** -9, (8 + frac) * _pow2(expo - 10))
    v = torch.where(q >= 128, -v, v)
    for i in range(-(-q.shape[0] // 128)):
        unit = _pow2(s[i].int() - 127).repeat_interleave(128)[:cols]
        v[128 * i:128 * i + 128] *= unit
    return v


def _exact_kept(s, c):
    rows, cols, packs = c["rows"], c["cols"], -(-c["cols"] // 8)
    out = torch.empty((rows, cols), dtype=torch.bool, device="cuda")
    m = (1 << 32) - 1

    def product(const, v):  # 64-bit product as two 32-bit words, from four 16 x 16 products
        x0, x1, y0, y1 = v % 65536, v // 65536, const % 65536, const // 65536
        low, mid, high = x0 * y0, x0 * y1 + x1 * y0, x1 * y1
        mid = mid + low // 65536
        return high + mid // 65536, (mid % 65536) * 65536 + low % 65536

    for a in range(0, rows, 1024):
        n = torch.arange(a, min(rows, a + 1024), device="cuda")[:, None] * packs + torch.arange(packs, device="cuda") + s["offset"]
        words = []
        for third in (0, 1):
            ctr = [n % (1 << 32), n // (1 << 32), torch.zeros_like(n) + third, torch.zeros_like(n)]
            key = [s["seed"] % (1 << 32), s["seed"] // (1 << 32)]
            for r in range(10):
                if r:
                    key = [(key[0] + 2654435769) & m, (key[1] + 3144134277) & m]
                h0, l0 = product(3528531795, ctr[0])
                h1, l1 = product(3449720151, ctr[2])
                ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
            words.append(ctr)
        u = torch.empty((*n.shape, 8), dtype=F64, device="cuda")
        for j in range(8):
            h, l = (words[i][j // 2] // (65536 if j % 2 else 1) % 65536 for i in (0, 1))
            u[..., j] = (h * 65536 + l).double() / 2.0 ** 32
        out[a:a + 1024] = (u.view(n.shape[0], -1) >= round(c["p"] * 2 ** 32) / 2.0 ** 32)[:, :cols]
    return out


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "route":
        return _exact_route(s, c)
    if op == "hold":
        if not c["tiles"]:
            return _exact_rows(s["x"])
        out = torch.empty(s["x"].shape, dtype=F64, device="cuda")
        for i in range(0, c["rows"], 128):
            for j in range(0, c["cols"], 128):
                b = s["x"][:, i:i + 128, j:j + 128].double()
                unit = _exact_unit(b.abs().flatten(1).max(-1).values)[:, None, None]
                out[:, i:i + 128, j:j + 128] = _nearest_e4m3(b / unit) * unit
        return out
    if op == "product":
        a = _exact_rows(s["x"])
        if s["order"] is not None:
            a = a[torch.div(s["order"].long(), c["top_k"], rounding_mode="floor")]
        out = torch.zeros((c["rows"], c["k"] if c["back"] else c["n"]), dtype=F64, device="cuda")
        for i in range(c["groups"]):
            lo, hi = s["ends"][i], s["ends"][i + 1]
            if hi > lo:
                w = _from_bytes(s["w"][i], s["ws"][i], c["k"])
                out[lo:hi] = a[lo:hi] @ (w if c["back"] else w.t())
        return out
    if op == "norm":
        names = ["x", "y", "post", "pre"] + ([] if s["gate"] is None else ["gate"])
        v = {k: s[k].double().requires_grad_(c["backward"]) for k in names}
        u = v["y"] / torch.sqrt(v["y"].pow(2).mean(-1, keepdim=True) + s["eps"]) * v["post"]
        if "gate" in v:
            u = u * v["gate"]
        r = s["alpha"] * v["x"] + s["beta"] * u
        z = r / torch.sqrt(r.pow(2).mean(-1, keepdim=True) + s["eps"]) * v["pre"]
        if not c["backward"]:
            return r, z
        grads = torch.autograd.grad((r, z), [v[k] for k in names], (s["dres"].double(), s["dnormed"].double()))
        return (r.detach(), z.detach(), *grads)
    keep = _exact_kept(s, c)
    scale = 1.0 / (1.0 - round(c["p"] * 2 ** 32) / 2.0 ** 32)
    return s["residual"].double() + keep * (s["x"].double() * scale), keep * (s["dy"].double() * scale)
