"""The operators of a training step around the optimizer, as measured cases.

Four operators, each with its plain form (elementary torch operations in 32
bits, rounded once at the end), its call into this package, and its definition
in 64 bits:

  embed    token embedding: lookup with scaling, and the table's gradient
  policy   clipped policy loss with a KL term on logits, with the gradient of
           the logits; token log probabilities (the loss's old and reference
           inputs)
  ckpt     activations held for the backward pass in 8 bits: store and load,
           and the gated activation silu(gate) * up that keeps gate and up so
  wgrad    the weight gradient of a linear layer, or of a stack of experts,
           from its input held in 8 bits

The 8-bit form. A row of `cols` values is cut into blocks of 32. A block holds
int8 values q and one scale byte E: the value is q * 2^(E - 133). E is the
exponent field of the largest magnitude in the block as a float32, at least 7;
q = round_half_even(x * 2^(133 - E)), at most 127 in magnitude. A block with
an infinity or NaN has E = 255 and reads back as NaN. Rows of q are padded to
a multiple of 16 bytes and rows of scales to a multiple of 4, with zeros.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF16, "f32": F32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the input side of a step over a packed batch of 32768 tokens: rows of a large bf16 table
        dict(name="lookup-long", op="lookup", tokens=32768, vocab=131072, dim=4096, dtype="bf16", pad=0.02),
        # its gradient, dense over the vocabulary, with the few very frequent tokens of natural text
        dict(name="embed-grad-long", op="embed_grad", tokens=32768, vocab=131072, dim=4096, dtype="bf16",
             accumulate=False, pad=0.02),
        # a tied table: a short odd batch added onto the output head's fp32 gradient, rows of odd length
        dict(name="embed-grad-add-odd", op="embed_grad", tokens=509, vocab=50021, dim=1023, dtype="f32",
             accumulate=True, pad=0.1),
        # old or reference log probabilities of the last few tokens of a rollout
        dict(name="logp-few", op="logp", rows=7, vocab=32768, dtype="bf16", masked=0.0),
        # the loss and the logits' gradient of a full batch, a quarter of it prompt tokens without loss
        dict(name="policy-long", op="policy", rows=8192, vocab=131072, dtype="bf16", masked=0.25, kl=True, old=True),
        # fp32 logits, odd row count and vocabulary, first pass over fresh rollouts (no old policy), no KL term
        dict(name="policy-odd-f32", op="policy", rows=1021, vocab=50021, dtype="f32", masked=0.25, kl=False,
             old=False),
        # a layer's fp32 input kept in 8 bits and read back, odd sizes
        dict(name="store-odd-f32", op="store", rows=4093, cols=6143, dtype="f32"),
        # the gated activation of a wide feed-forward layer: forward, and backward from the 8-bit values
        dict(name="gated-long", op="gated", rows=16384, cols=14336, dtype="bf16"),
        # the same for a short odd batch
        dict(name="gated-odd", op="gated", rows=331, cols=2303, dtype="bf16"),
        # weight gradient of one dense matrix over a full batch
        dict(name="wgrad-dense", op="wgrad", rows=8192, n_out=8192, n_in=6144, groups=1, dtype="bf16", grad="bf16",
             accumulate=False),
        # weight gradients of a stack of 76 experts whose tokens are packed one expert after the other
        dict(name="wgrad-experts", op="wgrad", rows=38912, n_out=2048, n_in=6144, groups=76, dtype="bf16",
             grad="bf16", accumulate=False),
        # a small matrix in fp32 throughout, added onto the gradient of earlier micro-batches
        dict(name="wgrad-small-f32", op="wgrad", rows=301, n_out=640, n_in=1000, groups=1, dtype="f32", grad="f32",
             accumulate=True),
    ]


def _between(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm, odd half of the time."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v |= 1
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["lookup", "embed_grad", "logp", "policy", "store", "gated", "wgrad", "wgrad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    pad = rng.choice([0.0, 0.02, 0.3])
    while True:
        if op == "lookup":
            c = dict(op=op, tokens=_between(rng, 1, 32768), vocab=_between(rng, 512, 131072), dim=_between(rng, 64, 4096),
                     dtype=dtype, pad=pad)
        elif op == "embed_grad":
            c = dict(op=op, tokens=_between(rng, 1, 32768), vocab=_between(rng, 512, 131072), dim=_between(rng, 64, 4096),
                     dtype=dtype, accumulate=rng.random() < 0.5, pad=pad)
        elif op == "logp":
            c = dict(op=op, rows=_between(rng, 4, 8192), vocab=_between(rng, 1024, 131072), dtype=dtype,
                     masked=rng.choice([0.0, 0.25]))
        elif op == "policy":
            c = dict(op=op, rows=_between(rng, 16, 8192), vocab=_between(rng, 1024, 131072), dtype=dtype,
                     masked=rng.choice([0.0, 0.25, 0.6]), kl=rng.random() < 0.5, old=rng.random() < 0.7)
        elif op == "store":
            c = dict(op=op, rows=_between(rng, 1, 16384), cols=_between(rng, 32, 14336), dtype=dtype)
        elif op == "gated":
            c = dict(op=op, rows=_between(rng, 1, 16384), cols=_between(rng, 32, 14336), dtype=dtype)
        else:
            c = dict(op=op, rows=_between(rng, 1, 32768), n_out=_between(rng, 64, 8192), n_in=_between(rng, 64, 8192),
                     groups=rng.choice([1, 1, 3, 16]), dtype=dtype, grad=rng.choice(["bf16", "f32"]),
                     accumulate=rng.random() < 0.3)
        if c.get("tokens", 64) < 64:  # too few for some of them to be padding
            c["pad"] = 0.0
        if c.get("rows", 16) < 16 and "masked" in c:
            c["masked"] = 0.0
        w = work(c)
        heavy = w["flops"] > 9e11 if op == "wgrad" else w["bytes"] > 4e9
        if op == "wgrad" and c["groups"] * c["n_out"] * c["n_in"] > 1 << 28:
            heavy = True
        if c.get("dtype") == "f32" and op == "wgrad" and w["flops"] > 2e11:
            heavy = True
        if not heavy:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ids(n, vocab, g, pad):
    """Token ids as frequent as words are (the k-th most frequent in proportion to 1/k), the frequent ones anywhere
    in the vocabulary; a share `pad` of the positions is padding (-1)."""
    u = torch.rand(n, device="cuda", generator=g, dtype=torch.float64)
    k = torch.exp(u * math.log(vocab + 1)).long().clamp_(1, vocab) - 1
    step = 48271
    while math.gcd(step, vocab) != 1:
        step += 2
    ids = (k * step + 17) % vocab
    hole = torch.rand(n, device="cuda", generator=g) < pad
    return torch.where(hole, torch.full_like(ids, -1), ids)


def _normal(shape, g, dtype, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g, dtype=F32) * std).to(dtype)


def _activations(rows, cols, g, dtype):
    """Values as a layer's activations are spread: each row with its own size, and a few columns much larger."""
    x = torch.randn((rows, cols), device="cuda", generator=g, dtype=F32)
    x *= torch.exp(0.5 * torch.randn((rows, 1), device="cuda", generator=g))
    x *= torch.exp(0.7 * torch.randn((1, cols), device="cuda", generator=g))
    return x.to(dtype)


def _offsets(rows, groups, seed):
    """Ends of the groups' packed rows: uneven shares, the first group empty where there are more than two."""
    r = np.random.RandomState(int(seed) % (1 << 31))
    w = np.exp(0.5 * r.randn(groups))
    if groups > 2:
        w[0] = 0.0
    return [0] + [int(v) for v in np.rint(np.cumsum(w) / w.sum() * rows)]


def prepare(case, seed):
    c, g, s = case, _gen(seed), dict(case=case)
    dt = DT[c["dtype"]]
    op = c["op"]
    if op in ("lookup", "embed_grad"):
        s["tokens"] = _ids(c["tokens"], c["vocab"], g, c["pad"])
        s["scale"] = math.sqrt(c["dim"])
        if op == "lookup":
            s["table"] = _normal((c["vocab"], c["dim"]), g, dt, 0.02)
        else:
            s["dout"] = _normal((c["tokens"], c["dim"]), g, dt, 1e-2)
            if c["accumulate"]:
                s["grad"] = _normal((c["vocab"], c["dim"]), g, dt, 1e-2)
    elif op in ("logp", "policy"):
        n, v = c["rows"], c["vocab"]
        x = _normal((n, v), g, dt, 2.0)
        y = _ids(n, v, g, 0.0)
        at = torch.arange(n, device="cuda")
        x[at, y] += 7.0
        x[:, v - v // 64:] = -math.inf  # entries of the output head that no token uses
        y = torch.where(y >= v - v // 64, y % max(1, v - v // 64), y)
        live = torch.rand(n, device="cuda", generator=g) >= c["masked"]
        x[~live, :3] = math.nan  # rows without loss are not looked at, whatever they hold
        s.update(logits=x, targets=torch.where(live, y, torch.full_like(y, -100)), temperature=0.8)
        if op == "policy":
            lp = torch.empty(n, device="cuda", dtype=F32)
            for a in range(0, n, 1024):
                lp[a:a + 1024] = torch.log_softmax(x[a:a + 1024].float() / 0.8, -1).gather(1, y[a:a + 1024, None])[:, 0]
            lp = torch.where(live, lp, torch.zeros_like(lp))
            s["old"] = lp + 0.2 * _normal((n,), g, F32) if c["old"] else None
            s["ref"] = lp + 0.3 * _normal((n,), g, F32) if c["kl"] else None
            s["adv"] = _normal((n,), g, F32) + 1.0
            s["weights"] = live.float() / max(1, n)
            s["kl_coef"] = 0.05 if c["kl"] else 0.0
    elif op == "store":
        s["x"] = _activations(c["rows"], c["cols"], g, dt)
    elif op == "gated":
        s["gu"] = _activations(c["rows"], 2 * c["cols"], g, dt)
        s["dh"] = _normal((c["rows"], c["cols"]), g, dt, 1e-2)
    else:
        s["dy"] = _normal((c["rows"], c["n_out"]), g, dt, 1e-2)
        q, e = _quantise(_activations(c["rows"], c["n_in"], g, F32))
        s["q"], s["e"] = q, e
        off = _offsets(c["rows"], c["groups"], seed)
        s["longest"] = max(b - a for a, b in zip(off, off[1:]))
        s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda") if c["groups"] > 1 else None
        if c["accumulate"]:
            s["grad"] = _normal((c["groups"], c["n_out"], c["n_in"]), g, DT[c["grad"]], 0.05)
    return s


# ------------------------------------------------------------------ plain forms
def _pad_to(x, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1]))


def _quantise(x):
    """(q, scales) of a float32 matrix in the 8-bit form."""
    rows, cols = x.shape
    b = _pad_to(x, -(-cols // 32) * 32).view(rows, -1, 32)
    e = ((b.abs().amax(-1).view(torch.int32) >> 23) & 255).clamp_(min=7)
    up = ((260 - e.clamp(max=254)) << 23).view(F32)
    q = torch.round(b * up[..., None]).clamp_(-127, 127)
    q = torch.where((e == 255)[..., None], torch.zeros_like(q), q).to(torch.int8).view(rows, -1)[:, :cols]
    return _pad_to(q, -(-cols // 16) * 16), _pad_to(e.to(torch.uint8), -(-e.shape[1] // 4) * 4)


def _values(q, e, cols):
    """The float32 values that the 8-bit form stands for."""
    e = e[:, : -(-cols // 32)].int()
    unit = torch.where(e == 255, torch.full_like(e, 0x7FC00000), (e - 6).clamp(min=1) << 23).view(F32)
    return q[:, :cols].float() * unit.repeat_interleave(32, 1)[:, :cols]


def _plain_lookup(s):
    live = s["tokens"] >= 0
    rows = s["table"][s["tokens"].clamp(min=0)].float() * s["scale"]
    return torch.where(live[:, None], rows, torch.zeros_like(rows)).to(s["table"].dtype)


def _plain_embed_grad(s, c):
    live = s["tokens"] >= 0
    rows = s["dout"].float() * s["scale"]
    rows = torch.where(live[:, None], rows, torch.zeros_like(rows))
    g = torch.zeros((c["vocab"], c["dim"]), device=rows.device, dtype=F32)
    g.index_add_(0, s["tokens"].clamp(min=0), rows)
    if c["accumulate"]:
        s["grad"].copy_((s["grad"].float() + g).to(s["grad"].dtype))
        return s["grad"]
    return g.to(s["dout"].dtype)


def _plain_logp(s):
    """(log probability of the target, z - max, sum of exp) with the rows without loss read as zeros."""
    live = s["targets"] >= 0
    z = s["logits"].float() * (1.0 / s["temperature"])
    z = torch.where(live[:, None], z, torch.zeros_like(z))
    z = z - z.amax(-1, keepdim=True)
    total = z.exp().sum(-1)
    at = s["targets"].clamp(min=0)
    lp = z.gather(1, at[:, None])[:, 0] - total.log()
    return torch.where(live, lp, torch.zeros_like(lp)), z, total, live, at


def _plain_policy(s, low=0.2, high=0.28):
    lp, z, total, live, at = _plain_logp(s)
    adv, w = s["adv"], s["weights"]
    r = (lp - s["old"]).exp() if s["old"] is not None else torch.ones_like(lp)
    a, b = r * adv, r.clamp(1 - low, 1 + high) * adv
    d = s["ref"] - lp if s["ref"] is not None else torch.zeros_like(lp)
    kl = torch.where(live, torch.expm1(d) - d, torch.zeros_like(d))
    loss = torch.where(live, w * (s["kl_coef"] * kl - torch.minimum(a, b)), torch.zeros_like(lp)).sum()
    slope = torch.where(a <= b, -a, torch.zeros_like(a)) - s["kl_coef"] * torch.expm1(d)
    slope = torch.where(live, slope * w * (1.0 / s["temperature"]), torch.zeros_like(slope))
    p = z.exp() / total[:, None]
    g = -slope[:, None] * p
    g.scatter_add_(1, at[:, None], slope[:, None])
    return loss, lp, kl, g.to(s["logits"].dtype)


def _plain_gated(s, c):
    f, dt = c["cols"], s["gu"].dtype
    gu = s["gu"].float()
    gate, up = gu[:, :f].contiguous(), gu[:, f:].contiguous()
    h = (gate / (1 + (-gate).exp()) * up).to(dt)
    gate, up = _values(*_quantise(gate), f), _values(*_quantise(up), f)
    dh = s["dh"].float()
    sig = 1 / (1 + (-gate).exp())
    act = gate * sig
    dgate = dh * up * (sig * (1 + gate * (1 - sig)))
    return h, torch.cat([dgate, dh * act], 1).to(dt), (act * up).to(dt)


def _plain_wgrad(s, c):
    x, dy = _values(s["q"], s["e"], c["n_in"]), s["dy"].float()
    if s["offsets"] is None:
        g = torch.matmul(dy.t(), x)[None]
    else:
        first, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
        at = first[:, None] + torch.arange(max(1, s["longest"]), device=x.device)
        inside = at < end[:, None]
        at = at.clamp(max=c["rows"] - 1)
        dy = torch.where(inside[..., None], dy[at], torch.zeros((), device=x.device))
        g = torch.matmul(dy.transpose(1, 2), x[at])
    if c["accumulate"]:
        s["grad"].copy_((s["grad"].float() + g).to(s["grad"].dtype))
        return s["grad"]
    return g.to(DT[c["grad"]])


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        return _own(s, c, op)
    if op == "lookup":
        return _plain_lookup(s)
    if op == "embed_grad":
        return _plain_embed_grad(s, c)
    if op == "logp":
        return _plain_logp(s)[0]
    if op == "policy":
        return _plain_policy(s)
    if op == "store":
        return _values(*_quantise(s["x"].float()), c["cols"]).to(s["x"].dtype)
    if op == "gated":
        return _plain_gated(s, c)
    return _plain_wgrad(s, c)


# ------------------------------------------------------------------ this package's calls
def _own(s, c, op):
    from newton_schulz_quintic_gb300 import api
    if op == "lookup":
        return api.embed_lookup(s["table"], s["tokens"], scale=s["scale"])
    if op == "embed_grad":
        if c["accumulate"]:
            return api.embed_grad(s["dout"], s["tokens"], grad=s["grad"], scale=s["scale"], accumulate=True)
        return api.embed_grad(s["dout"], s["tokens"], vocab=c["vocab"], scale=s["scale"])
    if op == "logp":
        return api.token_logprobs(s["logits"], s["targets"], temperature=s["temperature"])
    if op == "policy":
        r = api.policy_loss(s["logits"], s["targets"], s["adv"], s["weights"], old_logp=s["old"], ref_logp=s["ref"],
                            clip_low=0.2, clip_high=0.28, kl_coef=s["kl_coef"], temperature=s["temperature"])
        return r.loss, r.logp, r.kl, r.dlogits
    if op == "store":
        return api.checkpoint_load(api.checkpoint_store(s["x"]), dtype=s["x"].dtype)
    if op == "gated":
        f = c["cols"]
        h, ck_gate, ck_up = api.gated_forward(s["gu"][:, :f], s["gu"][:, f:])
        dgu, again = api.gated_backward(s["dh"], ck_gate, ck_up)
        return h, dgu, again
    ck = api.Checkpoint8(s["q"], s["e"], c["n_in"])
    if c["accumulate"]:
        return api.checkpoint_wgrad(s["dy"], ck, offsets=s["offsets"], grad=s["grad"], accumulate=True)
    return api.checkpoint_wgrad(s["dy"], ck, offsets=s["offsets"], dtype=DT[c["grad"]])


# ------------------------------------------------------------------ least work
def _distinct(n, vocab):
    """Expected number of distinct ids among n of _ids()."""
    k = np.arange(1, vocab + 1, dtype=np.float64)
    p = np.log1p(1 / k) / math.log(vocab + 1)
    return float(np.sum(-np.expm1(n * np.log1p(-p))))


def work(case):
    c = case
    op, z = c["op"], SIZE[c["dtype"]]
    if op == "lookup":
        n = c["tokens"] * (1 - c["pad"])
        return dict(bytes=(_distinct(n, c["vocab"]) + c["tokens"]) * c["dim"] * z + 8 * c["tokens"],
                    flops=n * c["dim"])
    if op == "embed_grad":
        n = c["tokens"] * (1 - c["pad"])
        rows = 2 * _distinct(n, c["vocab"]) if c["accumulate"] else c["vocab"]
        return dict(bytes=(n + rows) * c["dim"] * z + 8 * c["tokens"], flops=2 * n * c["dim"])
    if op in ("logp", "policy"):
        read = c["rows"] * (1 - c["masked"]) * c["vocab"]
        grad = op == "policy"
        return dict(bytes=(read + (c["rows"] * c["vocab"] if grad else 0)) * z + 40 * c["rows"],
                    flops=read * (6 if grad else 4))
    n = c["rows"] * c.get("cols", 0)
    if op == "store":  # written and read back
        return dict(bytes=n * (2 * z + 2 * (1 + 1 / 32)), flops=4 * n)
    if op == "gated":  # gate, up and dh in; h, two gradients and h again out; two 8-bit values out and in
        return dict(bytes=n * (7 * z + 4 * (1 + 1 / 32)), flops=30 * n)
    g = c["groups"] * c["n_out"] * c["n_in"] * SIZE[c["grad"]] * (2 if c["accumulate"] else 1)
    return dict(bytes=c["rows"] * (c["n_out"] * z + c["n_in"] * (1 + 1 / 32)) + g,
                flops=2.0 * c["rows"] * c["n_out"] * c["n_in"])


# ------------------------------------------------------------------ 64 bits
def _held(x):
    """The values that the 8-bit form of x holds, from its definition, in float64."""
    rows, cols = x.shape
    out = torch.empty((rows, cols), device=x.device, dtype=torch.float64)
    for a in range(0, rows, 2048):
        p = x[a:a + 2048].double()
        n = -(-cols // 32) * 32
        b = torch.zeros((p.shape[0], n), device=x.device, dtype=torch.float64)
        b[:, :cols] = p
        b = b.reshape(p.shape[0], n // 32, 32)
        top = b.abs().max(-1).values
        expo = torch.frexp(top).exponent.double() + 126  # the exponent field of a float32
        expo = torch.where(top == 0, torch.full_like(expo, 7.0), expo.clamp(min=7))
        unit = torch.pow(2.0, expo - 133)[..., None]
        q = (b / unit).round().clamp(-127, 127)
        out[a:a + 2048] = (q * unit).reshape(p.shape[0], n)[:, :cols]
    return out


def _exact_rows(s, a, b):
    x = s["logits"][a:b].double() / s["temperature"]
    y = s["targets"][a:b]
    ok = y >= 0
    x[~ok] = 0
    lse = torch.logsumexp(x, -1)
    return x, lse, y.clamp(min=0), ok


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "lookup":
        t = s["tokens"]
        out = s["table"][t.clamp(min=0)].double() * s["scale"]
        out[t < 0] = 0
        return out
    if op == "embed_grad":
        t = s["tokens"]
        out = s["grad"].double() if c["accumulate"] else torch.zeros((c["vocab"], c["dim"]), device="cuda",
                                                                     dtype=torch.float64)
        order = torch.argsort(t[t >= 0], stable=True)
        ids, count = torch.unique_consecutive(t[t >= 0][order], return_counts=True)
        rows = s["dout"][t >= 0][order]
        end = torch.cumsum(count, 0).tolist()
        first = 0
        total = torch.zeros((len(end), c["dim"]), device="cuda", dtype=torch.float64)
        for a in range(0, rows.shape[0], 8192):  # segments of the sorted rows
            b = min(rows.shape[0], a + 8192)
            which = torch.searchsorted(torch.cumsum(count, 0), torch.arange(a, b, device="cuda"), right=True)
            total.index_put_((which,), rows[a:b].double(), accumulate=True)
        out[ids] += total * s["scale"]
        return out
    if op == "logp":
        out = torch.zeros(c["rows"], device="cuda", dtype=torch.float64)
        for a in range(0, c["rows"], 1024):
            x, lse, y, ok = _exact_rows(s, a, a + 1024)
            out[a:a + 1024] = torch.where(ok, x.gather(1, y[:, None])[:, 0] - lse, torch.zeros_like(lse))
        return out
    if op == "policy":
        n, low, high, beta = c["rows"], 0.2, 0.28, s["kl_coef"]
        lp, kl = (torch.zeros(n, device="cuda", dtype=torch.float64) for _ in range(2))
        g = torch.zeros((n, c["vocab"]), device="cuda", dtype=torch.float64)
        loss = torch.zeros((), device="cuda", dtype=torch.float64)
        for a in range(0, n, 1024):
            b = min(n, a + 1024)
            x, lse, y, ok = _exact_rows(s, a, b)
            l = x.gather(1, y[:, None])[:, 0] - lse
            adv, w = s["adv"][a:b].double(), s["weights"][a:b].double()
            ratio = torch.exp(l - s["old"][a:b].double()) if s["old"] is not None else torch.ones_like(l)
            gain = torch.minimum(ratio * adv, torch.clamp(ratio, 1 - low, 1 + high) * adv)
            k = torch.exp(s["ref"][a:b].double() - l) - (s["ref"][a:b].double() - l) - 1 if c["kl"] else 0 * l
            loss += (w * (beta * k - gain))[ok].sum()
            # d loss / d l: the clipped side is constant in l
            free = ~(((adv > 0) & (ratio > 1 + high)) | ((adv < 0) & (ratio < 1 - low)))
            dl = -(ratio * adv) * free
            if c["kl"]:
                dl = dl + beta * (1 - torch.exp(s["ref"][a:b].double() - l))
            dl = torch.where(ok, dl * w / s["temperature"], torch.zeros_like(l))
            p = torch.exp(x - lse[:, None])
            p = -p * dl[:, None]
            p[torch.arange(b - a, device="cuda"), y] += dl
            g[a:b], lp[a:b], kl[a:b] = p, torch.where(ok, l, 0 * l), torch.where(ok, k, 0 * l)
        return loss, lp, kl, g
    if op == "store":
        return _held(s["x"])
    if op == "gated":
        f = c["cols"]
        g, u = s["gu"][:, :f], s["gu"][:, f:]
        h = g.double() * torch.sigmoid(g.double()) * u.double()
        g, u, dh = _held(g), _held(u), s["dh"].double()
        sig = torch.sigmoid(g)
        dgu = torch.empty((c["rows"], 2 * f), device="cuda", dtype=torch.float64)
        dgu[:, f:] = dh * g * sig
        dgu[:, :f] = dh * u * (sig + g * sig * (1 - sig))
        return h, dgu, g * sig * u
    x = torch.empty((c["rows"], c["n_in"]), device="cuda", dtype=torch.float64)
    for k in range(-(-c["n_in"] // 32)):
        e = s["e"][:, k:k + 1].double()
        x[:, 32 * k:32 * k + 32] = s["q"][:, 32 * k:min(32 * k + 32, c["n_in"])].double() * torch.pow(2.0, e - 133)
    off = s["offsets"].tolist() if s["offsets"] is not None else [0, c["rows"]]
    out = torch.zeros((c["groups"], c["n_out"], c["n_in"]), device="cuda", dtype=torch.float64)
    for i in range(c["groups"]):
        a, b = off[i], off[i + 1]
        if b > a:
            out[i] = s["dy"][a:b].double().t() @ x[a:b]
    if c["accumulate"]:
        out += s["grad"].double()
    return out
