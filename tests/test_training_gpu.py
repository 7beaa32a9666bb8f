"""GPU tests of the training operators (embedding, policy loss, 8-bit
activations, weight gradients) against their definitions in 64 bits.

Tolerances are rounding bounds, element by element, written where they are
used. U is the unit roundoff of the output type (half a unit in the last
place, relative), E = 2^-24 that of fp32 arithmetic."""
import math

import pytest
import torch

from newton_schulz_quintic_gb300 import api

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
E = 2.0 ** -24
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from newton_schulz_quintic_gb300 import build
    build.build()
    api.load_library()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(shape, g, dtype=F32, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def within(got, ref, bound):
    """Every element of got within bound of ref (NaN where ref is NaN)."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan)
    same = got == ref  # infinities
    bad = ~(nan | same | ((got - ref).abs() <= bound))
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs()[bad].max()))


def padded(x, extra, shift=0):
    """x as a view with a longer row pitch, `shift` elements into its buffer;
    returns (view, buffer)."""
    n, m = x.shape
    buf = torch.full((n * (m + extra) + shift + 64,), 7.0, dtype=x.dtype, device=x.device)
    v = buf[shift:shift + n * (m + extra)].view(n, m + extra)[:, :m]
    v.copy_(x)
    return v, buf


# ------------------------------------------------------------------ embedding
def make_ids(n, vocab, g, hot=0.3, pad=0.1, dtype=torch.int64):
    ids = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    r = torch.rand(n, device="cuda", generator=g)
    ids[r < hot] = vocab // 2
    ids[r > 1 - pad] = -1
    return ids.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,vocab,dim,idt", [(1, 1, 1, torch.int32), (1, 300, 4096, torch.int64), (33, 7, 130, torch.int64),
                                             (257, 1000, 1023, torch.int32), (1000, 511, 2304, torch.int64)])
def test_lookup(dtype, n, vocab, dim, idt):
    g = gen(n + dim)
    table, ids = normal((vocab, dim), g, dtype, 0.02), make_ids(n, vocab, g, dtype=idt)
    if n > 40:
        ids[5], ids[6] = vocab, -(1 << 30)  # outside on either side
    out = api.embed_lookup(table, ids, scale=1.7)
    live = (ids >= 0) & (ids < vocab)
    ref = table[ids.long().clamp(0, vocab - 1)].double() * float(torch.tensor(1.7)) * live[:, None]
    within(out, ref, ref.abs() * (U[dtype] + 2 * E))
    assert torch.all(out[~live] == 0)


def test_lookup_views_shapes_and_long_ids():
    g = gen(1)
    table = normal((100, 64), g, BF16)
    wide, _ = padded(table, 8, 3)  # rows 16 bytes longer, base 6 bytes off
    ids = make_ids(24, 100, g).view(2, 3, 4)
    a = api.embed_lookup(table, ids)
    assert a.shape == (2, 3, 4, 64)
    assert torch.equal(a, api.embed_lookup(wide, ids))
    out, buf = padded(torch.zeros(24, 64, dtype=BF16, device="cuda"), 3)
    assert api.embed_lookup(table, ids, out=out) is out
    assert torch.equal(out, a.view(24, 64))
    assert torch.all(buf.view(-1)[-64:] == 7) and torch.all(buf[:24 * 67].view(24, 67)[:, 64:] == 7)
    ids = torch.full((4,), (1 << 33) + 5, device="cuda")  # wraps to a valid id in 32 bits
    assert torch.all(api.embed_lookup(table, ids) == 0)
    assert api.embed_lookup(table, ids[:0]).shape == (0, 64)


def test_lookup_past_32_bit_offsets():
    vocab, dim = (1 << 20) + 3, 2304  # 2.4e9 elements
    table = torch.empty((vocab, dim), dtype=BF16, device="cuda")
    table[-2:] = normal((2, dim), gen(2), BF16)
    out = api.embed_lookup(table, torch.tensor([vocab - 1, vocab - 2], device="cuda"))
    assert torch.equal(out, table[[vocab - 1, vocab - 2]])


def embed_reference(dout, ids, vocab, scale):
    live = (ids >= 0) & (ids < vocab)
    total = torch.zeros((vocab, dout.shape[1]), dtype=F64, device="cuda")
    mag = torch.zeros_like(total)
    k = ids[live].long()
    total.index_put_((k,), dout[live].double(), accumulate=True)
    mag.index_put_((k,), dout[live].double().abs(), accumulate=True)
    most = int(torch.bincount(k, minlength=1).max()) if k.numel() else 0
    s = float(torch.tensor(scale, dtype=F32))
    return total * s, mag * abs(s), most


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (3, 5000, 64), (61, 9, 130), (509, 1021, 1023), (4096, 300, 256),
                                         (9001, 40000, 136), (20000, 131072, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad(dtype, gdtype, n, vocab, dim, accumulate):
    g = gen(n + dim)
    ids, dout = make_ids(n, vocab, g), normal((n, dim), g, dtype)
    dout[ids < 0] = NAN  # rows of padding are not read
    old = normal((vocab, dim), g, gdtype)
    ref, mag, most = embed_reference(dout, ids, vocab, 0.37)
    if accumulate:
        got = api.embed_grad(dout, ids, grad=old.clone(), scale=0.37, accumulate=True)
        ref, mag = ref + old.double(), mag + old.double().abs()
        untouched = torch.ones(vocab, dtype=torch.bool, device="cuda")
        untouched[ids[ids >= 0]] = False
        assert torch.equal(got[untouched], old[untouched])
    else:
        got = api.embed_grad(dout, ids, vocab=vocab, scale=0.37, dtype=gdtype)
    # sums of at most `most` terms in fp32 in any order, scaled and added: (most + 2) roundings of at most mag
    within(got, ref, (most + 2) * E * mag + U[gdtype] * ref.abs() * (1 + 2 ** -7))
    if not accumulate:
        assert torch.equal(got, api.embed_grad(dout, ids, vocab=vocab, scale=0.37, dtype=gdtype))  # same bits again


@pytest.mark.parametrize("n", [40, 30011])
def test_embed_grad_edges(n):
    g = gen(3)
    vocab, dim = 70001, 40
    dout = normal((n, dim), g, BF16)
    for ids in (torch.full((n,), vocab - 1, device="cuda"), torch.full((n,), 0, device="cuda"),
                torch.full((n,), -1, device="cuda"), torch.full((n,), vocab, device="cuda"),
                torch.arange(n, device="cuda"), torch.arange(n, device="cuda") // 32, torch.arange(n, device="cuda") // 33,
                torch.randint(0, vocab, (n,), device="cuda", generator=g, dtype=torch.int32)):
        ref, mag, most = embed_reference(dout, ids, vocab, 1.0)
        within(api.embed_grad(dout, ids, vocab=vocab), ref, (most + 2) * E * mag + U[BF16] * ref.abs() * (1 + 2 ** -7))
    empty = api.embed_grad(dout[:0], ids[:0], vocab=vocab)
    assert torch.all(empty == 0)
    kept = normal((vocab, dim), g, F32)
    assert torch.equal(api.embed_grad(dout[:0], ids[:0], grad=kept.clone(), accumulate=True), kept)


def test_embed_grad_of_many_positions_and_strided_buffers():
    g = gen(4)
    n, vocab, dim = 70001, 3001, 24
    ids = make_ids(n, vocab, g)
    dout, _ = padded(normal((n, dim), g, BF16), 5, 1)
    grad, buf = padded(torch.zeros((vocab, dim), device="cuda"), 9, 3)
    api.embed_grad(dout, ids, grad=grad)
    ref, mag, most = embed_reference(dout, ids, vocab, 1.0)
    within(grad, ref, (most + 2) * E * mag)
    assert torch.all(buf[:3] == 7) and torch.all(buf[3:3 + vocab * 33].view(vocab, 33)[:, dim:] == 7)


def test_embed_grad_is_the_derivative_of_lookup():
    # L = sum(w * lookup(T)) is linear in T: its differences are exact up to rounding
    g = gen(5)
    vocab, dim, n = 50, 12, 200
    table, ids, w = normal((vocab, dim), g), make_ids(n, vocab, g), normal((n, dim), g)
    grad = api.embed_grad(w, ids, vocab=vocab, scale=2.0)
    for v, c in [(25, 3), (0, 0), (49, 11), (7, 5)]:
        up, down = table.clone(), table.clone()
        up[v, c] += 0.5
        down[v, c] -= 0.5
        h = float(up[v, c].double() - down[v, c].double())
        diff = (w.double() * (api.embed_lookup(up, ids, 2.0).double() - api.embed_lookup(down, ids, 2.0).double())).sum() / h
        # each difference of looked-up values carries two roundings of values below 8, times |w|, over h = 1
        tol = float((w[ids == v, c].double().abs().sum() + 1) * 4 * 16 * E) + 200 * E * abs(float(diff))
        assert abs(float(diff) - float(grad[v, c])) <= tol


# ------------------------------------------------------------------ policy loss
def policy_reference(x, y, adv, w, old, ref, low, high, beta, temp):
    """loss, logp, kl, dlogits, slope in float64 by the definition."""
    n, vocab = x.shape
    live = (y >= 0) & (y < vocab) & (w != 0)
    live &= ~torch.all(x == -INF, dim=1)
    z = torch.where(live[:, None], x.double() / temp, torch.zeros((), dtype=F64, device="cuda"))
    lse = torch.logsumexp(z, -1)
    yy = torch.where(live, y.long(), torch.zeros_like(y.long()))
    lp = z.gather(1, yy[:, None])[:, 0] - lse
    r = torch.exp(lp - old.double()) if old is not None else torch.ones_like(lp)
    a, wd = adv.double(), w.double()
    gain = torch.minimum(r * a, r.clamp(1 - low, 1 + high) * a)
    slope = torch.where(r * a <= r.clamp(1 - low, 1 + high) * a, -r * a, torch.zeros_like(a))
    k = torch.zeros_like(lp)
    if ref is not None:
        d = ref.double() - lp
        k = torch.exp(d) - d - 1
        slope = slope + beta * (1 - torch.exp(d))
    zero = torch.zeros_like(lp)
    loss = torch.where(live, wd * (beta * k - gain), zero)
    slope = torch.where(live, wd * slope / temp, zero)
    p = torch.exp(z - lse[:, None])
    g = -slope[:, None] * p
    g[torch.arange(n, device="cuda"), yy] += slope
    return loss, torch.where(live, lp, zero), torch.where(live, k, zero), g, slope, p * live[:, None], z, live


def policy_bounds(x, z, temp):
    """Bound on |logp - exact|: z and z - max rounded (4 E max|z|), the exp of a
    sum's terms (2 ulp of the hardware's exponential and E |z - max| of its
    argument, at most 2^-20 of the sum since x exp(-x) < 1), the additions
    (a chain of vocab / 128 + 64 at most), the logarithm (2 ulp of at most 12)."""
    vocab = x.shape[1]
    near = z > z.amax(1, keepdim=True) - 100  # the others add nothing
    top = torch.where(near, z.abs(), torch.zeros_like(z)).amax(1)
    return 4 * E * top + 2.0 ** -20 + (vocab / 128 + 64) * E + 24 * 2 * E


def make_policy(n, vocab, dtype, seed, ragged=0):
    g = gen(seed)
    x = normal((n, vocab), g, dtype, 2.0)
    y = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    x[torch.arange(n, device="cuda"), y] += 4
    if ragged:
        x, _ = padded(x, ragged, 1)
    lp = torch.log_softmax(x.double(), -1).gather(1, y[:, None])[:, 0].float()
    old, ref = lp + 0.3 * normal((n,), g), lp + 0.3 * normal((n,), g)
    return x, y, normal((n,), g), torch.rand(n, device="cuda", generator=g) + 0.1, old, ref


def check_policy(x, y, adv, w, old, ref, low=0.2, high=0.28, beta=0.05, temp=1.0, **kw):
    got = api.policy_loss(x, y, adv, w, old_logp=old, ref_logp=ref, clip_low=low, clip_high=high, kl_coef=beta,
                          temperature=temp, **kw)
    loss, lp, k, g, slope, p, z, live = policy_reference(x, y, adv, w, old, ref, low, high, beta, temp)
    tol = policy_bounds(x, z, temp)
    within(got.logp, lp, tol * live)
    # r and exp(d) move with logp: relative tol + 4 ulp; k = (e^d - 1) - d cancels, so its error is absolute
    d = ref.double() - lp if ref is not None else torch.zeros_like(lp)
    ktol = torch.where(live, (torch.exp(d) - 1).abs() * (tol + 4 * E) + (torch.exp(d) + 1 + d.abs()) * 4 * E, 0 * lp)
    within(got.kl, k, ktol)
    r = torch.exp(lp - old.double()) if old is not None else torch.ones_like(lp)
    ltol = torch.where(live, w.double() * (r * adv.double().abs() * (tol + 8 * E) + beta * (ktol + 4 * E)), 0 * lp)
    total = loss.sum()
    assert abs(float(got.loss) - float(total)) <= float(ltol.sum() + (12 + x.shape[0] / 1024) * E * loss.abs().sum())
    if kw.get("grad", True):
        stol = torch.where(live, w.double() / temp * (r * adv.double().abs() * (tol + 8 * E)
                                                      + beta * (torch.exp(d) + 1) * (tol + 8 * E)), 0 * lp)
        ptol = p * (2 * tol[:, None] + 2.0 ** -20)
        bound = stol[:, None] * (p + (torch.arange(x.shape[1], device="cuda") == y.long()[:, None])) \
            + slope.abs()[:, None] * (ptol + 4 * E * p)
        within(got.dlogits, g, bound + U[x.dtype] * g.abs() * (1 + 2 ** -7) + 1e-37)
    else:
        assert got.dlogits is None
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,vocab,ragged", [(1, 2, 0), (1, 131072, 0), (3, 33, 0), (5, 1000, 8), (17, 50021, 0), (40, 4096, 0),
                                            (9, 32767, 3), (4, 262147, 0), (2, 600000, 0)])
def test_policy_loss(dtype, n, vocab, ragged):
    x, y, adv, w, old, ref = make_policy(n, vocab, dtype, n + vocab, ragged)
    got = check_policy(x, y, adv, w, old, ref)
    again = api.policy_loss(x, y, adv, w, old_logp=old, ref_logp=ref, clip_high=0.28, kl_coef=0.05)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    within(api.token_logprobs(x, y), got.logp, 0)
    check_policy(x, y, adv, w, None, None, temp=0.5)
    check_policy(x, y.int(), adv, w, old, None, beta=0.0, grad=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [129, 40000, 40001])
def test_policy_masks_infinities_and_nan(dtype, vocab):
    n = 24
    x, y, adv, w, old, ref = make_policy(n, vocab, dtype, 11)
    y[0], y[1] = -100, vocab          # no target
    w[2] = 0                          # no weight
    x[:3] = NAN                       # masked rows hold anything,
    adv[:3], old[:3], ref[:3] = NAN, INF, NAN
    x[3] = -INF                       # no distribution
    x[4:8, ::2] = -INF                # masked vocabulary entries
    x[4:8, 1::4] = torch.finfo(dtype).min
    for t in range(4, 8):
        y[t] = 3
        x[t, 3] = 0.5
    x[8, 5] = torch.finfo(dtype).max  # one certain token
    y[8] = 5
    old[4:9], ref[4:9] = -1.0, -1.0
    got = check_policy(x, y, adv, w, old, ref)
    assert torch.all(got.dlogits[:4] == 0) and torch.all(got.logp[:4] == 0) and torch.all(got.kl[:4] == 0)
    assert torch.isfinite(got.loss)
    x[9, 7] = NAN                     # a NaN that counts reaches its own row and the loss, nothing else
    bad = api.policy_loss(x, y, adv, w, old_logp=old, ref_logp=ref, clip_high=0.28, kl_coef=0.05)
    assert torch.isnan(bad.logp[9]) and torch.isnan(bad.dlogits[9]).all() and torch.isnan(bad.loss)
    keep = torch.arange(n, device="cuda") != 9
    assert torch.equal(bad.dlogits[keep], got.dlogits[keep]) and torch.equal(bad.logp[keep], got.logp[keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [65, 40000])
@pytest.mark.parametrize("temp", [1.0, 0.05, 40.0])
def test_policy_rows_of_the_types_extreme_values(dtype, vocab, temp):
    # rows of one value are uniform whatever it is: logp = -log(vocab); next to -inf or smaller values those have none
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).min
    x = torch.empty((6, vocab), dtype=dtype, device="cuda")
    x[0], x[1], x[2] = low, top, low
    x[2, ::2] = -INF
    x[3], x[4], x[5] = low, -INF, top
    x[3, :3] = 0
    x[4, 1] = low
    x[5, 1::2] = 0
    y = torch.tensor([5, 5, 5, 1, 1, 6], device="cuda")
    live = torch.tensor([vocab, vocab, vocab // 2, 3, 1, (vocab + 1) // 2], device="cuda").double()
    got = api.policy_loss(x, y, torch.ones(6, device="cuda"), torch.ones(6, device="cuda"), temperature=temp)
    within(got.logp, -live.log(), policy_bounds(torch.zeros_like(x), torch.zeros_like(x).double(), 1.0))
    # on-policy with A = 1: the gradient is softmax - onehot over the temperature
    p = torch.zeros((6, vocab), dtype=F64, device="cuda")
    p[0], p[1], p[2, 1::2], p[3, :3], p[4, 1], p[5, ::2] = (float(1 / n) for n in live)
    p[torch.arange(6, device="cuda"), y] -= 1
    # the softmax carries the sum's error (policy_bounds') and one of its own, the type one rounding
    within(got.dlogits, p / temp, (p.abs() + (p < 0)) / temp * ((vocab / 128 + 200) * E + 2.0 ** -18 + U[dtype]))


def test_policy_in_place_and_no_rows():
    x, y, adv, w, old, ref = make_policy(37, 30001, BF16, 5)
    a = api.policy_loss(x, y, adv, w, old_logp=old)
    z = x.clone()
    b = api.policy_loss(z, y, adv, w, old_logp=old, dlogits=z)
    assert b.dlogits is z and torch.equal(a.dlogits, z) and torch.equal(a.loss, b.loss)
    out, buf = padded(torch.zeros_like(x), 11, 2)
    api.policy_loss(x, y, adv, w, old_logp=old, dlogits=out)
    assert torch.equal(out, z) and torch.all(buf[2:2 + 37 * 30012].view(37, 30012)[:, 30001:] == 7)
    e = api.policy_loss(x[:0], y[:0], adv[:0], w[:0])
    assert float(e.loss) == 0 and e.dlogits.shape == (0, 30001)
    assert api.token_logprobs(x[:0], y[:0]).shape == (0,)


def test_policy_many_rows():
    x, y, adv, w, old, ref = make_policy(5000, 700, BF16, 6)
    check_policy(x, y, adv, w, old, ref)


def test_policy_gradient_by_differences():
    # central differences of the definition in 64 bits: error h^2 / 6 times a third derivative below 8 |slope|
    x, y, adv, w, old, ref = make_policy(6, 40, F32, 7)
    got = api.policy_loss(x, y, adv, w, old_logp=old, ref_logp=ref, kl_coef=0.1)
    h = 1e-4
    for t in range(6):
        r = math.exp(float(got.logp[t] - old[t]))
        if min(abs(r - 0.8), abs(r - 1.2)) < 1e-3:
            continue  # at the kink
        for j in (int(y[t]), 0, 39):
            d = torch.zeros((6, 40), dtype=F64, device="cuda")
            d[t, j] = h
            f = [policy_reference(x.double() + s * d, y, adv, w, old, ref, 0.2, 0.2, 0.1, 1.0)[0].sum() for s in (1, -1)]
            assert abs(float((f[0] - f[1]) / (2 * h)) - float(got.dlogits[t, j])) <= 1e-5 * (1 + abs(float(adv[t])))


# ------------------------------------------------------------------ 8-bit activations
def power_of_two(k):
    """2^k in float64 from its bits (torch.pow on the GPU is off by a unit in the last place)."""
    return ((k.long() + 1023) << 52).view(F64)


def held_reference(x):
    """(q, E) of the 8-bit form in 64 bits, without padding."""
    n, m = x.shape
    blocks = -(-m // 32)
    b = torch.zeros((n, blocks * 32), dtype=F64, device="cuda")
    b[:, :m] = x.double()
    b = b.view(n, blocks, 32)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    top = torch.where(bad, torch.ones_like(top), top)
    e = torch.where(top > 0, torch.frexp(top).exponent + 126, torch.full_like(top, 7).int()).clamp(min=7)
    q = (b * power_of_two(133 - e)[..., None]).round().clamp(-127, 127)
    q[bad] = 0
    e[bad] = 255
    return q.view(n, -1)[:, :m], e


def held_values(q, e, m):
    unit = torch.where(e == 255, torch.full_like(e.double(), NAN), power_of_two(e - 133))
    return q.double() * unit.repeat_interleave(32, 1)[:, :m]


def special(x):
    """Zeros, tiny, huge and non-finite values in blocks of their own."""
    n, m = x.shape
    x[0] = 0
    if n > 4:
        x[1] *= 1e-38
        x[2, : min(m, 32)] = torch.finfo(x.dtype).max
        x[3, 0] = INF
        x[4, m - 1] = NAN
        x[n - 1] = 1e-44 if x.dtype == F32 else 1e-40
    return x


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,m", [(1, 1), (1, 16), (3, 31), (5, 32), (7, 48), (9, 2303), (33, 1024), (130, 6143), (64, 4112)])
def test_store_and_load_exactly(dtype, n, m):
    g = gen(n * m)
    x = special((normal((n, m), g) * torch.exp(3 * normal((n, 1), g))).to(dtype))
    for view in (x, padded(x, 8, 0)[0], padded(x, 1, 1)[0]):
        ck = api.checkpoint_store(view)
        q, e = held_reference(x)
        assert torch.equal(ck.q[:, :m].double(), q) and torch.equal(ck.scales[:, :e.shape[1]].int(), e.int())
        assert torch.all(ck.q[:, m:] == 0) and torch.all(ck.scales[:, e.shape[1]:] == 0)
        ref = held_values(q, e, m)
        for dt in (BF16, F32):
            got = api.checkpoint_load(ck, dtype=dt)
            within(got, ref, 0)  # exact in either type
            out, buf = padded(torch.zeros((n, m), dtype=dt, device="cuda"), 5, 1)
            assert torch.equal(torch.nan_to_num(api.checkpoint_load(ck, out=out)), torch.nan_to_num(got))
            assert torch.all(buf[1:1 + n * (m + 5)].view(n, m + 5)[:, m:] == 7)


def test_store_error_bound():
    # half a unit, a unit being at most 1/64 of the block's largest magnitude; one unit where 127 holds 127.5 .. 128
    x = normal((257, 4096), gen(9))
    ref = x.double().view(257, 128, 32).abs().amax(-1, keepdim=True).expand(-1, -1, 32).reshape(257, 4096)
    err = (api.checkpoint_load(api.checkpoint_store(x), dtype=F32).double() - x.double()).abs()
    assert torch.all(err <= ref / 128 * (1 + 1e-9))


def gated_reference(g, u, dh):
    s = torch.sigmoid(g)
    return g * s * u, dh * u * (s + g * s * (1 - s)), dh * g * s


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,f", [(1, 1), (2, 33), (5, 2303), (64, 1024), (301, 48), (12, 14336)])
@pytest.mark.parametrize("halves", [True, False])
def test_gated(dtype, n, f, halves):
    r = gen(n * f)
    gu = normal((n, 2 * f), r, dtype, 2.0)
    gate, up = (gu[:, :f], gu[:, f:]) if halves else (gu[:, :f].contiguous(), gu[:, f:].contiguous())
    dh = normal((n, f), r, dtype)
    h, a, b = api.gated_forward(gate, up)
    href, _, _ = gated_reference(gate.double(), up.double(), dh.double())
    # sigmoid: exp within 2 ulp + |x| E of its argument, add, divide: (8 + |x|) E; two products; one rounding
    sig = lambda x: (12 + 2 * x.abs()) * E  # noqa: E731
    within(h, href, href.abs() * (sig(gate.double()) + U[dtype] * (1 + 2 ** -7)) + 1e-37)
    for ck, x in ((a, gate), (b, up)):
        q, e = held_reference(x)
        assert torch.equal(ck.q[:, :f].double(), q) and torch.equal(ck.scales[:, :e.shape[1]].int(), e.int())
        assert torch.all(ck.q[:, f:] == 0) and torch.all(ck.scales[:, e.shape[1]:] == 0)
    dgu, again = api.gated_backward(dh, a, b)
    g8, u8 = api.checkpoint_load(a, dtype=F32).double(), api.checkpoint_load(b, dtype=F32).double()
    hh, dg, du = gated_reference(g8, u8, dh.double())
    s = torch.sigmoid(g8)
    mag = (dh.double() * u8).abs() * s * (1 + g8.abs() * (1 - s))  # the gate's slope may cancel: bound by its parts
    within(again, hh, hh.abs() * (sig(g8) + U[dtype] * (1 + 2 ** -7)) + 1e-37)
    within(dgu[:, f:], du, du.abs() * (sig(g8) + U[dtype] * (1 + 2 ** -7)) + 1e-37)
    within(dgu[:, :f], dg, mag * 2 * (sig(g8) + 4 * E) + U[dtype] * dg.abs() * (1 + 2 ** -7) + 1e-37)
    assert api.gated_backward(dh, a, b, recompute=False)[1] is None
    assert torch.equal(api.gated_backward(dh, a, b, recompute=False)[0], dgu)


def test_gated_extremes():
    gate = torch.tensor([[100.0, -100.0, 0.0, -0.0, 1e30, -1e30, 88.0, -88.0]], device="cuda")
    up = torch.full_like(gate, 2.0)
    h, a, b = api.gated_forward(gate, up)
    within(h, torch.tensor([[200.0, 0, 0, 0, 2e30, 0, 176.0, 0]], device="cuda"), 1e-5 * h.double().abs() + 1e-30)
    dgu, _ = api.gated_backward(torch.ones_like(gate), a, b)
    assert torch.isfinite(dgu).all()
    bad = torch.full((2, 64), 1.0, device="cuda", dtype=BF16)
    bad[0, 40] = INF
    h, a, b = api.gated_forward(bad, torch.ones_like(bad))
    dgu, _ = api.gated_backward(torch.ones_like(bad), a, b)
    assert torch.isnan(dgu[0, 32:64]).all() and torch.isfinite(dgu[0, :32]).all() and torch.isfinite(dgu[1]).all()


def test_gated_backward_by_differences():
    # at the held values, in 64 bits: central differences with error h^2 / 6 times a third derivative below 1
    r = gen(8)
    gate, up, dh = normal((4, 96), r), normal((4, 96), r), normal((4, 96), r)
    _, a, b = api.gated_forward(gate, up)
    dgu, _ = api.gated_backward(dh, a, b)
    g8, u8 = api.checkpoint_load(a, dtype=F32).double(), api.checkpoint_load(b, dtype=F32).double()
    f = lambda g, u: (g * torch.sigmoid(g) * u * dh.double())  # noqa: E731
    h = 1e-4
    dg = (f(g8 + h, u8) - f(g8 - h, u8)) / (2 * h)
    du = (f(g8, u8 + h) - f(g8, u8 - h)) / (2 * h)
    scale = (dh.double() * (1 + u8.abs())).abs()
    within(dgu[:, :96], dg, 1e-6 * scale)
    within(dgu[:, 96:], du, 1e-6 * scale * (1 + g8.abs()))


# ------------------------------------------------------------------ weight gradients
def wgrad_reference(dy, ck, off):
    x = api.checkpoint_load(ck, dtype=F32).double()
    out, mag = [], []
    for a, b in zip(off, off[1:]):
        d = dy[a:b].double()
        out.append(d.t() @ x[a:b])
        mag.append(d.abs().t() @ x[a:b].abs())
    return torch.stack(out), torch.stack(mag)


def wgrad_bound(mag, ref, gdtype, longest, dtype):
    """The tensor cores lose up to one ulp (2 E) of a partial sum per 16 rows for
    at most 512 rows (three times over for fp32's slices), then one fp32
    addition per 512 rows and per part of a split group; CUDA-core sums would
    stay below that too. Partial sums are at most mag."""
    parts = 3 if dtype == F32 else 1
    return (parts * 32 * 2 + longest / 512 + 160) * E * mag + U[gdtype] * ref.abs() * (1 + 2 ** -7) + 1e-37


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gdtype", [BF16, F32])
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 256, 256), (17, 33, 70), (64, 128, 512), (65, 300, 257), (300, 640, 1000),
                                   (1023, 129, 2303), (5000, 64, 96), (2048, 520, 776), (700, 1031, 1024)])
def test_wgrad(dtype, gdtype, t, n, k):
    r = gen(t + n + k)
    dy, ck = normal((t, n), r, dtype), api.checkpoint_store(normal((t, k), r))
    ref, mag = wgrad_reference(dy, ck, [0, t])
    got = api.checkpoint_wgrad(dy, ck, dtype=gdtype)
    assert got.shape == (1, n, k)
    within(got, ref, wgrad_bound(mag, ref, gdtype, t, dtype))
    assert torch.equal(got, api.checkpoint_wgrad(dy, ck, dtype=gdtype))
    old = normal((1, n, k), r, gdtype)
    acc = api.checkpoint_wgrad(dy, ck, grad=old.clone(), accumulate=True)
    total = ref + old.double()
    within(acc, total, wgrad_bound(mag + old.double().abs(), total, gdtype, t, dtype))
    view, _ = padded(dy, 3, 1)
    within(api.checkpoint_wgrad(view, ck, dtype=gdtype), ref, wgrad_bound(mag, ref, gdtype, t, dtype))
    view, _ = padded(dy, 8, 0)
    within(api.checkpoint_wgrad(view, ck, dtype=gdtype), ref, wgrad_bound(mag, ref, gdtype, t, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("off,n,k", [([0, 0, 64, 65, 300, 300], 130, 260), ([0, 1, 2, 3, 4], 256, 64), ([5, 70, 190], 64, 512),
                                     ([0, 0, 0], 32, 32), ([0, 700, 701, 1400, 1500], 260, 300)])
def test_wgrad_groups(dtype, off, n, k):
    r = gen(sum(off) + n)
    t = off[-1] + 9  # rows after the last group
    dy, x = normal((t, n), r, dtype), normal((t, k), r)
    ck = api.checkpoint_store(x)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    ref, mag = wgrad_reference(dy, ck, off)
    longest = max(b - a for a, b in zip(off, off[1:]))
    got = api.checkpoint_wgrad(dy, ck, offsets=offsets, dtype=F32)
    within(got, ref, wgrad_bound(mag, ref, F32, longest, dtype))
    old = normal(tuple(ref.shape), r, BF16)
    acc = api.checkpoint_wgrad(dy, ck, offsets=offsets, grad=old.clone(), accumulate=True)
    total = ref + old.double()
    within(acc, total, wgrad_bound(mag + old.double().abs(), total, BF16, longest, dtype))
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if a == b:
            assert torch.all(got[e] == 0) and torch.equal(acc[e], old[e])
    # rows of other groups, and rows of none, never reach a group's sum
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if b <= a:
            continue
        poisoned, px = torch.full_like(dy, NAN), torch.full_like(x, INF)
        poisoned[a:b], px[a:b] = dy[a:b], x[a:b]
        one = api.checkpoint_wgrad(poisoned, api.checkpoint_store(px), offsets=offsets, dtype=F32)
        assert torch.equal(one[e], got[e])


def test_wgrad_nan_reaches_its_columns_only():
    r = gen(12)
    dy, x = normal((100, 64), r, BF16), normal((100, 96), r)
    x[50, 40] = NAN  # the block of columns 32..63
    g = api.checkpoint_wgrad(dy, api.checkpoint_store(x), dtype=F32)[0]
    assert torch.isnan(g[:, 32:64]).all() and torch.isfinite(g[:, :32]).all() and torch.isfinite(g[:, 64:]).all()
    dy[3, 5] = INF
    x[50, 40] = 0
    g = api.checkpoint_wgrad(dy, api.checkpoint_store(x), dtype=F32)[0]
    rest = torch.arange(64, device="cuda") != 5
    assert torch.isfinite(g[rest]).all() and not torch.isfinite(g[5]).any()


def test_wgrad_fp32_beyond_bf16s_largest_value():
    # FLT_MAX rounds to infinity in bf16: its first slice has to stop below, the rest follows in the next ones
    r = gen(16)
    dy, x = normal((64, 40), r), normal((64, 64), r)
    big = torch.finfo(F32).max
    dy[7], x[7] = big, 0.25
    dy[8], x[8] = -big, 0.125
    ck = api.checkpoint_store(x)
    ref, mag = wgrad_reference(dy, ck, [0, 64])
    got = api.checkpoint_wgrad(dy, ck)
    assert torch.isfinite(got).all()
    within(got, ref, wgrad_bound(mag, ref, F32, 64, F32))


def test_wgrad_widens_x_the_same_way_in_one_launch_and_before():
    # a bf16 dY whose rows TMA reads has X widened within the product's launch, one off 16 bytes before it; the
    # sizes follow one another on a stream, larger and smaller, so each call has to leave its counters as it found them
    for t, n, k, groups in [(70, 40, 64, 1), (3000, 600, 1000, 5), (1, 8, 32, 1), (2100, 264, 520, 3), (3000, 600, 1000, 5),
                            (513, 1032, 2304, 1), (70, 40, 64, 1)]:
        r = gen(t + n + k)
        dy, ck = normal((t, n), r, BF16), api.checkpoint_store(normal((t, k), r))
        cuts = [0] + sorted(torch.randint(0, t + 1, (groups - 1,), generator=torch.Generator().manual_seed(t)).tolist()) + [t]
        offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda") if groups > 1 else None
        got = api.checkpoint_wgrad(dy, ck, offsets=offsets, dtype=F32)
        ref, mag = wgrad_reference(dy, ck, cuts)
        within(got, ref, wgrad_bound(mag, ref, F32, t, BF16))
        view, _ = padded(dy, 3, 1)
        assert torch.equal(got, api.checkpoint_wgrad(view, ck, offsets=offsets, dtype=F32))
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(got)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.checkpoint_wgrad(dy, ck, grad=out, stream=side)
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        api.checkpoint_wgrad(dy, ck, grad=out, stream=side)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)


def test_wgrad_beside_other_work():
    # the launch whose CTAs wait for one another, on two streams at once and beside kernels that fill the GPU
    r = gen(17)
    work = [(normal((t, n), r, BF16), api.checkpoint_store(normal((t, k), r))) for t, n, k in [(700, 1100, 2000), (1500, 500, 3000)]]
    logits, targets = normal((600, 9000), r, BF16), torch.randint(0, 9000, (600,), device="cuda", generator=r)
    ref = [api.checkpoint_wgrad(dy, ck, dtype=F32) for dy, ck in work]
    logp = api.token_logprobs(logits, targets)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, (dy, ck) in zip(streams, work):
            got.append(api.checkpoint_wgrad(dy, ck, dtype=F32, stream=s))
        got.append(api.token_logprobs(logits, targets, stream=streams[2]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, (*ref, logp)[i % 3]) for i, g in enumerate(got))
    assert api.get_status() == 0


def test_wgrad_offsets_are_clamped():
    r = gen(13)
    dy, ck = normal((50, 32), r, BF16), api.checkpoint_store(normal((50, 64), r))
    a = api.checkpoint_wgrad(dy, ck, offsets=torch.tensor([-5, 20, 10, 99], dtype=torch.int32, device="cuda"), dtype=F32)
    b = api.checkpoint_wgrad(dy, ck, offsets=torch.tensor([0, 20, 20, 20], dtype=torch.int32, device="cuda"), dtype=F32)
    assert torch.equal(a[0], b[0]) and torch.all(a[1] == 0)


def test_wgrad_no_rows():
    r = gen(14)
    dy, ck = normal((0, 40), r, BF16), api.checkpoint_store(normal((0, 64), r))
    assert torch.all(api.checkpoint_wgrad(dy, ck) == 0)
    old = normal((1, 40, 64), r)
    assert torch.equal(api.checkpoint_wgrad(dy, ck, grad=old.clone(), accumulate=True), old)


def test_wgrad_by_differences():
    # L(W) = sum(dy * (X W^T)) is linear: a difference quotient in 64 bits is the gradient itself
    r = gen(15)
    dy, ck = normal((70, 40), r), api.checkpoint_store(normal((70, 96), r))
    x, w = api.checkpoint_load(ck, dtype=F32).double(), normal((40, 96), r).double()
    got = api.checkpoint_wgrad(dy, ck)[0]
    for i, j in [(0, 0), (39, 95), (17, 33)]:
        d = torch.zeros_like(w)
        d[i, j] = 1.0
        diff = float((dy.double() * (x @ (w + d).t() - x @ (w - d).t())).sum() / 2)
        bound = float((dy[:, i].double().abs() * x[:, j].abs()).sum()) * 256 * E
        assert abs(diff - float(got[i, j])) <= bound + 1e-9


# ------------------------------------------------------------------ streams, graphs, launches
def everything(seed, stream=None):
    r = gen(seed)
    ids = make_ids(777, 3000, r)
    table, dout = normal((3000, 256), r, BF16), normal((777, 256), r, BF16)
    x, y, adv, w, old, ref = make_policy(65, 5000, BF16, seed)
    gu, dh = normal((130, 512), r, BF16), normal((130, 256), r, BF16)
    torch.cuda.synchronize()

    def go():
        out = [api.embed_lookup(table, ids, 2.0, stream=stream), api.embed_grad(dout, ids, vocab=3000, stream=stream)]
        p = api.policy_loss(x, y, adv, w, old_logp=old, ref_logp=ref, kl_coef=0.1, stream=stream)
        h, a, b = api.gated_forward(gu[:, :256], gu[:, 256:], stream=stream)
        dgu, again = api.gated_backward(dh, a, b, stream=stream)
        g = api.checkpoint_wgrad(dgu, a, stream=stream)
        return out + [p.loss, p.logp, p.kl, p.dlogits, h, dgu, again, g, api.checkpoint_load(b, stream=stream)]
    return go


def test_other_streams_and_graph():
    ref = everything(3)()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = everything(3, side)()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    go = everything(3)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        go()
    s.synchronize()
    before = api.num_workspace_allocations()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = go()
    assert api.num_workspace_allocations() == before
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    assert api.get_status() == 0


def test_launches_are_counted_and_timed():
    go = everything(4)
    go()
    before = api.num_kernel_launches()
    api.set_kernel_timing(True)
    go()
    t = api.kernel_times()
    api.set_kernel_timing(False)
    for kind in ("embed_lookup", "embed_grad", "policy", "checkpoint", "wgrad"):
        assert t[kind][1] > 0 and t[kind][0] > 0, kind
    assert api.num_kernel_launches() - before >= sum(launches for _, launches in t.values()) >= 5
