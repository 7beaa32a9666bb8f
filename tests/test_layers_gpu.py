"""GPU tests of the expert-layer operators (router, 8-bit blocks and their
product, block norms, dropout) against their definitions in 64 bits.

Tolerances are rounding bounds, element by element, written where they are
used. U is the unit roundoff of the output type (half a unit in the last place,
relative), E = 2^-24 that of fp32 arithmetic."""
import math

import numpy as np
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
    """Every element of got within bound of ref (NaN where ref is NaN). A value beyond the largest of got's type is that
    type's infinity: no finite number of the type is nearer."""
    largest = torch.finfo(got.dtype).max
    got, ref = got.double(), ref.double()
    ref = torch.where(ref.abs() > largest * (1 + U[BF16]), ref.sign() * INF, ref)
    assert got.shape == ref.shape
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan)
    bad = ~(nan | (got == ref) | ((got - ref).abs() <= bound))
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs()[bad].max()))


def padded(x, extra, shift=0):
    """x as a view with a longer row pitch, `shift` elements into its buffer."""
    n, m = x.shape
    buf = torch.full((n * (m + extra) + shift + 64,), 7.0, dtype=x.dtype, device=x.device)
    v = buf[shift:shift + n * (m + extra)].view(n, m + extra)[:, :m]
    v.copy_(x)
    return v


# ------------------------------------------------------------------ router
def chosen_of(x, top_k, live):
    """Experts by the definition, in Python: largest first, ties to the lower index, NaN above all, -infinity never."""
    out = []
    for row, ok in zip(x.double().cpu().tolist(), live.cpu().tolist()):
        order = sorted((i for i, v in enumerate(row) if v != -INF), key=lambda i: (-(INF if row[i] != row[i] else row[i]), row[i] == row[i], i))
        order = sorted(order, key=lambda i: (0 if row[i] != row[i] else 1, -row[i] if row[i] == row[i] else 0, i))
        out.append((order[:top_k] if ok else []) + [-1] * (top_k - (min(len(order), top_k) if ok else 0)))
    return torch.tensor(out, dtype=torch.int32).view(len(out), top_k)


def check_route(x, top_k, live=None, renormalise=True, cb=0.03, cz=0.002, dw=None):
    n, e = x.shape
    r = api.route(x, top_k, live=live, renormalise=renormalise, balance_coef=cb, z_coef=cz)
    ok = torch.ones(n, dtype=torch.bool, device="cuda") if live is None else live.clone()
    ok &= ~(x == -INF).all(-1)
    ids = chosen_of(x, top_k, ok)
    assert torch.equal(r.experts.cpu(), ids)
    ids = ids.cuda().long()
    has = ids >= 0
    counts = torch.bincount(ids[has], minlength=e)
    assert torch.equal(r.counts.long(), counts)
    assert torch.equal(r.offsets.long(), torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), counts.cumsum(0)]))
    flat = ids.reshape(-1)
    slots = torch.nonzero(flat >= 0)[:, 0]
    slots = slots[torch.argsort(flat[slots] * (n * top_k) + slots)]
    assert torch.equal(r.order[:slots.numel()].long(), slots) and torch.all(r.order[slots.numel():] == -1)
    t = int(ok.sum())
    assert int(r.live_rows) == t
    z = x.double().clone()
    z[~ok] = 0
    p = torch.softmax(z, -1)
    logz = torch.where(ok, torch.logsumexp(z, -1), 0.0)
    finite = z.masked_fill(~torch.isfinite(z), 0)
    span = float((finite.amax() - finite.amin())) if n else 0.0
    # exp's argument: |x - max| E; exp, sums of up to 64 terms a lane and tree, division: below 90 roundings
    rel = (span + 90) * E
    w = torch.where(has, p.gather(1, ids.clamp(min=0)), 0.0)
    if renormalise:
        w = torch.where(has, w / w.sum(-1, keepdim=True), 0.0)
    within(r.weights, w, rel * w.abs())
    within(r.logz, logz, rel * 2 + 2 * E * logz.abs())
    # sums of non-negative terms: at most one rounding a row, a stretch and an expert
    if t:
        loss = cb * e / (top_k * t * t) * (counts * p[ok].sum(0)).sum() + cz * (logz[ok] ** 2).sum() / t
        parts = abs(cb) * e / (top_k * t * t) * (counts * p[ok].sum(0)).sum() + abs(cz) * (logz[ok] ** 2).sum() / t
    else:
        loss = parts = torch.zeros((), dtype=F64, device="cuda")
    within(r.loss, loss, float((n + 400) * E * parts + 6 * rel * parts) if not torch.isnan(loss) else 0.0)
    # the gradient against the formula and against autograd
    dw = normal((n, top_k), gen(5), F32) if dw is None else dw
    d = api.route_backward(x, r, dw, renormalise=renormalise, balance_coef=cb, z_coef=cz)
    if not torch.isfinite(z[ok]).all():
        return r, d
    zz = z.clone().requires_grad_(True)
    pp = torch.softmax(zz, -1)
    ww = pp.gather(1, ids.clamp(min=0)) * has
    if renormalise:
        ww = ww / ww.sum(-1, keepdim=True).clamp(min=1e-300)
    s = cb * e / (top_k * max(t, 1) ** 2) * counts.double()
    total = (pp[ok] * s).sum() + cz / max(t, 1) * (torch.logsumexp(zz, -1)[ok] ** 2).sum() + (ww * torch.where(has, dw.double(), 0.0))[ok].sum()
    ref = torch.autograd.grad(total, zz)[0] if t else torch.zeros_like(z)
    ref[~ok] = 0
    dwm = torch.where(has, dw.double().abs(), 0.0)
    full = torch.zeros_like(z).scatter_add_(1, ids.clamp(min=0), dwm)
    mag = p * (s.abs() + (p * (s.abs() + full)).sum(-1, keepdim=True) + 2 * abs(cz) / max(t, 1) * logz.abs()[:, None] + full)
    mag = mag + torch.zeros_like(z).scatter_add_(1, ids.clamp(min=0), w * (dwm + (w * dwm).sum(-1, keepdim=True)))
    within(d, ref, 8 * rel * mag + U[x.dtype] * ref.abs())
    return r, d


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (1, 8, 8), (7, 33, 4), (33, 64, 2), (257, 76, 3), (40, 129, 6), (300, 256, 8),
                                   (65, 500, 32), (19, 1024, 9), (2500, 16, 1)])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route(dtype, n, e, k, renormalise):
    g = gen(n + e)
    x = normal((n, e), g, dtype, 2.0)
    if dtype == BF16:
        x = (x * 4).round() / 4  # many ties
    live = torch.rand(n, device="cuda", generator=g) > 0.2 if n > 5 else None
    if live is not None:
        x[~live] = NAN
    check_route(x, k, live, renormalise)


def test_route_rows_with_little_to_choose_from():
    g = gen(3)
    x = normal((12, 40), g, F32)
    x[0] = -INF                      # counts as padding
    x[1, 1:] = -INF                  # one expert
    x[2, 5:] = -INF                  # fewer than top_k
    x[3] = torch.finfo(F32).min      # the type's lowest value: a distribution, all equal
    x[4] = 0.0
    x[4, ::2] = -0.0                 # equal zeros
    x[5] = 88.0
    x[5, 7] = -88.0
    for dt in (F32, BF16):
        r, d = check_route(x.to(dt), 8)
        assert torch.all(r.experts[0] == -1) and torch.all(r.weights[0] == 0) and torch.all(d[0] == 0)
        assert r.experts[1].tolist() == [0] + [-1] * 7 and r.weights[1, 0] == 1
        # fp32's lowest value is beyond bf16's range: its conversion is -infinity, and the row counts as padding
        assert r.experts[3].tolist() == (list(range(8)) if dt == F32 else [-1] * 8) and r.experts[4].tolist() == list(range(8))
    low = torch.full((3, 12), torch.finfo(BF16).min, dtype=BF16, device="cuda")
    low[1, 5] = 0.0
    r = api.route(low, 3)
    assert r.experts.tolist() == [[0, 1, 2], [5, 0, 1], [0, 1, 2]] and torch.equal(r.weights[1].cpu(), torch.tensor([1.0, 0.0, 0.0]))
    within(r.weights[0], torch.full((3,), 1 / 3, dtype=F64, device="cuda"), 4 * E)
    # nothing lives
    r = api.route(torch.full((5, 9), -INF, device="cuda"), 2)
    assert float(r.loss) == 0 and int(r.live_rows) == 0 and torch.all(r.counts == 0) and torch.all(r.order == -1)
    r = api.route(torch.zeros((0, 9), device="cuda"), 2, balance_coef=1.0)
    assert float(r.loss) == 0 and r.experts.shape == (0, 2) and torch.all(r.offsets == 0)
    assert api.route_backward(torch.zeros((0, 9), device="cuda"), r).shape == (0, 9)


def test_route_nan_and_infinity():
    x = normal((6, 20), gen(4), F32)
    x[1, 7] = NAN
    x[2, 3] = INF
    x[3, 2], x[3, 9] = NAN, INF
    r = api.route(x, 3, balance_coef=0.1, z_coef=0.1)
    assert torch.equal(r.experts.cpu(), chosen_of(x, 3, torch.ones(6, dtype=torch.bool)))
    assert r.experts[1, 0] == 7 and r.experts[3, :2].tolist() == [2, 9] and r.experts[2, 0] == 3
    assert torch.isnan(r.weights[1:4]).all() and torch.isnan(r.logz[[1, 3]]).all() and torch.isnan(r.loss)
    assert torch.isfinite(r.weights[[0, 4, 5]]).all()
    d = api.route_backward(x, r, r.weights.nan_to_num(), balance_coef=0.0)
    assert torch.isnan(d[1]).all() and torch.isfinite(d[[0, 4, 5]]).all()


def test_route_views_in_place_and_many_rows():
    g = gen(6)
    x = normal((1001, 76), g, BF16)
    a = api.route(x, 4, balance_coef=0.1)
    wide = padded(x, 5, 3)
    b = api.route(wide, 4, balance_coef=0.1)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    dw = normal((1001, 4), g)
    d = api.route_backward(x, a, dw, balance_coef=0.1)
    assert api.route_backward(wide, b, dw, balance_coef=0.1, dlogits=wide) is wide and torch.equal(wide, d)
    x = normal((40000, 24), g, F32)  # every stretch and warp of the second launch
    check_route(x, 5, torch.rand(40000, device="cuda", generator=g) > 0.5)


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("n,e,k", [(10001, 136, 4), (5003, 264, 8), (5003, 512, 3), (2503, 1024, 16), (4, 200, 32)])
def test_route_wide_rows_several_a_warp(n, e, k, renormalise):
    # bf16 rows that packs fit, more of them than warps: the next row is read while one is worked on. The fast exponential
    # is off by (2 + 1.2 |l - logz|) 2 E at most, within the 8 (span + 90) E that check_route allows a gradient's terms.
    g = gen(e)
    x = normal((n, e), g, BF16, 2.0)
    x[1] = -INF                       # padding by its logits
    x[2, 1:] = -INF                   # one expert
    x[3, e // 2:] = -INF
    live = torch.rand(n, device="cuda", generator=g) > 0.3
    live[:4] = True
    x[~live] = NAN
    dw = normal((n, k), g, F32)
    kw = dict(renormalise=renormalise, balance_coef=0.03, z_coef=0.002)
    r, d = check_route(x, k, live, renormalise, dw=dw)
    assert torch.isfinite(d).all() and torch.all(d[1] == 0) and torch.all(d[~live] == 0)
    # -infinity is a probability of zero: the row's gradient is the short row's (zero where nothing was held)
    assert torch.all(d[2, 1:] == 0) and torch.all(d[3, e // 2:] == 0)
    ok = live.clone()
    ok[1:4] = False
    z = x.double().masked_fill(~ok[:, None], 0).requires_grad_(True)
    p = torch.softmax(z, -1)
    has = ok[:, None] & (r.experts >= 0)
    ids = r.experts.clamp(min=0).long()
    w = p.gather(1, ids) * has
    if renormalise:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    t = int(r.live_rows)
    s = 0.03 * e / (k * t * t) * r.counts.double()
    total = (p[ok] * s).sum() + 0.002 / t * (torch.logsumexp(z, -1)[ok] ** 2).sum() + (w * dw.double())[ok].sum()
    ref = torch.autograd.grad(total, z)[0]
    dwm = torch.where(has, dw.double().abs(), 0.0)
    p, w = p.detach(), w.detach()
    full = torch.zeros_like(p).scatter_add_(1, ids, dwm)
    lz = torch.logsumexp(z, -1).abs().detach()[:, None]
    mag = p * (s + (p * (s + full)).sum(-1, keepdim=True) + 0.004 / t * lz + full)
    mag = mag + torch.zeros_like(p).scatter_add_(1, ids, w * (dwm + (w * dwm).sum(-1, keepdim=True)))
    span = float(z.detach().amax() - z.detach().amin())
    within(d[ok], ref[ok], (8 * (span + 90) * E * mag + U[BF16] * ref.abs())[ok])
    # a view that packs fit, in place; one that they do not fit
    wide, odd = padded(x, 8, 16), padded(x, 5, 3)
    assert api.route_backward(wide, r, dw, dlogits=wide, **kw) is wide and torch.equal(wide, d)
    within(api.route_backward(odd, r, dw, **kw)[ok], ref[ok], (8 * (span + 90) * E * mag + U[BF16] * ref.abs())[ok])


def test_route_gradient_by_differences():
    # the loss moves by the gradient along a direction that leaves the choice as it is
    g = gen(7)
    x = normal((64, 16), g, F32, 2.0)
    kw = dict(balance_coef=2.0, z_coef=0.5)
    r = api.route(x, 2, **kw)
    d = api.route_backward(x, r, None, **kw)
    v = normal((64, 16), g, F32)
    h = 1e-2
    a, b = api.route(x + h * v, 2, **kw), api.route(x - h * v, 2, **kw)
    same = torch.equal(a.counts, r.counts) and torch.equal(b.counts, r.counts)
    slope = (float(a.loss) - float(b.loss)) / (2 * h)
    if same:  # second order differences: h^2 of a smooth function of size 1, and roundings of the loss over h
        assert abs(slope - float((d * v).sum())) <= 0.05 * h + 64 * E * float(r.loss) / h
    want = torch.autograd.functional.jvp(lambda y: 2.0 * 16 / (2 * 64 * 64) * (r.counts.double() * torch.softmax(y, -1).sum(0)).sum()
                                         + 0.5 / 64 * (torch.logsumexp(y, -1) ** 2).sum(), x.double(), v.double())[1]
    assert abs(float(want) - float((d.double() * v.double()).sum())) <= 200 * E * float((d.abs() * v.abs()).sum())


# ------------------------------------------------------------------ 8-bit blocks
def e4m3(v):
    """float64 to the nearest e4m3 value (at most 448), ties to even."""
    m, ex = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    return np.rint(v / step) * step


def held(x, tiles):
    """The values that the form holds of a float32 matrix, by its definition, in numpy float64."""
    x = x.double().cpu().numpy()
    n, m = x.shape
    out = np.empty_like(x)
    for a in range(0, n, 128 if tiles else 1):
        for b in range(0, m, 128):
            blk = x[a:a + (128 if tiles else 1), b:b + 128]
            if not np.isfinite(blk).all():
                out[a:a + blk.shape[0], b:b + 128] = NAN
                continue
            top = np.abs(blk).max()
            s = 1
            if top > 0:
                s = max(1, int(np.frexp(top)[1]) - 9 + 127)
                while top > np.ldexp(448.0, s - 127):
                    s += 1
            out[a:a + blk.shape[0], b:b + 128] = np.ldexp(e4m3(np.ldexp(blk, 127 - s)), s - 127)
    return torch.from_numpy(out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,m", [(1, 1), (3, 8), (5, 127), (2, 128), (7, 129), (130, 200), (9, 1023), (4, 2304), (129, 264)])
@pytest.mark.parametrize("tiles", [False, True])
def test_blocks_hold_their_definition(dtype, n, m, tiles):
    g = gen(n * m)
    x = normal((n, m), g, F32) * torch.exp(4 * normal((n, 1), g)) * torch.exp(4 * normal((1, m), g))
    x = x.to(dtype)
    b = api.blocks_store(x, tiles=tiles)
    want = held(x.float(), tiles)
    got = api.blocks_load(b, dtype=F32)
    got = got[0] if tiles else got
    assert torch.equal(got.double().cpu(), want)  # exact: e4m3 times a power of two
    assert torch.equal(api.blocks_load(b, dtype=BF16).double().cpu().reshape(n, m), want.bfloat16().double())
    q = b.q.reshape(-1, b.q.shape[-1])
    assert torch.all(q[:, m:] == 0) and torch.all(b.scales[..., -(-m // 128):] == 0)
    wide = padded(x, 3, 1)
    c = api.blocks_store(wide, tiles=tiles)
    assert torch.equal(c.q, b.q) and torch.equal(c.scales, b.scales)
    out = padded(torch.zeros((n, m), dtype=F32, device="cuda"), 5, 2)
    api.blocks_load(b, out=out)
    assert torch.equal(out.double().cpu(), want)


def test_blocks_ends_of_the_range():
    x = torch.zeros((8, 256), device="cuda")
    x[0, :4] = torch.tensor([1e-45, 3e-39, 1.2e-38, 2e-42])     # subnormals
    x[1, :3] = torch.tensor([3.4028235e38, 1.0, -2e38])
    x[2, 5], x[2, 200] = INF, 1.0                                # the second block lives
    x[3, 7] = NAN
    x[4, :3] = torch.tensor([448.0, 447.9, 449.0])
    x[5, :2] = torch.tensor([1.75 * 2 ** -20, 1.75 * 2 ** -20 * (1 + 2 ** -23)])  # either side of a change of scale
    x[6] = torch.finfo(F32).min
    b = api.blocks_store(x)
    assert torch.equal(b.scales[2:4, :2].cpu(), torch.tensor([[255, int(b.scales[2, 1])], [255, 1]], dtype=torch.uint8))
    # 256 units of 2^120, what the largest numbers round to, are beyond fp32: infinity
    got, want = api.blocks_load(b, dtype=F32).double().cpu(), held(x, False).float().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m", [64, 1000, 1023])
def test_blocks_gather(dtype, m):
    g = gen(m)
    x = normal((50, m), g, dtype)
    rows = torch.randint(-3, 160, (333,), device="cuda", generator=g).int()  # some negative, some beyond the last row
    b = api.blocks_store(x, rows=rows, per=3)
    src = torch.where(rows < 0, -1, rows // 3)
    src = torch.where(src >= 50, -1, src)
    all_, want = api.blocks_store(x), api.blocks_load(b, dtype=F32)
    ref = api.blocks_load(all_, dtype=F32)[src.clamp(min=0).long()] * (src >= 0)[:, None]
    assert torch.equal(want, ref)
    empty = api.blocks_store(x, rows=rows[:0], per=3)
    assert empty.rows == 0 and api.blocks_load(empty).shape == (0, m)


def products(a, w, back, ends, rows, n):
    ref, mag = (torch.zeros((rows, n), dtype=F64, device="cuda") for _ in range(2))
    for i in range(len(ends) - 1):
        lo, hi = ends[i], ends[i + 1]
        m = w[i] if back else w[i].t()
        ref[lo:hi], mag[lo:hi] = a[lo:hi] @ m, a[lo:hi].abs() @ m.abs()
    return ref, mag


def check_product(rows, k, n, back, out, groups=1, ends=None, seed=0, use_out=False):
    """k: depth, n: columns of the result."""
    g = gen(seed + rows + n)
    x = normal((rows, k), g) * torch.exp(3 * normal((rows, 1), g)) * torch.exp(2 * normal((1, k), g))
    shape = (groups, k, n) if back else (groups, n, k)
    w = normal(shape, g) * torch.exp(2 * normal((groups, shape[1], 1), g)) * torch.exp(2 * normal((groups, 1, shape[2]), g))
    a, b = api.blocks_store(x), api.blocks_store(w, tiles=True)
    off = None
    if ends is not None:
        off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    dst = None
    if use_out:
        dst = padded(torch.zeros((rows, n), dtype=out, device="cuda"), 3, 1)
    got = api.blocks_matmul(a, b, transpose=back, offsets=off, dtype=out, out=dst)
    ref, mag = products(api.blocks_load(a, dtype=F32).double(), api.blocks_load(b, dtype=F32).double(), back, ends or [0, rows], rows, n)
    # products are exact; the tensor cores lose up to a unit in the last place (2 E) of the running sum per instruction, 32
    # instructions between two drains, and 2 more for the sum within an instruction; the drains' sums E each
    within(got, ref, ((32 + 2) * 2 * E + (k / 1024 + 5) * E) * mag + U[out] * ref.abs())
    assert api.get_status() == 0


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("rows,k,n", [(1, 1, 1), (1, 128, 256), (3, 64, 300), (16, 1024, 8), (17, 129, 257), (40, 2304, 520),
                                      (65, 1000, 1000), (129, 4500, 130), (200, 640, 2303), (700, 1100, 515), (2000, 256, 600)])
def test_product(back, rows, k, n):
    check_product(rows, k, n, back, F32)
    check_product(rows, k, n, back, BF16, use_out=rows % 2 == 1)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("rows,k,n,ends", [(300, 256, 200, [0, 0, 100, 100, 300]), (300, 500, 300, [7, 20, 290]), (64, 130, 64, [64, 64, 64]),
                                           (1000, 384, 260, [0, 1, 2, 500, 999]), (5, 128, 128, [0, 5, 5, 5, 5, 5]),
                                           (900, 128, 128, list(range(0, 901, 10)))])
def test_product_of_a_stack(back, rows, k, n, ends):
    check_product(rows, k, n, back, F32, len(ends) - 1, ends)
    check_product(rows, k, n, back, BF16, len(ends) - 1, ends, use_out=True)


def test_product_split_depth():
    # few columns and rows, a long depth: the depth is split over a cluster
    for rows in (1, 9, 33, 64):
        for back in (False, True):
            check_product(rows, 8300, 300, back, F32)
            check_product(rows, 4096, 256, back, BF16)
    check_product(10, 6144, 256, False, F32, 2, [1, 4, 9])


def test_product_rows_of_no_group_are_zeros_whatever_was_there():
    a, b = api.blocks_store(normal((100, 128), gen(1))), api.blocks_store(normal((2, 64, 128), gen(2)), tiles=True)
    out = torch.full((100, 64), NAN, device="cuda")
    api.blocks_matmul(a, b, offsets=torch.tensor([10, 20, 60], dtype=torch.int32, device="cuda"), out=out)
    assert torch.all(out[:10] == 0) and torch.all(out[60:] == 0) and torch.isfinite(out).all() and (out[10:60] != 0).any()
    none = api.Blocks8(b.q[:0].contiguous(), b.scales[:0].contiguous(), 128, tiles=True)
    out.fill_(NAN)
    api.blocks_matmul(a, none, offsets=torch.tensor([5], dtype=torch.int32, device="cuda"), out=out)
    assert torch.all(out == 0)


def test_product_nan_stays_in_its_row_or_columns():
    g = gen(8)
    x, w = normal((70, 300), g), normal((300, 300), g)
    x[3, 200] = INF
    w[140, 10] = NAN                       # the block of rows 128..255, depth 0..127
    got = api.blocks_matmul(api.blocks_store(x), api.blocks_store(w, tiles=True), dtype=F32)
    bad = torch.isnan(got)
    want = torch.zeros_like(bad)
    want[3], want[:, 128:256] = True, True
    assert torch.equal(bad, want)
    # and rows of one group never reach another's
    x[3, 200] = 0.0
    x[30:40] = NAN
    w = normal((3, 64, 300), g)
    off = torch.tensor([0, 30, 40, 70], dtype=torch.int32, device="cuda")
    got = api.blocks_matmul(api.blocks_store(x), api.blocks_store(w, tiles=True), offsets=off, dtype=F32)
    assert torch.isfinite(got[:30]).all() and torch.isnan(got[30:40]).all() and torch.isfinite(got[40:]).all()


def test_product_near_the_ends_of_fp32():
    # scales that multiply to far beyond fp32 on the way, results within it
    x, w = torch.full((4, 128), 2.0 ** 120, device="cuda"), torch.full((128, 128), 2.0 ** -124, device="cuda")
    got = api.blocks_matmul(api.blocks_store(x), api.blocks_store(w, tiles=True), dtype=F32)
    assert torch.all(got == 8.0)
    got = api.blocks_matmul(api.blocks_store(x), api.blocks_store(x[:1].expand(128, 128).contiguous(), tiles=True), dtype=F32)
    assert torch.isinf(got).all()
    assert torch.all(api.blocks_matmul(api.blocks_store(x * 0), api.blocks_store(w, tiles=True)) == 0)


# ------------------------------------------------------------------ block norms
def norm_reference(x, y, gate, post, pre, a, b, eps, dres=None, dz=None):
    """(r, z, gradients) in 64 bits by autograd, and the sizes of what their roundings are relative to."""
    names = dict(x=x, y=y, gate=gate, post=post, pre=pre)
    v = {k: t.double().requires_grad_(True) for k, t in names.items() if t is not None}
    r = a * v["x"]
    if y is not None:
        u = v["y"]
        if post is not None:
            u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * v["post"]
        r = r + b * (v["gate"] * u if gate is not None else u)
    z = None if pre is None else r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * v["pre"]
    outs, douts = [], []
    if dres is not None:
        outs.append(r)
        douts.append(dres.double())
    if z is not None and dz is not None:
        outs.append(z)
        douts.append(dz.double())
    grads = dict(zip(v, torch.autograd.grad(outs, list(v.values()), douts))) if outs else {}
    with torch.no_grad():
        X, Y = x.double(), None if y is None else y.double()
        ry = 1.0 if post is None else 1 / torch.sqrt((Y * Y).mean(-1, keepdim=True) + eps)
        g = 1.0 if gate is None else gate.double()
        w1, w2 = 1.0 if post is None else post.double(), 1.0 if pre is None else pre.double()
        yh = 0.0 if y is None else Y * ry
        rm = a * X.abs() + (abs(b) * (g * w1 * yh).abs() if y is not None else 0.0) if a >= 0 else abs(a) * X.abs() + abs(b) * abs(g * w1 * yh)
        size = dict(r=rm)
        rr = 0.0 if pre is None else 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
        if pre is not None:
            size["z"] = rm * rr * w2.abs()
        if outs:
            d = torch.zeros_like(X) if dres is None else dres.double().abs()
            if pre is not None:
                gz = (dz.double() * w2).abs()
                d = d + rr * (gz + rm * rr * (gz * rm * rr).mean(-1, keepdim=True))
                size["pre"] = (dz.double().abs() * rm * rr).sum(0)
            size["x"] = abs(a) * d
            if y is not None:
                gm = g.abs() if gate is not None else 1.0
                k = abs(b) * gm * (w1.abs() if post is not None else 1.0) * d
                size["y"] = ry * (k + (yh.abs() * (k * yh.abs()).mean(-1, keepdim=True) if post is not None else 0.0))
                if post is not None:
                    size["post"] = (abs(b) * gm * d * yh.abs()).sum(0)
                if gate is not None:
                    dg = abs(b) * d * (w1.abs() if post is not None else 1.0) * yh.abs()
                    size["gate"] = dg.sum(0) if gate.dim() == 1 else dg.sum(-1, keepdim=True) if gate.shape != x.shape else dg
    return r.detach(), None if z is None else z.detach(), grads, size


# statistics: sums of squares of up to 32 terms a thread and a tree, rsqrt, three products: below 64 roundings; what
# follows takes them in twice
K = 160


def check_norm(rows, cols, xt=BF16, yt=BF16, wt=BF16, gate="cols", post=True, pre=True, with_y=True, dres=True, a=0.9, b=0.7, seed=0,
               view=False):
    g = gen(seed + rows * cols)
    make = lambda *s, dt, std=1.0: normal(s, g, dt, std)  # noqa: E731
    x = make(rows, cols, dt=xt) * torch.exp(normal((rows, 1), g)).to(xt)
    y = make(rows, cols, dt=yt, std=2.0) if with_y else None
    shape = dict(none=None, cols=(cols,), rows=(rows, 1), full=(rows, cols))[gate if with_y else "none"]
    gt = None if shape is None else make(*shape, dt=wt if gate == "cols" else yt)
    w1 = make(cols, dt=wt) if post and with_y else None
    w2 = make(cols, dt=wt) if pre else None
    dr = make(rows, cols, dt=xt) if dres else None
    dz = make(rows, cols, dt=yt if with_y else xt) if pre else None
    if view:
        x, dr = padded(x, 3, 1), None if dr is None else padded(dr, 5, 2)
        y, dz = None if y is None else padded(y, 1, 3), None if dz is None else padded(dz, 8)
    kw = dict(gate=gt, post_weight=w1, pre_weight=w2, residual_scale=a, block_scale=b)
    f = api.block_norm(x, y, eps=1e-5, **kw)
    af, bf, eps = (float(torch.tensor(v, dtype=F32)) for v in (a, b, 1e-5))
    r, z, grads, size = norm_reference(x, y, gt, w1, w2, af, bf, eps, dr, dz)
    within(f.residual, r, K * E * size["r"] + U[xt] * r.abs())
    if pre:
        within(f.normed, z, K * E * size["z"] + U[f.normed.dtype] * z.abs())
    else:
        assert f.normed is None
    got = api.block_norm_backward(dr, dz, x, y, f, **kw)
    out = dict(x=got.dx, y=got.dy, gate=got.dgate, post=got.dpost_weight, pre=got.dpre_weight)
    for name, t in out.items():
        if name not in grads:
            assert t is None, name
            continue
        n = rows + 2 * K if name in ("post", "pre") or name == "gate" and gate == "cols" else 4 * K
        if name == "gate" and gate == "rows":
            n = cols + 4 * K
        assert t.shape == grads[name].shape
        within(t, grads[name], 2 * n * E * size[name] + U[t.dtype] * grads[name].abs())
    assert api.get_status() == 0


@pytest.mark.parametrize("xt,yt,wt", [(BF16, BF16, BF16), (F32, F32, F32), (F32, BF16, BF16), (BF16, BF16, F32)])
@pytest.mark.parametrize("rows,cols,gate", [(1, 1, "none"), (3, 8, "cols"), (5, 40, "rows"), (70, 127, "full"), (9, 256, "cols"),
                                            (300, 264, "rows"), (33, 2048, "none"), (7, 2303, "rows"), (20, 4104, "cols"),
                                            (400, 1000, "cols"), (5, 8192, "full"), (3, 8200, "cols"), (4, 10175, "rows"),
                                            (2, 16384, "cols"), (2, 16383, "full")])
def test_block_norm(xt, yt, wt, rows, cols, gate):
    check_norm(rows, cols, xt, yt, wt, gate)


@pytest.mark.parametrize("gate", ["none", "cols", "rows", "full"])
@pytest.mark.parametrize("post,pre,dres", [(True, False, True), (False, True, True), (False, False, True), (True, True, False)])
def test_block_norm_parts(gate, post, pre, dres):
    check_norm(37, 320, gate=gate, post=post, pre=pre, dres=dres)
    check_norm(37, 321, F32, BF16, F32, gate, post=post, pre=pre, dres=dres, a=-1.5)


@pytest.mark.parametrize("cols", [64, 513, 6144])
def test_block_norm_without_a_block(cols):
    check_norm(50, cols, with_y=False, gate="none")
    check_norm(50, cols, F32, F32, BF16, with_y=False, gate="none", dres=False)


@pytest.mark.parametrize("cols", [96, 2304, 8192])
def test_block_norm_views_and_many_rows(cols):
    check_norm(31, cols, view=True)
    check_norm(31, cols, F32, F32, F32, "full", view=True)
    check_norm(3001, cols, F32, BF16, F32, "rows")


def test_block_norm_in_place():
    g = gen(9)
    x, y, w = normal((40, 520), g, BF16), normal((40, 520), g, BF16), normal((520,), g, BF16)
    dr, dz = normal((40, 520), g, BF16), normal((40, 520), g, BF16)
    kw = dict(post_weight=w, pre_weight=w)
    f = api.block_norm(x, y, **kw)
    b = api.block_norm_backward(dr, dz, x, y, f, **kw)
    xx, yy = x.clone(), y.clone()
    h = api.block_norm(xx, yy, residual=xx, normed=yy, **kw)
    assert h.residual is xx and torch.equal(xx, f.residual) and torch.equal(yy, f.normed) and torch.equal(h.rstd, f.rstd)
    d, e = dr.clone(), dz.clone()
    c = api.block_norm_backward(d, e, x, y, f, dx=d, dy=e, **kw)
    assert torch.equal(d, b.dx) and torch.equal(e, b.dy) and torch.equal(c.dpre_weight, b.dpre_weight)


def test_block_norm_special_values():
    g = gen(10)
    x, y, w = normal((6, 256), g), normal((6, 256), g), normal((256,), g)
    x[1], y[1] = 0.0, 0.0                                # eps keeps zero rows finite
    x[2, 3], y[3, 4] = NAN, INF
    y[4] = 1e18                                          # squares within fp32, sums too
    f = api.block_norm(x, y, post_weight=w, pre_weight=w)
    assert torch.all(f.residual[1] == 0) and torch.all(f.normed[1] == 0)
    assert torch.isnan(f.normed[2]).all() and torch.isfinite(f.residual[[0, 1, 4, 5]]).all() and torch.isfinite(f.normed[[0, 1, 4, 5]]).all()
    z = api.block_norm(x[:0], y[:0], post_weight=w, pre_weight=w)
    assert z.residual.shape == (0, 256)
    b = api.block_norm_backward(x[:0], y[:0], x[:0], y[:0], z, post_weight=w, pre_weight=w)
    assert torch.all(b.dpost_weight == 0) and torch.all(b.dpre_weight == 0)


def test_block_norm_gradient_by_differences():
    g = gen(11)
    x, y = normal((4, 96), g), normal((4, 96), g)
    w1, w2, gate = normal((96,), g), normal((96,), g), normal((4, 1), g)
    cr, cz = normal((4, 96), g), normal((4, 96), g)

    def value(x, y, w1, w2, gate):
        f = api.block_norm(x, y, gate=gate, post_weight=w1, pre_weight=w2, residual_scale=0.8, block_scale=1.3)
        return float((f.residual.double() * cr.double()).sum() + (f.normed.double() * cz.double()).sum())
    f = api.block_norm(x, y, gate=gate, post_weight=w1, pre_weight=w2, residual_scale=0.8, block_scale=1.3)
    b = api.block_norm_backward(cr, cz, x, y, f, gate=gate, post_weight=w1, pre_weight=w2, residual_scale=0.8, block_scale=1.3)
    args = [x, y, w1, w2, gate]
    for i, d in enumerate((b.dx, b.dy, b.dpost_weight, b.dpre_weight, b.dgate)):
        v = normal(args[i].shape, g)
        h = 2.0 ** -8
        up, down = ([t + s * h * v if k == i else t for k, t in enumerate(args)] for s in (1, -1))
        slope = (value(*up) - value(*down)) / (2 * h)
        # roundings of 800 terms of size about 1 over h, and h^2 of the third derivative (of the size of the gradient's terms)
        size = float((d.abs() * v.abs()).sum())
        assert abs(slope - float((d.double() * v.double()).sum())) <= 800 * 4 * K * E / h + 4 * h * h * (size + 100)


# ------------------------------------------------------------------ dropout
M32 = np.uint64(0xFFFFFFFF)


def philox(n, seed, third):
    """Philox4x32-10 of 64-bit counters (numpy uint64), by its definition."""
    a, b, c, d = n & M32, n >> np.uint64(32), np.full_like(n, third), np.zeros_like(n)
    k0, k1 = np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32)
    for _ in range(10):
        p, q = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, d = (q >> np.uint64(32)) ^ b ^ k0, q & M32, (p >> np.uint64(32)) ^ d ^ k1, p & M32
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & M32, (k1 + np.uint64(0xBB67AE85)) & M32
    return np.stack([a, b, c, d], -1)


def kept(rows, cols, p, seed, offset):
    packs = -(-cols // 8)
    n = (np.uint64(offset) + np.arange(rows * packs, dtype=np.uint64)) if rows * packs else np.zeros(0, np.uint64)
    h, l = philox(n, seed, 0), philox(n, seed, 1)
    v = np.empty((rows * packs, 8), np.uint64)
    for j in range(8):
        s = np.uint64(16 * (j % 2))
        v[:, j] = (((h[:, j // 2] >> s) & np.uint64(0xFFFF)) << np.uint64(16)) | ((l[:, j // 2] >> s) & np.uint64(0xFFFF))
    limit = int(np.rint(p * 2.0 ** 32))
    return torch.from_numpy((v >= np.uint64(limit)).reshape(rows, packs * 8)[:, :cols]).cuda(), limit


def test_philox_known_answers():
    # the published test vectors of the generator (counter and key of zeros, and of ones), against the reference above
    z = philox(np.zeros(1, np.uint64), 0, 0)[0]
    assert [int(v) for v in z] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (2, 1000), (70, 33), (257, 264), (9, 2303)])
@pytest.mark.parametrize("p", [0.0, 1e-6, 0.1, 0.5, 0.999999, 1.0])
def test_dropout(dtype, rows, cols, p):
    g = gen(rows + cols)
    x, res = normal((rows, cols), g, dtype), normal((rows, cols), g, dtype)
    seed, offset = 0x123456789ABCDEF0, (1 << 32) - 3
    keep, limit = kept(rows, cols, p, seed, offset)
    scale = 0.0 if limit == 1 << 32 else 2.0 ** 32 / (2 ** 32 - limit)
    sf = float(torch.tensor(scale, dtype=F32))
    got = api.dropout(x, p, seed, offset)
    assert torch.equal(got, torch.where(keep, (x.float() * sf), torch.zeros((), device="cuda")).to(dtype))
    got = api.dropout(x, p, seed, offset, residual=res)
    ref = res.double() + keep * (x.double() * sf)
    # one fused multiply-add, rounded to fp32 and to the type
    within(got, ref, E * ref.abs() + U[dtype] * (1 + E) * ref.abs())
    if dtype == BF16:
        wide = res.float()
        got = api.dropout(x, p, seed, offset, residual=wide)
        assert got.dtype == F32
        within(got, ref, E * ref.abs())


def test_dropout_forms_agree():
    g = gen(12)
    for cols in (520, 521):
        x, res = normal((40, cols), g, BF16), normal((40, cols), g, BF16)
        a, s = api.dropout(x, 0.3, 5, 9, residual=res), api.dropout(x, 0.3, 5, 9)
        assert torch.equal(api.dropout(padded(x, 3, 1), 0.3, 5, 9, residual=padded(res, 5, 2)), a)
        assert torch.equal(api.dropout(padded(x, 8), 0.3, 5, 9, out=padded(x, 1, 1)), s)
        y = x.clone()
        assert api.dropout(y, 0.3, 5, 9, out=y) is y and torch.equal(y, s)
        y = res.clone()
        assert api.dropout(x, 0.3, 5, 9, residual=y, out=y) is y and torch.equal(y, a)
        state = torch.tensor([2, 4], dtype=torch.int64, device="cuda")
        assert torch.equal(api.dropout(x, 0.3, 3, 5, state=state), s)
        state = torch.tensor([-1, -2], dtype=torch.int64, device="cuda")  # modulo 2^64
        assert torch.equal(api.dropout(x, 0.3, 6, 11, state=state), s)
        # rows in two calls, the second from the counter that the first leaves
        top = api.dropout(x[:11], 0.3, 5, 9)
        rest = api.dropout(x[11:], 0.3, 5, 9 + api.dropout_counters(11, cols))
        assert torch.equal(torch.cat([top, rest]), s)
    x = torch.full((4, 16), NAN, device="cuda")
    d = api.dropout(x, 0.5, 1)
    keep, _ = kept(4, 16, 0.5, 1, 0)
    assert torch.equal(torch.isnan(d), keep) and torch.all(d[~keep] == 0)
    assert api.dropout(x[:0], 0.5, 1).shape == (0, 16)


def test_dropout_share():
    n = 1 << 22
    x = torch.ones((n // 1024, 1024), device="cuda")
    for p in (0.1, 0.37):
        got = api.dropout(x, p, 77)
        share = float((got == 0).double().mean())
        assert abs(share - p) <= 6 * math.sqrt(p * (1 - p) / n)  # six standard deviations


# ------------------------------------------------------------------ sizes, streams, graphs
def test_more_than_2_to_the_31_elements():
    rows, cols = (1 << 20) + 3, 2056
    x = torch.empty((rows, cols), dtype=BF16, device="cuda")
    x[-2:] = normal((2, cols), gen(13), BF16)
    x[: rows - 2].fill_(1.0)
    packs = api.dropout_counters(1, cols)
    assert torch.equal(api.dropout(x, 0.2, 3)[-2:], api.dropout(x[-2:], 0.2, 3, (rows - 2) * packs))
    w = normal((cols,), gen(14), BF16)
    f = api.block_norm(x, x, post_weight=w, pre_weight=w)
    s = api.block_norm(x[-2:], x[-2:], post_weight=w, pre_weight=w)
    assert torch.equal(f.normed[-2:], s.normed) and torch.equal(f.residual[-2:], s.residual)
    b = api.block_norm_backward(x, x, x, x, f, post_weight=w, pre_weight=w)
    c = api.block_norm_backward(x[-2:], x[-2:], x[-2:], x[-2:], s, post_weight=w, pre_weight=w)
    assert torch.equal(b.dx[-2:], c.dx) and torch.equal(b.dy[-2:], c.dy)
    del f, b
    h = api.blocks_store(x)
    t = api.blocks_store(x[-2:])
    assert torch.equal(h.q[-2:], t.q) and torch.equal(api.blocks_load(h)[-2:], api.blocks_load(t))
    last = torch.tensor([rows - 1, -1, rows - 2], dtype=torch.int32, device="cuda")
    assert torch.equal(api.blocks_store(x, rows=last).q[[0, 2]], t.q.flip(0))
    v = api.blocks_store(normal((2304, cols), gen(15), BF16), tiles=True)
    assert torch.equal(api.blocks_matmul(h, v)[-2:], api.blocks_matmul(t, v))
    assert api.get_status() == 0


def everything(seed):
    """A call of every operator on inputs of its own; returns a function that makes them all and lists what they give."""
    g = gen(seed)
    logits, x, y = normal((300, 40), g, BF16), normal((300, 520), g, BF16), normal((300, 520), g, BF16)
    w, gate = normal((520,), g, BF16), normal((520,), g, BF16)
    experts = api.blocks_store(normal((40, 256, 520), g, BF16, 0.05), tiles=True)
    torch.cuda.synchronize()

    def go():
        r = api.route(logits, 3, balance_coef=0.1, z_coef=0.01)
        d = api.route_backward(logits, r, r.weights, balance_coef=0.1, z_coef=0.01)
        f = api.block_norm(x, y, gate=gate, post_weight=w, pre_weight=w)
        a = api.blocks_store(f.normed, rows=r.order, per=3)
        h = api.blocks_matmul(a, experts, offsets=r.offsets)
        back = api.blocks_matmul(api.blocks_store(h), experts, transpose=True, offsets=r.offsets)
        b = api.block_norm_backward(x, y, x, y, f, gate=gate, post_weight=w, pre_weight=w)
        o = api.dropout(x, 0.2, 5, residual=y)
        return [*r, d, f.residual, f.normed, f.rstd, h, back, *b, o, api.blocks_load(a)]
    return go


def test_same_bits_each_time_and_on_other_streams():
    go = everything(20)
    ref = go()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = go()
    again = go()
    torch.cuda.synchronize()
    for a, b, c in zip(ref, out, again):
        assert torch.equal(a, b) and torch.equal(a, c)
    s = torch.cuda.Stream()
    x = normal((64, 128), gen(21), BF16)
    torch.cuda.synchronize()
    assert torch.equal(api.dropout(x, 0.5, 1, stream=s), (s.synchronize(), api.dropout(x, 0.5, 1))[1])


def test_two_captured_graphs_replayed_side_by_side():
    # their scratch is their own: graphs of the same calls may run at once
    makers = [everything(30), everything(31)]
    refs = [m() for m in makers]
    torch.cuda.synchronize()
    stream, graphs, outs = torch.cuda.Stream(), [], []
    for m in makers:
        with torch.cuda.stream(stream):
            m()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(m())
        graphs.append(graph)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for graph, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for ref, out in zip(refs, outs):
        assert all(torch.equal(a, b) for a, b in zip(ref, out))
    assert api.get_status() == 0


def test_a_captured_dropout_draws_anew():
    x = torch.ones((64, 256), device="cuda")
    state = torch.zeros(2, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        api.dropout(x, 0.5, 3, state=state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = api.dropout(x, 0.5, 3, state=state)
        state[1] += api.dropout_counters(64, 256)
    torch.cuda.synchronize()
    state.zero_()
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, api.dropout(x, 0.5, 3, k * api.dropout_counters(64, 256)))


def test_launches_are_counted_and_timed():
    go = everything(40)
    go()
    before = api.num_kernel_launches()
    api.set_kernel_timing(True)
    go()
    t = api.kernel_times()
    api.set_kernel_timing(False)
    for kind in ("route", "blocks", "blocks_matmul", "block_norm", "dropout"):
        assert t[kind][1] > 0 and t[kind][0] > 0, kind
    assert api.num_kernel_launches() - before >= sum(n for _, n in t.values()) >= 5
