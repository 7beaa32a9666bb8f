"""GPU tests of the expert-layer operators where a bound taken over a whole call says nothing: rows of logits far from
zero, each with its own bound; sums that a coefficient of zero leaves out; forms that other tests leave out.

U is the unit roundoff of a type, E = 2^-24 that of fp32 arithmetic."""
import math

import pytest
import torch

from newton_schulz_quintic_gb300 import api
from test_layers_gpu import check_norm

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
E = 2.0 ** -24
TINY = 2.0 ** -126  # what fp32 may lose below its normal numbers
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
    """Every element of got within bound of ref; a reference beyond the type's numbers is its infinity."""
    largest = torch.finfo(got.dtype).max
    got, ref = got.double(), ref.double()
    ref = torch.where(ref.abs() > largest * (1 + U[BF16]), ref.sign() * INF, ref)
    assert got.shape == ref.shape
    bad = ~((got == ref) | ((got - ref).abs() <= bound))
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist())


# ------------------------------------------------------------------ router
def check_rows(x, top_k, renormalise, cb, cz, seed=0):
    """A routing and its gradient against the formulas in 64 bits, every row by its own bound. x holds no NaN and no
    +infinity.

    A logit's distance to its row's largest, D, is rounded once (D E relative in the exponential); a kernel that takes
    another number of the row's size in its place is at most 16 from it. exp: 2 units in the last place, or
    (2 + 1.2 D) 2^-23 for the fast one of bf16. Sums of 1024 terms by 32 lanes: 37 roundings. So a probability is off by
    rel = (4 D + 4 sum p D + 120) E of itself, and what underflows by TINY."""
    n, e = x.shape
    kw = dict(renormalise=renormalise, balance_coef=cb, z_coef=cz)
    r = api.route(x, top_k, **kw)
    z = x.double()
    live = (z > -INF).any(-1)
    z = torch.where(live[:, None], z, 0.0)
    top = z.amax(-1, keepdim=True)
    far = (top - z).clamp(max=1e6) + 16  # beyond 1e6 (beyond 110) the exponential is 0 in any precision
    q = torch.exp(z - top)
    total = q.sum(-1, keepdim=True)
    p = torch.where(live[:, None], q / total, 0.0)
    logz = torch.where(live, (top + total.log())[:, 0], 0.0)
    spread = (p * far).sum(-1, keepdim=True)
    rel = (4 * far + 4 * spread + 120) * E
    ids = r.experts.long()
    has = ids >= 0
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :top_k]
    want = torch.where(live[:, None] & (z.gather(1, order) > -INF), order, -1)
    assert torch.equal(ids, want)
    at = ids.clamp(min=0)
    w, wrel = torch.where(has, p.gather(1, at), 0.0), rel.gather(1, at)
    if renormalise:
        w = torch.where(has, w / w.sum(-1, keepdim=True).clamp(min=1e-300), 0.0)
        wrel = wrel + (w * wrel).sum(-1, keepdim=True)
    within(r.weights, w, wrel * w + TINY)
    lz_err = (4 * spread[:, 0] + 120) * E + E * logz.abs()  # of a total and its logarithm, the sum rounded
    within(r.logz, logz, lz_err)
    t = max(int(live.sum()), 1)
    counts = torch.bincount(ids[has], minlength=e).double()
    assert torch.equal(r.counts.double(), counts)
    share = cb * e / (top_k * t * t)
    balance, zterm = share * (counts * p.sum(0)).sum(), cz / t * (logz ** 2).sum()
    # sums of n terms of one sign in fp32 (at most one rounding a row, a stretch and an expert), and what they take over
    err = (n + 400) * E * (abs(balance) + abs(zterm)) + abs(share) * (counts * (p * rel).sum(0)).sum()
    err = err + abs(cz) / t * (2 * logz.abs() * lz_err).sum()
    within(r.loss, balance + zterm, err)
    dw = normal((n, top_k), gen(seed + 1))
    d = api.route_backward(x, r, dw, **kw)
    dwd = torch.where(has, dw.double(), 0.0)
    s = (share * counts)[None].expand(n, e)
    zero = torch.zeros_like(z)
    if renormalise:
        own = w * (dwd - (w * dwd).sum(-1, keepdim=True))
        own_err = w * (dwd.abs() + (w * dwd.abs()).sum(-1, keepdim=True)) * (2 * wrel + 40 * E)
        own, own_err = zero.scatter_add(1, at, own), zero.scatter_add(1, at, own_err)
    else:
        s = s.scatter_add(1, at, dwd)
        own = own_err = zero
    zl = 2 * cz / t * logz[:, None]
    want = p * (s - (p * s).sum(-1, keepdim=True) + zl) + own
    want = torch.where(live[:, None], want, 0.0)
    inner = (p * s.abs() * (rel + 40 * E)).sum(-1, keepdim=True)
    err = p * ((s.abs() + (p * s.abs()).sum(-1, keepdim=True) + zl.abs()) * (rel + 40 * E) + inner + abs(2 * cz / t) * lz_err[:, None])
    within(d, want, err + own_err + U[x.dtype] * want.abs() + TINY)
    return r, d


OFFSETS = [0.0, -40.0, 1e3, -1e4, 1e5, -1e6, 1e7, -1e9, 1e12, -1e20, 1e30, -3e38]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("e,k", [(5, 2), (40, 8), (76, 3), (256, 8), (264, 4), (512, 3), (1000, 16), (1024, 32)])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_of_logits_far_from_zero(dtype, e, k, renormalise):
    # probabilities are those of the distances within a row, wherever the row lies
    g = gen(e)
    rows = torch.tensor(OFFSETS, device="cuda").repeat(5)
    x = (normal((rows.numel(), e), g, F32, 3.0) + rows[:, None]).clamp(min=torch.finfo(dtype).min).to(dtype)
    check_rows(x, k, renormalise, 0.03, 0.0, e)   # (a z term of such rows hides the balance)
    check_rows(x[(rows.abs() < 2e7)], k, renormalise, 0.03, 0.002, e)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_route_of_the_lowest_logits(dtype):
    # a row masked by the type's lowest number is a distribution, all equal: its probabilities sum to 1, forward and back
    low = torch.finfo(dtype).min
    for e in (24, 256, 1000):
        x = torch.full((6, e), low, dtype=dtype, device="cuda")
        x[1, 3:] = 2.0
        x[2, :e // 2] = -INF
        x[3] = normal((e,), gen(2), dtype)
        r, d = check_rows(x, 4, True, 0.05, 0.0)
        assert float(r.loss) > 0
        r, d = check_rows(x, 4, False, 0.05, 0.0)
        # without the weights' part only the balance is left, and its gradient is small beside it: s - sum p s
        d = api.route_backward(x, r, None, renormalise=False, balance_coef=0.05)
        assert float(d.double().sum(-1).abs().max()) <= 2 * e * U[dtype] * float(d.double().abs().max()) + e * TINY


def test_route_z_term_stays_out_of_the_loss_at_coefficient_zero():
    # squares of these rows' logz are beyond fp32: a coefficient of zero takes no part of them
    for dtype in (BF16, F32):
        x = normal((7, 40), gen(3), dtype)
        want = api.route(x[:5], 3, balance_coef=0.0)
        assert float(want.loss) == 0
        x[5], x[6] = torch.finfo(dtype).min, 1e25
        r = api.route(x, 3)
        assert float(r.loss) == 0
        r, _ = check_rows(x, 3, True, 0.1, 0.0)
        assert math.isfinite(float(r.loss)) and float(r.loss) > 0
        # with a coefficient they count: infinite in fp32
        assert float(api.route(x, 3, z_coef=1e-3).loss) == INF
        # a NaN reaches the loss at any coefficient
        x[0, 0] = NAN
        assert math.isnan(float(api.route(x, 3).loss))


@pytest.mark.parametrize("e,k", [(16, 2), (256, 8)])
def test_route_loss_moves_by_its_gradient(e, k):
    # logits at least 1/2 apart and steps of at most 1/16: the choice stays as it is
    g = gen(e)
    n, cb, cz = 64, 2.0, 0.5
    place = torch.argsort(torch.rand((n, e), device="cuda", generator=g), dim=-1)
    x = place.float() * 0.5 - e / 8
    v = normal((n, e), g).clamp(-4, 4)
    h = 2.0 ** -6
    kw = dict(balance_coef=cb, z_coef=cz)
    r = api.route(x, k, **kw)
    a, b = api.route(x + h * v, k, **kw), api.route(x - h * v, k, **kw)
    assert torch.equal(a.experts, r.experts) and torch.equal(b.experts, r.experts)
    d = api.route_backward(x, r, None, **kw)
    slope = float((d.double() * v.double()).sum())

    def value(step):
        y = x.double() + step * v.double()
        p = torch.softmax(y, -1)
        return float(cb * e / (k * n * n) * (r.counts.double() * p.sum(0)).sum() + cz / n * (torch.logsumexp(y, -1) ** 2).sum())

    def quotient(step):
        return (value(step) - value(-step)) / (2 * step)
    rest = 2 * abs(quotient(h) - quotient(h / 2))  # the third derivative's share is 4/3 of that
    # x + h v is rounded (E of up to e / 4 a logit, which the gradient multiplies); the losses' own roundings, see check_rows
    inputs = float(d.double().abs().sum()) * (e / 4 + 1) * E * 2 / (2 * h)
    losses = 2 * (n + 400 + 4 * 60 + 240) * E * float(r.loss) * 1.1 / (2 * h)
    assert abs((float(a.loss) - float(b.loss)) / (2 * h) - slope) <= rest + inputs + losses + 400 * E * float((d.abs() * v.abs()).sum())


# ------------------------------------------------------------------ block norms
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("rows,cols", [(1, 8), (700, 64), (5, 1000), (9, 2303), (400, 4096), (3, 8200), (320, 8192), (4, 12289), (2, 16384)])
def test_block_norm_backward_without_a_second_norm(xt, yt, rows, cols):
    # X is not read then, whatever it holds
    for post in (True, False):
        for gate in ("cols", "rows"):
            check_norm(rows, cols, xt, yt, yt, gate, post=post, pre=False)
    g = gen(cols)
    x, y, dr, w = normal((rows, cols), g, xt), normal((rows, cols), g, yt), normal((rows, cols), g, xt), normal((cols,), g, yt)
    f = api.block_norm(x, y, post_weight=w)
    a = api.block_norm_backward(dr, None, x, y, f, post_weight=w)
    b = api.block_norm_backward(dr, None, torch.full_like(x, NAN), y, f, post_weight=w)
    assert torch.equal(a.dx, b.dx) and torch.equal(a.dy, b.dy) and torch.equal(a.dpost_weight, b.dpost_weight)


@pytest.mark.parametrize("dtype,cols", [(BF16, 3), (BF16, 259), (BF16, 1001), (F32, 333), (BF16, 4099), (F32, 2305)])
def test_block_norm_ragged_rows_wherever_they_lie(dtype, cols):
    # rows of an odd width start at another place of a 16-byte word each, and so do those that share a slot in turn: what a row
    # gives does not depend on it
    g = gen(cols)
    n = 6000 if cols < 2000 else 1500
    x, y, dr, dz = (normal((n, cols), g, dtype) for _ in range(4))
    w1, w2 = normal((cols,), g, dtype), normal((cols,), g, dtype)
    kw = dict(post_weight=w1, pre_weight=w2)
    f = api.block_norm(x, y, **kw)
    b = api.block_norm_backward(dr, dz, x, y, f, **kw)
    order = torch.randperm(n, device="cuda", generator=g)
    xs, ys, drs, dzs = (t[order] for t in (x, y, dr, dz))
    for _ in range(3):
        fs = api.block_norm(xs, ys, **kw)
        bs = api.block_norm_backward(drs, dzs, xs, ys, fs, **kw)
        assert torch.equal(fs.residual, f.residual[order]) and torch.equal(fs.normed, f.normed[order]) and torch.equal(fs.rstd, f.rstd[:, order])
        assert torch.equal(bs.dx, b.dx[order]) and torch.equal(bs.dy, b.dy[order])
    # and it is the row's alone
    one = api.block_norm(x[5:6], y[5:6], **kw)
    assert torch.equal(one.normed[0], f.normed[5]) and torch.equal(one.residual[0], f.residual[5])


def test_block_norm_gradients_of_no_columns_and_of_no_rows(monkeypatch):
    # sums over nothing are zeros, whatever the memory held
    from newton_schulz_quintic_gb300 import layers

    def garbage(shape, dtype, device):
        t = torch.empty(shape, dtype=dtype, device=device)
        return t.fill_(NAN) if t.is_floating_point() else t
    monkeypatch.setattr(layers, "_empty", garbage)
    for xt, yt in ((BF16, BF16), (F32, BF16), (F32, F32)):
        x, y, w = torch.zeros((5, 0), dtype=xt, device="cuda"), torch.zeros((5, 0), dtype=yt, device="cuda"), torch.zeros(0, dtype=yt, device="cuda")
        for gate in (torch.ones((5, 1), dtype=yt, device="cuda"), torch.ones((5, 7), dtype=F32, device="cuda")[:, 3:4]):
            f = api.block_norm(x, y, gate=gate, post_weight=w, pre_weight=w)
            b = api.block_norm_backward(x, y, x, y, f, gate=gate, post_weight=w, pre_weight=w)
            assert b.dgate.shape == (5, 1) and torch.all(b.dgate == 0) and b.dx.shape == (5, 0) and b.dpost_weight.shape == (0,)
        for kw in (dict(pre_weight=w), dict(post_weight=w), dict(gate=w, post_weight=w, pre_weight=w), dict(gate=y, pre_weight=w)):
            f = api.block_norm(x, y, **kw)
            b = api.block_norm_backward(x, y if "pre_weight" in kw else None, x, y, f, **kw)
            assert f.residual.shape == b.dx.shape == b.dy.shape == (5, 0)
        assert api.block_norm(x, pre_weight=torch.zeros(0, dtype=yt, device="cuda")).residual.shape == (5, 0)
    x, w = torch.zeros((0, 40), dtype=BF16, device="cuda"), torch.ones(40, dtype=BF16, device="cuda")
    f = api.block_norm(x, x, gate=w, post_weight=w, pre_weight=w)
    b = api.block_norm_backward(x, x, x, x, f, gate=w, post_weight=w, pre_weight=w)
    for t in (b.dgate, b.dpost_weight, b.dpre_weight):
        assert t.shape == (40,) and torch.all(t == 0)
