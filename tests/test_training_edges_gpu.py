"""GPU tests of the training operators where a caller's streams, buffers and
values are out of the ordinary. Tolerances as in test_training_gpu.py: U is the
unit roundoff of the output type, E = 2^-24 that of fp32 arithmetic."""
import math
import os
import subprocess
import sys
import textwrap
import threading

import pytest
import torch

from newton_schulz_quintic_gb300 import api

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

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


# ------------------------------------------------------------------ embedding
def test_sliced_ids_on_another_stream():
    # the ids of a batch without its last column are not contiguous: their copy has to run on the call's stream, which
    # waits for nothing here, and must not be handed out again while the call still reads it
    g = gen(1)
    vocab, dim = 5000, 64
    table = normal((vocab, dim), g, BF16)
    batch = torch.randint(0, vocab, (16, 2049), device="cuda", generator=g)
    dout = normal((16 * 2048, dim), g, BF16)
    ids = batch[:, :-1]
    flat = ids.reshape(-1)
    looked_up, grad = api.embed_lookup(table, flat), api.embed_grad(dout, flat, vocab=vocab)
    other = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        torch.cuda._sleep(20_000_000)  # about 10 ms on the current stream
        for s in other:
            a = api.embed_lookup(table, ids, stream=s)
            b = api.embed_grad(dout, ids, vocab=vocab, stream=s)
            torch.full((16, 2048), -1, device="cuda")  # what takes the memory that the current stream has free
            s.synchronize()  # the current stream still sleeps
            assert torch.equal(a.cpu().view(-1, dim), looked_up.cpu()) and torch.equal(b.cpu(), grad.cpu())
    torch.cuda.synchronize()


# ------------------------------------------------------------------ graphs
def step_inputs(seed, rows, vocab, t, n, k, ids):
    r = gen(seed)
    x, y = normal((rows, vocab), r, BF16), torch.randint(0, vocab, (rows,), device="cuda", generator=r)
    dy, ck = normal((t, n), r, BF16), api.checkpoint_store(normal((t, k), r))
    tokens, dout = torch.randint(0, 700, (ids,), device="cuda", generator=r), normal((ids, 64), r, BF16)
    mats = [normal((n, k), r, BF16), normal((24, 200), r, BF16)]

    def go():
        p = api.policy_loss(x, y, torch.ones(rows, device="cuda"), torch.ones(rows, device="cuda"))
        out = [m.clone() for m in mats]
        return [p.loss, p.logp, p.dlogits, api.checkpoint_wgrad(dy, ck, dtype=F32),
                api.embed_grad(dout, tokens, vocab=700), out], out
    return go


def run_step(go, mats=None):
    got, out = go()
    api.orthogonalize_batched(mats if mats is not None else out)
    return got[:-1] + list(mats if mats is not None else out)


@pytest.mark.parametrize("warm", [True, False])
def test_a_graph_outlives_larger_calls_on_its_stream(warm):
    # every operator with scratch of its own (and the orthogonalization) is captured small; larger calls on the same
    # stream then replace that scratch, and the graph's addresses have to stay good: its loss is summed by counters that
    # start at 0, its weight gradient waits for counters of its own. Without a call before the capture, the scratch
    # made during it serves the calls behind it too.
    small = step_inputs(5, 40, 3000, 600, 264, 520, 1500)
    large = step_inputs(6, 900, 3000, 9000, 1032, 1544, 40000)
    ref, ref_large = run_step(small), run_step(large)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mats = small()[1]
    start = [m.clone() for m in mats]
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        if warm:
            run_step(small, mats)
    s.synchronize()
    with torch.cuda.graph(graph, stream=s):
        out = run_step(small, mats)
    with torch.cuda.stream(s):
        if not warm:  # calls of the captured sizes, before the graph ever runs
            assert all(torch.equal(a, b) for a, b in zip(ref, run_step(small)))
        for k in range(3):
            assert all(torch.equal(a, b) for a, b in zip(ref_large, run_step(large)))
            for a, b in zip(mats, start):
                a.copy_(b)
            for a in out[:-2]:
                a.zero_()
            graph.replay()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(ref, out)), k
            for m in range(9):  # more batches than the cache keeps tables of
                api.orthogonalize_batched([torch.ones((64 + m, 256), device="cuda", dtype=BF16)])
    s.synchronize()
    assert api.get_status() == 0


# ------------------------------------------------------------------ policy loss
def policy_rows(vocab, dtype, seed=7, n=8):
    g = gen(seed)
    x, y = normal((n, vocab), g, dtype, 2.0), torch.randint(0, vocab, (n,), device="cuda", generator=g)
    one = torch.ones(n, device="cuda")
    return x, y, one, api.token_logprobs(x, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [65, 40001])
@pytest.mark.parametrize("where,ref", [(w, r) for w in ("logits", "old", "advantage", "weight") for r in (True, False)]
                         + [("ref", True)])
@pytest.mark.parametrize("advantage", [1.0, -1.0, 0.0])
def test_policy_nan_of_a_live_row_reaches_the_loss(dtype, vocab, where, ref, advantage):
    # min(r A, clip(r) A) and clip(r) are NaN where r or A is; what is NaN must not read as a clipped ratio
    x, y, one, lp = policy_rows(vocab, dtype)
    given = dict(old=lp + 0.1, ref=lp - 0.1, advantage=one * advantage, weight=one.clone())
    call = lambda **kw: api.policy_loss(x, y, given["advantage"], given["weight"], old_logp=given["old"],  # noqa: E731
                                        ref_logp=given["ref"] if ref else None, kl_coef=0.1 if ref else 0.0, **kw)
    clean = call()
    assert torch.isfinite(clean.loss) and torch.isfinite(clean.dlogits).all()
    if where == "logits":
        x[3, (int(y[3]) + 7) % vocab] = NAN
    else:
        given[where][3] = NAN
    got, alone = call(), call(grad=False)
    assert torch.isnan(got.loss) and torch.isnan(alone.loss)
    assert torch.isnan(got.dlogits[3]).all()
    assert bool(torch.isnan(got.logp[3])) == (where == "logits")
    keep = torch.arange(8, device="cuda") != 3
    for a, b in ((got.dlogits, clean.dlogits), (got.logp, clean.logp), (got.kl, clean.kl)):
        assert torch.equal(a[keep], b[keep])


def test_policy_overflowing_ratio_without_advantage():
    # r = exp(logp - old) beyond fp32's largest value times A = 0 is 0; times another A it is what the clip leaves
    x, y, one, lp = policy_rows(300, F32)
    old = lp - 120.0
    none = api.policy_loss(x, y, one * 0, one, old_logp=old)
    assert float(none.loss) == 0 and torch.all(none.dlogits == 0)
    up = api.policy_loss(x, y, one, one, old_logp=old, clip_high=0.25)
    assert float(up.loss) == -8 * 1.25 and torch.all(up.dlogits == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_policy_kl_far_apart_without_its_coefficient(dtype):
    # kl_coef = 0: the term is watched, not trained on. k beyond fp32's largest value (its row's target has become
    # impossible next to the reference) is written as infinity and leaves loss and gradient as they are without it
    x, y, one, lp = policy_rows(500, dtype)
    ref = lp.clone()
    ref[1], ref[2] = lp[1] + 95, lp[2] + 1000
    got = api.policy_loss(x, y, one, one, old_logp=lp, ref_logp=ref, kl_coef=0.0)
    plain = api.policy_loss(x, y, one, one, old_logp=lp)
    assert torch.equal(got.loss, plain.loss) and torch.equal(got.dlogits, plain.dlogits)
    # logp is written rounded to fp32: d is up to 2^-21 there, k is d^2 / 2 and a rounding of d
    assert torch.isinf(got.kl[1:3]).all() and torch.all(got.kl[3:].abs() <= 2.0 ** -40)
    x[4, int(y[4])] = -INF  # the target's own logit
    got = api.policy_loss(x, y, one, one, ref_logp=ref, kl_coef=0.0)
    plain = api.policy_loss(x, y, one, one)
    assert torch.equal(got.loss, plain.loss) and torch.equal(got.dlogits, plain.dlogits)
    assert torch.isfinite(got.loss) and torch.isfinite(got.dlogits).all()


# ------------------------------------------------------------------ gated activation
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate_far_below_zero(dtype):
    # silu(g) = g s with s = 1 / (1 + exp(-g)), about exp(g): below g = -87.3 s is a subnormal, above its smallest down
    # to -103; large values of up carry it back into range. As test_gated, and s and g s rounded to 2^-149
    gate = torch.linspace(-104, -80, 24 * 64, device="cuda").view(24, 64).to(dtype)
    up = torch.full_like(gate, 1e30)
    dh = normal((24, 64), gen(9), dtype)
    h, a, b = api.gated_forward(gate, up)

    def near(got, ref, g, far):
        bound = ref.abs() * ((12 + 2 * g.abs()) * 2 * E + U[dtype] * (1 + 2 ** -7)) + far * (2 * g.abs() + 2) * 2.0 ** -149
        assert torch.all((got.double() - ref).abs() <= bound)

    g, u = gate.double(), up.double()
    ref = g * torch.sigmoid(g) * u
    assert float(ref.abs().min()) > 1e-15
    near(h, ref, g, u)
    dgu, again = api.gated_backward(dh, a, b)
    g, u = api.checkpoint_load(a, dtype=F32).double(), api.checkpoint_load(b, dtype=F32).double()
    s, d = torch.sigmoid(g), dh.double()
    near(again, g * s * u, g, u)
    if dtype == F32:  # du = d g s without up lies below bf16's normal range
        near(dgu[:, 64:], d * g * s, g, d.abs() + 1)
    near(dgu[:, :64], d * u * (s + g * s * (1 - s)), g, (d * u).abs())


# ------------------------------------------------------------------ buffers
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("f", [64, 63])
def test_inputs_and_outputs_in_columns_of_one_buffer(dtype, f):
    g = gen(11)
    n = 37
    buf = normal((n, 4 * f), g, dtype)
    a, b, c, d = (buf[:, k * f:(k + 1) * f] for k in range(4))
    h, ck_a, ck_b = api.gated_forward(a, b)
    kept = buf.clone()
    api.gated_forward(a, b, out=c)
    assert torch.equal(c, h) and torch.equal(buf[:, :2 * f], kept[:, :2 * f]) and torch.equal(d, kept[:, 3 * f:])
    ref, _ = api.gated_backward(d, ck_a, ck_b)
    api.gated_backward(d, ck_a, ck_b, dgu=buf[:, :2 * f])
    assert torch.equal(buf[:, :2 * f], ref) and torch.equal(c, h) and torch.equal(d, kept[:, 3 * f:])
    ids = torch.randint(-1, n, (n,), device="cuda", generator=g)
    ref = api.embed_lookup(a, ids)
    api.embed_lookup(a, ids, out=b)
    assert torch.equal(b, ref) and torch.equal(c, h)
    ref = api.embed_grad(a, ids, vocab=n)
    api.embed_grad(a, ids, grad=c)
    assert torch.equal(c, ref) and torch.equal(d, kept[:, 3 * f:])
    y, one = torch.randint(0, f, (n,), device="cuda", generator=g), torch.ones(n, device="cuda")
    ref = api.policy_loss(d, y, one, one)
    got = api.policy_loss(d, y, one, one, dlogits=b)
    assert torch.equal(b, ref.dlogits) and torch.equal(got.loss, ref.loss) and torch.equal(c, api.embed_grad(a, ids, vocab=n))


# ------------------------------------------------------------------ long rows, long lists, many elements
def padded(x, extra):
    """x as a view with `extra` elements more between its rows, one element into its buffer."""
    n, m = x.shape
    v = torch.full((n * (m + extra) + 64,), 7.0, dtype=x.dtype, device=x.device)[1:1 + n * (m + extra)].view(n, m + extra)[:, :m]
    v.copy_(x)
    return v


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n,vocab,dim,extra", [(3000, 700, 2304, 0), (3000, 50, 1543, 0), (1025, 3, 4096, 0), (5000, 300, 2048, 3),
                                               (20000, 7, 1032, 0)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_of_long_lists_and_several_column_ranges(dtype, gdtype, n, vocab, dim, extra, accumulate):
    # more than 1024 positions and rows longer than a CTA covers (1024 bf16 or 512 fp32 columns in pieces, 512 or 128 in
    # joins); a third of the positions share one id, whose run crosses many pieces
    g = gen(n + dim)
    ids = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    u = torch.rand(n, device="cuda", generator=g)
    ids[u < 0.3], ids[u > 0.95] = vocab // 2, -1
    dout = normal((n, dim), g, dtype)
    dout[ids < 0] = NAN
    old = normal((vocab, dim), g, gdtype)
    live = ids >= 0
    ref, mag = (torch.zeros((vocab, dim), dtype=F64, device="cuda") for _ in range(2))
    ref.index_put_((ids[live],), dout[live].double(), accumulate=True)
    mag.index_put_((ids[live],), dout[live].double().abs(), accumulate=True)
    most, scale = int(torch.bincount(ids[live]).max()), 0.37
    ref, mag = ref * float(torch.tensor(scale)), mag * scale
    grad = old.clone() if accumulate else torch.full_like(old, 3.0)
    if extra:
        dout, grad = padded(dout, extra), padded(grad, extra)
    if accumulate:
        ref, mag = ref + old.double(), mag + old.double().abs()
    got = api.embed_grad(dout, ids, grad=grad, scale=scale, accumulate=accumulate).double()
    # sums of `most` terms in fp32 in any order, scaled and added: (most + 2) roundings of at most mag
    assert torch.all((got - ref).abs() <= (most + 2) * E * mag + U[gdtype] * ref.abs() * (1 + 2 ** -7))


def test_wgrad_holds_every_slice_of_fp32():
    # one row a group: an entry of G is one product, so dY's three bf16 slices show. Their products are exact and their
    # two additions lose up to a unit (2 E) each: below 6 E with the slices' own remainder, where two slices alone
    # err by up to 2^-17 (128 E)
    r = gen(13)
    dy, ck = normal((6, 200), r), api.checkpoint_store(normal((6, 264), r))
    x = api.checkpoint_load(ck, dtype=F32).double()
    off = torch.arange(7, dtype=torch.int32, device="cuda")
    ref = dy.double()[:, :, None] * x[:, None, :]
    for view in (dy, padded(dy, 3)):
        got = api.checkpoint_wgrad(view, ck, offsets=off)
        assert torch.all((got.double() - ref).abs() <= 6 * E * ref.abs())
    high = dy.to(BF16).double()
    two = high + (dy.double() - high).to(BF16).double()
    assert torch.any((two[:, :, None] * x[:, None, :] - ref).abs() > 24 * E * ref.abs())


@pytest.mark.parametrize("k", [64, 63])
def test_wgrad_adds_to_subnormals(k):
    # added by TMA where G's rows are 16-byte aligned, element by element where not: neither drops a subnormal of G,
    # of the sum 1.5 * 2^-125 - 1.25 * 2^-125 = 2^-127, or of nothing added
    x = torch.zeros((8, k), device="cuda")
    x[0] = 2.0 ** -120
    dy = torch.zeros((8, 40), device="cuda", dtype=BF16)
    dy[0, :20] = -1.25 * 2.0 ** -5
    ck = api.checkpoint_store(x)
    grad = torch.full((1, 40, k), 1.5 * 2.0 ** -125, device="cuda")
    grad[:, 20:] = 2.0 ** -130
    api.checkpoint_wgrad(dy, ck, grad=grad, accumulate=True)
    assert torch.all(grad[:, :20].double() == 2.0 ** -127) and torch.all(grad[:, 20:].double() == 2.0 ** -130)


def test_offsets_past_32_bits():
    # more than 2^31 elements each; what the last rows give is compared with a call of those rows alone
    g = gen(14)
    tail = 64
    # the table's gradient
    vocab, dim = (1 << 20) + 3, 2304
    dout = normal((1500, dim), g, BF16)
    ids = torch.full((1500,), vocab - 1, device="cuda")
    ids[700:] = torch.arange(vocab - 801, vocab - 1, device="cuda")
    grad = torch.empty((vocab, dim), dtype=BF16, device="cuda")
    for part in (slice(0, 1500), slice(600, 800)):  # by sorting, and by searching the list
        grad[-900:] = 5
        api.embed_grad(dout[part], ids[part], grad=grad)
        small = api.embed_grad(dout[part], torch.where(ids[part] >= vocab - 900, ids[part] - (vocab - 900), -1), vocab=900)
        assert torch.equal(grad[-900:], small)
    del grad, dout
    # gated activation and its 8-bit form
    n, f = 150001, 14336
    gu, dh = torch.zeros((n, 2 * f), dtype=BF16, device="cuda"), torch.zeros((n, f), dtype=BF16, device="cuda")
    gu[-tail:], dh[-tail:] = normal((tail, 2 * f), g, BF16), normal((tail, f), g, BF16)
    h, a, b = api.gated_forward(gu[:, :f], gu[:, f:])
    hs, sa, sb = api.gated_forward(gu[-tail:, :f], gu[-tail:, f:])
    assert torch.equal(h[-tail:], hs) and torch.equal(a.q[-tail:], sa.q) and torch.equal(b.scales[-tail:], sb.scales)
    dgu, again = api.gated_backward(dh, a, b)
    ds, ags = api.gated_backward(dh[-tail:], sa, sb)
    assert torch.equal(dgu[-tail:], ds) and torch.equal(again[-tail:], ags)
    del h, dgu, again
    # a weight gradient from the last rows of both operands: the rows before them are zeros
    off = torch.tensor([0, n - tail, n], dtype=torch.int32, device="cuda")
    big = api.checkpoint_wgrad(dh[:, :32], a, offsets=off, dtype=F32)
    assert torch.all(big[0] == 0) and torch.equal(big[1], api.checkpoint_wgrad(dh[-tail:, :32], sa, dtype=F32)[0])
    wide = api.checkpoint_store(normal((n, 32), g))
    got = api.checkpoint_wgrad(dh, wide, offsets=off, dtype=F32)[1].double()
    x = api.checkpoint_load(wide, dtype=F32)[-tail:].double()
    d = dh[-tail:].double()
    assert torch.all((got - d.t() @ x).abs() <= 64 * 2 * E * (d.abs().t() @ x.abs()) + 1e-37)
    del gu, dh, a, b, wide
    # the policy loss
    n, vocab = 16390, 131080
    x = torch.zeros((n, vocab), dtype=BF16, device="cuda")
    x[-tail:] = normal((tail, vocab), g, BF16, 2.0)
    y = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    one = torch.ones(n, device="cuda")
    ref = api.policy_loss(x[-tail:].clone(), y[-tail:], one[-tail:], one[-tail:])
    got = api.policy_loss(x, y, one, one, dlogits=x)
    # one row of either is summed in another order: vocab / 128 + 64 additions, and the bf16 rounding
    tol = (vocab / 128 + 64) * 2 * E
    assert torch.all((got.logp[-tail:] - ref.logp).abs() <= tol * 16)
    assert torch.all((x[-tail:].double() - ref.dlogits.double()).abs() <= ref.dlogits.double().abs() * (2.0 ** -7 + 32 * tol) + 1e-37)


def test_operators_from_several_threads():
    # each thread on a stream of its own, with scratch and counters of its own
    work = [step_inputs(20 + k, 40 + 60 * k, 3000, 600 + 300 * k, 264, 520, 1500 + 700 * k) for k in range(3)]
    ref = [run_step(w) for w in work]
    torch.cuda.synchronize()
    bad = []

    def go(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got = run_step(work[k])
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(ref[k], got)):
                        bad.append(k)
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=go, args=(k,)) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and api.get_status() == 0


CHILD = textwrap.dedent("""
    import os, sys
    import torch
    sys.path.insert(0, %r)
    from newton_schulz_quintic_gb300 import build, api
    os.environ["NS_LIBRARY_PATH"] = build.build()
    api.load_library()
    bf16, f32 = torch.bfloat16, torch.float32
    for dt, gd in ((bf16, bf16), (f32, f32), (bf16, f32), (f32, bf16)):
        for n, vocab, dim in ((3000, 700, 2304), (3000, 50, 1543)):
            ids = torch.randint(-1, vocab, (n,), device="cuda")
            ids[torch.rand(n, device="cuda") < 0.3] = vocab // 2
            dout = torch.randn(n, dim, device="cuda").to(dt)
            g = api.embed_grad(dout, ids, vocab=vocab, dtype=gd)
            api.embed_grad(dout, ids, grad=g, accumulate=True)
    assert api.get_status() == 0, "a bounds check fired"
    print("debug-bounds ok")
""") % ROOT


def test_debug_build_checks_several_column_ranges():
    env = dict(os.environ, NS_BUILD_TAG="debugbounds", NS_EXTRA_NVCC_FLAGS="-DNS_DEBUG_BOUNDS")
    env.pop("NS_LIBRARY_PATH", None)
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True, timeout=1200, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "debug-bounds ok" in r.stdout


def test_threads_that_use_the_per_thread_stream():
    # cudaStreamPerThread (handle 2) is another stream in each thread: they must not share scratch. (Every output is made
    # beforehand: torch's allocator goes by the handle.)
    r = gen(30)
    work = []
    for k in range(3):
        t, ids = 600 + 300 * k, 1500 + 700 * k
        dy, ck = normal((t, 264), r, BF16), api.checkpoint_store(normal((t, 520), r))
        tokens, dout = torch.randint(0, 700, (ids,), device="cuda", generator=r), normal((ids, 64), r, BF16)
        mats = [normal((264, 520 + 8 * k), r, BF16) for _ in range(8)]
        ref = [api.checkpoint_wgrad(dy, ck, dtype=F32), api.embed_grad(dout, tokens, vocab=700), mats[0].clone()]
        mats[1:] = [mats[0].clone() for _ in mats[1:]]
        api.orthogonalize_batched([ref[2]])
        out = [(torch.empty_like(ref[0]), torch.empty_like(ref[1]), m) for m in mats]
        work.append((dy, ck, dout, tokens, ref, out))
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(3)

    def go(dy, ck, dout, tokens, ref, out):
        try:
            s = torch.cuda.ExternalStream(2)
            with torch.cuda.stream(s):
                start.wait()
                for a, b, m in out:
                    api.checkpoint_wgrad(dy, ck, grad=a)
                    api.embed_grad(dout, tokens, grad=b)
                    api.orthogonalize_batched([m])
                s.synchronize()
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=go, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad and api.get_status() == 0
    for *_, ref, out in work:
        assert all(torch.equal(a, b) for got in out for a, b in zip(ref, got))
