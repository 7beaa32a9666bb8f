"""Refusals of the expert-layer operators, checked before anything is launched
(no GPU needed: fake device pointers, so only where nothing can launch), what
the Python layer rejects, and how it calls the library."""
import contextlib
import ctypes

import pytest
import torch

from newton_schulz_quintic_gb300 import api, build, layers, training

OK, EINVAL, EALIGN, ENOMEM, ENODEV = 0, -1, -2, -3, -6
NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="uses fake device pointers: only run where nothing can launch")
A, B, C, D, E_, F, G, H = (0x10000000 * k for k in range(1, 9))
P = 4096  # a page further


@pytest.fixture(scope="module")
def call():
    build.build()
    lib = api.load_library()

    def go(name, args, **change):
        assert set(change) <= set(args), set(change) - set(args)
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, training._PROTOTYPES[name]
        assert len(f.argtypes) == len(args)
        return f(*[{**args, **change}[k] for k in args])
    return go


ROUTE = dict(x=A, ld=40, rows=10, experts=40, k=4, live=B, renorm=1, cb=0.1, cz=0.1, ids=C, weights=C + P, logz=C + 2 * P, counts=C + 3 * P,
             offsets=C + 4 * P, order=C + 5 * P, live_rows=C + 6 * P, loss=C + 7 * P, work=D, bytes=1 << 20, dtype=1, stream=None)
BACK = dict(x=A, ld=40, rows=10, experts=40, k=4, ids=C, weights=C + P, dw=C + 2 * P, logz=C + 3 * P, counts=C + 4 * P, live_rows=C + 5 * P,
            renorm=1, cb=0.1, cz=0.1, d=D, ldd=40, dtype=1, stream=None)
STORE = dict(x=A, ld=64, xrows=10, index=None, per=1, rows=10, cols=64, q=B, s=C, dtype=1, stream=None)
TILES = dict(x=A, ld=64, groups=2, rows=10, cols=64, q=B, s=C, dtype=1, stream=None)
LOAD = dict(q=B, s=C, tiles=1, groups=2, rows=10, cols=64, out=A, ld=64, dtype=1, stream=None)
MM = dict(qa=A, sa=B, rows=10, k=64, qw=C, sw=D, n=48, back=0, off=E_, groups=2, out=F, ld=48, dtype=1, stream=None)
NORM = dict(x=A, ldx=64, y=B, ldy=64, gate=C, form=1, ldg=0, post=C + P, pre=C + 2 * P, rows=10, cols=64, a=1.0, b=1.0, eps=1e-6, r=D, ldr=64,
            z=E_, ldz=64, rstd1=F, rstd2=F + P, dtype=1, bdtype=1, wdtype=1, gdtype=1, stream=None)
NBACK = dict(dr=A, lddr=64, dz=B, lddz=64, x=C, ldx=64, y=D, ldy=64, gate=E_, form=1, ldg=0, post=E_ + P, pre=E_ + 2 * P, rstd1=F, rstd2=F + P,
             rows=10, cols=64, a=1.0, b=1.0, dx=G, lddx=64, dy=G + 16 * P, lddy=64, dgate=F + 2 * P, lddg=64, dpost=F + 3 * P, dpre=F + 4 * P,
             work=H, bytes=1 << 20, dtype=1, bdtype=1, wdtype=1, gdtype=1, stream=None)
DROP = dict(x=A, ldx=64, res=B, ldr=64, rows=10, cols=64, p=0.1, seed=1, offset=2, state=C, out=D, ldo=64, dtype=1, odtype=1, stream=None)
ALL = [("ns_route", ROUTE), ("ns_route_backward", BACK), ("ns_blocks_store_rows", STORE), ("ns_blocks_store_tiles", TILES), ("ns_blocks_load", LOAD),
       ("ns_blocks_matmul", MM), ("ns_block_norm", NORM), ("ns_block_norm_backward", NBACK), ("ns_dropout", DROP)]


@NO_GPU
@pytest.mark.parametrize("name,good", ALL)
def test_good_arguments_get_as_far_as_the_device(call, name, good):
    assert call(name, good) == ENODEV
    for k in ("dtype", "bdtype", "wdtype", "gdtype", "odtype"):
        if k in good:
            assert call(name, good, **{k: 2}) == EINVAL, k
    for k in ("ld", "ldd", "ldx", "ldy", "ldr", "ldz", "ldo", "lddr", "lddz", "lddx", "lddy"):
        if k in good:
            assert call(name, good, **{k: good[k] - 1}) == EINVAL, k
    for k in ("rows", "xrows", "cols", "n", "k", "experts"):
        if k in good:
            assert call(name, good, **{k: -1}) == EINVAL, k
            if k != "experts" and not (name.startswith("ns_route") and k == "k"):
                assert call(name, good, **{k: 1 << 31}) == EINVAL, k


@NO_GPU
def test_route_refusals(call):
    r = lambda **k: call("ns_route", ROUTE, **k)  # noqa: E731
    assert r(live=None) == ENODEV
    for k in ("x", "ids", "weights", "logz", "order", "counts", "offsets", "live_rows", "loss", "work"):
        assert r(**{k: None}) == EINVAL, k
    assert r(k=0) == EINVAL and r(k=33) == EINVAL and r(k=41, experts=41, ld=41) == EINVAL and r(experts=1025, ld=1025) == EINVAL
    assert r(experts=3, ld=40) == EINVAL and r(renorm=2) == EINVAL and r(cb=float("nan")) == EINVAL and r(cz=float("inf")) == EINVAL
    assert r(rows=1 << 29, live=None) == EINVAL  # more than 2^30 slots
    assert r(bytes=100) == ENOMEM
    assert r(ids=A + 400) == EINVAL and r(weights=C + 80) == EINVAL and r(work=C) == EINVAL and r(loss=D + 16) == EINVAL
    assert r(x=A + 1) == EALIGN and r(order=C + 5 * P + 2) == EALIGN and r(work=D + 1) == EALIGN
    assert r(rows=0, x=None, ids=None, weights=None, logz=None, order=None) == ENODEV  # writes counts and the loss
    lib = api.load_library()
    lib.ns_route_workspace.restype = ctypes.c_int64
    lib.ns_route_workspace.argtypes = [ctypes.c_int64, ctypes.c_int]
    assert lib.ns_route_workspace(10, 0) == -1 and lib.ns_route_workspace(-1, 4) == -1 and lib.ns_route_workspace(5, 1025) == -1
    for rows in (0, 1, 16, 17, 5000, 100000):  # what the Python layer allocates
        assert lib.ns_route_workspace(rows, 76) == 4 * max(1, min(-(-rows // 16), layers._MAX_STRETCHES)) * (2 * 76 + 2)
    b = lambda **k: call("ns_route_backward", BACK, **k)  # noqa: E731
    assert b(dw=None) == ENODEV and b(d=A) == ENODEV and b(rows=0, x=None) == OK
    assert b(d=A, ldd=41) == EINVAL and b(d=A + 2) == EINVAL and b(d=C) == EINVAL and b(d=D + 1) == EALIGN and b(ids=C + 2) == EALIGN
    for k in ("x", "ids", "weights", "logz", "counts", "live_rows", "d"):
        assert b(**{k: None}) == EINVAL, k


@NO_GPU
def test_blocks_refusals(call):
    s = lambda **k: call("ns_blocks_store_rows", STORE, **k)  # noqa: E731
    assert s(rows=9) == EINVAL and s(per=2) == EINVAL                  # only with an index
    assert s(index=D, rows=77, per=3) == ENODEV and s(index=D, per=0) == EINVAL and s(index=D + 2) == EALIGN
    assert s(index=D, rows=0, q=None) == OK and s(rows=0, xrows=0, x=None) == OK and s(index=D, xrows=0, x=None) == ENODEV
    assert s(q=B + 8) == EALIGN and s(s=C + 8) == EALIGN and s(x=A + 1) == EALIGN
    assert s(q=A + 64) == EINVAL and s(s=B + 16) == EINVAL and s(index=B, rows=10) == EINVAL and s(q=None) == EINVAL
    t = lambda **k: call("ns_blocks_store_tiles", TILES, **k)  # noqa: E731
    assert t(groups=-1) == EINVAL and t(groups=0) == OK and t(q=A) == EINVAL and t(s=A + 64) == EINVAL
    assert t(groups=1 << 30, rows=1 << 20) == EINVAL
    g = lambda **k: call("ns_blocks_load", LOAD, **k)  # noqa: E731
    assert g(tiles=0) == EINVAL and g(tiles=0, groups=1) == ENODEV and g(tiles=2) == EINVAL
    assert g(out=B) == EINVAL and g(out=C - 64) == EINVAL and g(out=A + 1) == EALIGN and g(out=None) == EINVAL and g(groups=0) == OK
    m = lambda **k: call("ns_blocks_matmul", MM, **k)  # noqa: E731
    assert m(off=None) == EINVAL and m(off=None, groups=1) == ENODEV and m(groups=-1) == EINVAL and m(back=2) == EINVAL
    assert m(back=1) == ENODEV and m(groups=0, qw=None, sw=None) == ENODEV   # writes zeros
    assert m(rows=0, qa=None, out=None) == OK and m(n=0, ld=0, out=None) == OK and m(k=0, qa=None, sa=None, qw=None, sw=None) == ENODEV
    for k in ("qa", "sa", "qw", "sw", "out"):
        assert m(**{k: None}) == EINVAL, k
        assert m(**{k: MM[k] + (8 if k != "out" else 1)}) == EALIGN, k
    assert m(off=E_ + 2) == EALIGN
    for at in (A, B, C, D, E_):
        assert m(out=at) == EINVAL
    assert m(groups=1 << 20, k=1 << 12, n=1 << 12, ld=1 << 12) == EINVAL     # a stack beyond 2^42 elements
    lib = api.load_library()
    for f, cases in (("ns_blocks_pitch", [(0, 0), (1, 16), (17, 32), (-1, -1)]), ("ns_blocks_scale_pitch", [(0, 0), (1, 4), (512, 4), (513, 8), (-1, -1)])):
        fn = getattr(lib, f)
        fn.restype, fn.argtypes = ctypes.c_int64, [ctypes.c_int64]
        for cols, want in cases:
            assert fn(cols) == want
            if cols >= 0:
                assert want == (layers._pitch if f == "ns_blocks_pitch" else layers._scale_pitch)(cols)


@NO_GPU
def test_block_norm_refusals(call):
    n = lambda **k: call("ns_block_norm", NORM, **k)  # noqa: E731
    assert n(r=A) == ENODEV and n(z=B) == ENODEV                             # over x and y
    assert n(r=A + 2) == EINVAL and n(r=A, ldr=65) == EINVAL and n(z=A) == EINVAL and n(r=B) == EINVAL and n(z=D) == EINVAL
    assert n(y=None) == EINVAL and n(y=None, gate=None, form=0, post=None) == ENODEV
    assert n(y=None, gate=None, form=0, post=None, pre=None) == EINVAL       # nothing to do
    assert n(gate=None) == EINVAL and n(form=0) == EINVAL and n(form=4) == EINVAL and n(form=2, ldg=1) == ENODEV and n(form=3, ldg=63) == EINVAL
    assert n(cols=16385, ldx=16385, ldy=16385, ldr=16385, ldz=16385) == EINVAL
    assert n(bdtype=0) == EINVAL and n(dtype=0, bdtype=1, r=D) == ENODEV     # y wider than x; an fp32 stream
    assert n(eps=-1.0) == EINVAL and n(eps=float("nan")) == EINVAL and n(a=float("inf")) == EINVAL
    assert n(rstd1=None) == EINVAL and n(rstd2=None) == EINVAL and n(z=None) == EINVAL and n(pre=None, z=None, rstd2=None) == ENODEV
    assert n(x=A + 1) == EALIGN and n(post=C + P + 1) == EALIGN and n(rstd1=F + 2) == EALIGN and n(rows=0, x=None, r=None) == OK
    assert n(rstd1=F + P) == EINVAL and n(rstd1=A) == EINVAL
    b = lambda **k: call("ns_block_norm_backward", NBACK, **k)  # noqa: E731
    assert b(dx=A) == ENODEV and b(dy=B) == ENODEV and b(dr=None) == ENODEV
    assert b(dx=C) == EINVAL and b(dx=B) == EINVAL and b(dy=A) == EINVAL and b(dpost=F) == EINVAL and b(dpre=F + 3 * P) == EINVAL
    assert b(dr=None, pre=None, dz=None) == EINVAL and b(pre=None, dz=None, dpre=None, rstd2=None) == ENODEV
    for k in ("dz", "x", "dx", "dy", "dgate", "dpost", "dpre", "rstd1", "rstd2", "work"):
        assert b(**{k: None}) == EINVAL, k
    assert b(bytes=4) == ENOMEM and b(work=A) == EINVAL and b(work=H + 2) == EALIGN
    assert b(rows=0, x=None, dr=None, dz=None, y=None, dx=None, dy=None) == ENODEV  # writes zeros
    lib = api.load_library()
    lib.ns_block_norm_workspace.restype = ctypes.c_int64
    lib.ns_block_norm_workspace.argtypes = [ctypes.c_int64, ctypes.c_int64]
    assert lib.ns_block_norm_workspace(5, 16385) == -1 and lib.ns_block_norm_workspace(-1, 5) == -1
    for rows in (0, 1, 303, 305, 10 ** 6):
        assert lib.ns_block_norm_workspace(rows, 100) == 4 * max(1, min(rows, layers._MAX_PARTS)) * 200


@NO_GPU
def test_dropout_refusals(call):
    d = lambda **k: call("ns_dropout", DROP, **k)  # noqa: E731
    assert d(state=None) == ENODEV and d(res=None) == ENODEV and d(out=A) == ENODEV and d(out=B) == ENODEV
    assert d(p=-0.1) == EINVAL and d(p=1.1) == EINVAL and d(p=float("nan")) == EINVAL and d(p=1.0) == ENODEV
    assert d(odtype=0, ldo=64) == ENODEV and d(odtype=0, res=None) == EINVAL and d(dtype=0) == EINVAL
    assert d(out=A + 2) == EINVAL and d(out=A, ldo=65) == EINVAL and d(out=B + 128) == EINVAL and d(out=C) == EINVAL
    assert d(odtype=0, out=A) == EINVAL                                      # over x, but wider
    assert d(state=C + 4) == EALIGN and d(x=A + 1) == EALIGN and d(rows=0, x=None, out=None) == OK and d(out=None) == EINVAL
    most = (1 << 30) - 1
    wide = dict(ldx=1 << 30, ldr=1 << 30, ldo=1 << 30, rows=2, res=1 << 44, out=1 << 45, state=None)
    assert d(cols=most, **wide) == ENODEV and d(cols=most + 1, **wide) == EINVAL


@NO_GPU
def test_columns_of_one_buffer_side_by_side(call):
    assert call("ns_dropout", DROP, ldx=256, ldo=256, out=A + 128) == ENODEV and call("ns_dropout", DROP, ldx=256, ldo=256, out=A + 126) == EINVAL
    assert call("ns_block_norm", NORM, ldx=256, ldr=256, r=A + 128) == ENODEV and call("ns_block_norm", NORM, ldx=256, ldr=256, r=A + 130 - 4) == EINVAL


def test_python_layer_rejects_before_the_library():
    x = torch.zeros(4, 8)
    for bad in (lambda: api.route(x, 2), lambda: api.blocks_store(x), lambda: api.blocks_store(x[None], tiles=True), lambda: api.block_norm(x, x),
                lambda: api.dropout(x, 0.1, 1), lambda: api.Blocks8(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8), 16),
                lambda: api.Blocks8(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8), 16, tiles=True),
                lambda: api.Blocks8(torch.zeros((4, 15), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8), 15)):
        with pytest.raises(ValueError):
            bad()
    assert api.dropout_counters(3, 17) == 9


# ------------------------------------------------------------------ the Python layer on stand-ins
DEV = torch.device("cuda", 0)


class Stub:
    """A CUDA tensor as far as the argument checks look at one."""

    is_cuda, device = True, DEV

    def __init__(self, shape, dtype, strides=None):
        self.shape, self.dtype, self.strides = tuple(shape), dtype, strides

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def stride(self, axis=None):
        s = [1] * len(self.shape)
        for k in range(len(s) - 2, -1, -1):
            s[k] = s[k + 1] * self.shape[k + 1]
        s = self.strides or s
        return tuple(s) if axis is None else s[axis]

    def is_contiguous(self):
        return self.strides is None

    def data_ptr(self):
        return 0x1000

    def unbind(self):
        return [Stub(self.shape[1:], self.dtype) for _ in range(self.shape[0])]


@pytest.fixture
def calls(monkeypatch):
    made = []

    @contextlib.contextmanager
    def on(device, stream):
        yield

    monkeypatch.setattr(layers, "_on", on)
    monkeypatch.setattr(layers, "_call", lambda name, *a: made.append((name, a)))
    monkeypatch.setattr(layers, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(layers, "_empty", lambda shape, dtype, device: Stub(shape if isinstance(shape, tuple) else (shape,), dtype))
    return made


BF16, F32 = torch.bfloat16, torch.float32


def test_argument_checks_of_the_python_layer(calls):
    m = lambda n, c, dt=BF16, **k: Stub((n, c), dt, **k)  # noqa: E731
    v = lambda c, dt=BF16: Stub((c,), dt)  # noqa: E731
    x, w = m(6, 16), v(16)
    bad = [
        lambda: api.block_norm(x), lambda: api.block_norm(x, m(6, 17)), lambda: api.block_norm(x, m(6, 16, F32), post_weight=w),
        lambda: api.block_norm(x, gate=w, pre_weight=w), lambda: api.block_norm(x, x, gate=v(15), pre_weight=w),
        lambda: api.block_norm(x, x, post_weight=w, pre_weight=v(16, F32)), lambda: api.block_norm(x, x, gate=m(5, 1), pre_weight=w),
        lambda: api.block_norm(x, x, normed=x), lambda: api.block_norm(x, x, residual=m(6, 16, F32)),
        lambda: api.block_norm(m(6, 16, strides=(16, 2)), x, pre_weight=w), lambda: api.block_norm(m(6, 16, strides=(8, 1)), x, pre_weight=w),
        lambda: api.dropout(x, 1.5, 0), lambda: api.dropout(x, 0.1, 0, residual=m(6, 15)), lambda: api.dropout(m(6, 16, F32), 0.1, 0, residual=x),
        lambda: api.dropout(x, 0.1, 0, state=v(2, F32)), lambda: api.dropout(x, 0.1, 0, out=m(6, 16, F32)), lambda: api.route(x, 0), lambda: api.route(x, 17),
        lambda: api.route(x, 2, live=v(6, torch.uint8)), lambda: api.route(x, 2, live=Stub((5,), torch.bool)),
        lambda: api.blocks_store(x, per=2), lambda: api.blocks_store(x, rows=v(9, torch.int32), per=0), lambda: api.blocks_store(x, rows=v(9, torch.int64)),
        lambda: api.blocks_store(x, tiles=True, rows=v(9, torch.int32)),
    ]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()
    a, b = layers.Blocks8._empty(1, 6, 16, False, DEV), layers.Blocks8._empty(2, 5, 16, True, DEV)
    one = layers.Blocks8._empty(1, 16, 5, True, DEV)
    for f in (lambda: api.blocks_matmul(b, b), lambda: api.blocks_matmul(a, a), lambda: api.blocks_matmul(a, b), lambda: api.blocks_matmul(a, one),
              lambda: api.blocks_matmul(a, b, offsets=v(2, torch.int32)), lambda: api.blocks_matmul(a, b, offsets=v(3, torch.int64)),
              lambda: api.blocks_matmul(a, one, transpose=True, dtype=torch.float16), lambda: api.blocks_load(a, dtype=torch.float16),
              lambda: api.blocks_matmul(a, one, transpose=True, out=m(6, 6))):
        with pytest.raises((ValueError, TypeError)):
            f()
    assert not calls
    assert api.blocks_matmul(a, one, transpose=True).shape == (6, 5)
    assert api.blocks_matmul(a, b, offsets=v(3, torch.int32)).shape == (6, 5)
    api.block_norm(x, x, gate=m(6, 1), pre_weight=w)
    f = api.block_norm(x, x, gate=m(6, 16), pre_weight=w, post_weight=w)
    for k in (lambda: api.block_norm_backward(x, None, x, x, f, pre_weight=w), lambda: api.block_norm_backward(None, None, x, x, f, post_weight=w),
              lambda: api.block_norm_backward(x, x, x, x, f._replace(rstd=v(6, F32)), pre_weight=w),
              lambda: api.block_norm_backward(x, x, x, None, f, pre_weight=w, dy=x)):
        with pytest.raises(ValueError):
            k()
    g = api.block_norm_backward(x, x, x, x, f, gate=m(6, 16), pre_weight=w, post_weight=w)
    assert g.dgate.shape == (6, 16) and g.dpost_weight.shape == (16,)
    api.dropout(x, 0.25, -1, offset=-3, residual=m(6, 16, F32))
    assert [c[0] for c in calls] == ["ns_blocks_matmul", "ns_blocks_matmul", "ns_block_norm", "ns_block_norm", "ns_block_norm_backward", "ns_dropout"]
    assert calls[-1][1][7:9] == ((1 << 64) - 1, (1 << 64) - 3)  # modulo 2^64
    assert [c[1][5] for c in calls[2:4]] == [2, 3]              # forms of the gate
