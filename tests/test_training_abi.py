"""Refusals of the training operators, checked before anything is launched
(no GPU needed: fake device pointers, so only where nothing can launch), and
the arguments that the Python layer rejects."""
import ctypes

import pytest
import torch

from newton_schulz_quintic_gb300 import api, build, training

OK, EINVAL, EALIGN, ENODEV = 0, -1, -2, -6
NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="uses fake device pointers: only run where nothing can launch")
A, B, C, D, E_, F = (0x10000000 * k for k in range(1, 7))


@pytest.fixture(scope="module")
def call():
    build.build()
    lib = api.load_library()

    def go(name, args, **change):
        names = list(args)
        assert set(change) <= set(names)
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, training._PROTOTYPES[name]
        return f(*[{**args, **change}[k] for k in names])
    return go


LOOKUP = dict(table=A, ld=64, vocab=100, dim=64, ids=B, idt=1, count=10, scale=1.0, out=C, ldo=64, dtype=1, stream=None)
GRAD = dict(dout=A, ld=64, ids=B, idt=1, count=10, scale=1.0, grad=C, ldg=64, vocab=100, dim=64, dtype=1, gdtype=0, acc=0,
            stream=None)
LOGP = dict(x=A, ld=100, rows=10, vocab=100, y=B, idt=1, it=1.0, logp=C, dtype=1, stream=None)
POLICY = dict(x=A, ld=100, rows=10, vocab=100, y=B, idt=1, old=B + 4096, ref=B + 8192, adv=B + 12288, w=B + 16384, it=1.0, lo=0.2,
              hi=0.2, beta=0.1, loss=C, logp=C + 4096, kl=C + 8192, d=D, ldd=100, dtype=1, stream=None)
STORE = dict(x=A, ld=64, rows=10, cols=64, q=B, s=C, dtype=1, stream=None)
LOAD = dict(q=B, s=C, rows=10, cols=64, out=A, ld=64, dtype=1, stream=None)
FORWARD = dict(gate=A, up=A + 128, ld=128, rows=10, cols=64, h=B, ldh=64, qg=C, sg=C + 4096, qu=D, su=D + 4096, dtype=1,
               stream=None)
BACKWARD = dict(dh=A, ld=64, qg=C, sg=C + 4096, qu=D, su=D + 4096, rows=10, cols=64, dg=B, du=B + 128, ldd=128, h=E_, ldh=64,
                dtype=1, stream=None)
WGRAD = dict(dy=A, ld=64, rows=10, n=64, q=B, s=C, k=64, off=D, groups=2, grad=E_, dtype=1, gdtype=1, acc=0, stream=None)


@NO_GPU
@pytest.mark.parametrize("name,good", [("ns_embed_lookup", LOOKUP), ("ns_embed_grad", GRAD), ("ns_token_logprobs", LOGP),
                                       ("ns_policy_loss", POLICY), ("ns_ckpt_store", STORE), ("ns_ckpt_load", LOAD),
                                       ("ns_gated_forward", FORWARD), ("ns_gated_backward", BACKWARD),
                                       ("ns_ckpt_wgrad", WGRAD)])
def test_good_arguments_get_as_far_as_the_device(call, name, good):
    assert call(name, good) == ENODEV
    assert call(name, good, dtype=2) == EINVAL
    for k in ("ld", "ldo", "ldg", "ldd", "ldh"):
        if k in good:
            assert call(name, good, **{k: 63 if good[k] <= 100 else 60}) == EINVAL, k
    for k in ("rows", "count", "vocab", "dim", "cols", "n", "k"):
        if k in good:
            assert call(name, good, **{k: -1}) == EINVAL, k
            assert call(name, good, **{k: 1 << 31}) == EINVAL, k


@NO_GPU
def test_embed_refusals(call):
    for name, good, out in (("ns_embed_lookup", LOOKUP, "out"), ("ns_embed_grad", GRAD, "grad")):
        assert call(name, good, idt=2) == EINVAL
        assert call(name, good, ids=None) == EINVAL
        assert call(name, good, ids=B + 4) == EALIGN
        assert call(name, good, ids=B + 4, idt=0) == ENODEV
        assert call(name, good, **{out: None}) == EINVAL
        assert call(name, good, **{out: A + 128}) == EINVAL       # inside the input
        assert call(name, good, **{out: B - 64}) == EINVAL        # reaching into the ids
        assert call(name, good, **{out: C + 1}) == EALIGN
    assert call("ns_embed_lookup", LOOKUP, table=A + 1) == EALIGN
    assert call("ns_embed_lookup", LOOKUP, count=0, ids=None, out=None) == OK
    assert call("ns_embed_lookup", LOOKUP, table=None, vocab=0) == ENODEV  # every id is padding
    assert call("ns_embed_grad", GRAD, acc=2) == EINVAL
    assert call("ns_embed_grad", GRAD, gdtype=3) == EINVAL
    assert call("ns_embed_grad", GRAD, grad=C + 2) == EALIGN
    assert call("ns_embed_grad", GRAD, count=0, acc=1) == OK
    assert call("ns_embed_grad", GRAD, count=0, ids=None, dout=None) == ENODEV  # writes zeros


@NO_GPU
def test_policy_refusals(call):
    assert call("ns_token_logprobs", LOGP, it=0.0) == EINVAL
    assert call("ns_token_logprobs", LOGP, it=float("nan")) == EINVAL
    assert call("ns_token_logprobs", LOGP, logp=A + 16) == EINVAL
    assert call("ns_token_logprobs", LOGP, logp=C + 2) == EALIGN
    assert call("ns_token_logprobs", LOGP, rows=0, x=None, y=None, logp=None) == OK
    p = lambda **k: call("ns_policy_loss", POLICY, **k)  # noqa: E731
    assert p(old=None) == ENODEV and p(ref=None) == ENODEV and p(d=None) == ENODEV and p(d=A) == ENODEV
    for k in ("adv", "w", "logp", "kl", "loss", "x", "y"):
        assert p(**{k: None}) == EINVAL, k
    for k in ("lo", "hi", "beta", "it"):
        assert p(**{k: -0.1}) == EINVAL and p(**{k: float("inf")}) == EINVAL and p(**{k: float("nan")}) == EINVAL
    assert p(d=A + 2) == EINVAL          # over the logits, shifted
    assert p(d=A, ldd=101) == EINVAL     # over the logits with another pitch
    assert p(d=D + 1) == EALIGN
    assert p(logp=B + 12288 + 16) == EINVAL and p(kl=C + 4096 + 8) == EINVAL and p(loss=D + 4) == EINVAL
    assert p(rows=0, x=None, y=None, adv=None, w=None, logp=None, kl=None, d=None) == ENODEV  # writes the loss


@NO_GPU
def test_checkpoint_refusals(call):
    assert call("ns_ckpt_store", STORE, q=B + 8) == EALIGN
    assert call("ns_ckpt_store", STORE, s=C + 4) == EALIGN
    assert call("ns_ckpt_store", STORE, q=A + 64) == EINVAL
    assert call("ns_ckpt_store", STORE, s=B + 16) == EINVAL
    assert call("ns_ckpt_store", STORE, rows=0, x=None) == OK
    assert call("ns_ckpt_load", LOAD, out=B + 64) == EINVAL
    assert call("ns_ckpt_load", LOAD, out=None) == EINVAL
    assert call("ns_ckpt_load", LOAD, out=A + 1) == EALIGN
    f = lambda **k: call("ns_gated_forward", FORWARD, **k)  # noqa: E731
    assert f(h=A + 256) == EINVAL and f(qg=B) == EINVAL and f(su=D) == EINVAL and f(up=None) == EINVAL
    assert f(qu=D + 4) == EALIGN and f(gate=A + 1) == EALIGN and f(cols=0, h=None) == OK
    b = lambda **k: call("ns_gated_backward", BACKWARD, **k)  # noqa: E731
    assert b(h=None) == ENODEV
    assert b(du=B + 126) == EINVAL       # the halves overlap by one element
    assert b(du=B + 130) == EINVAL       # the right half reaches into the next row's left half
    assert b(du=B + 256 * 16) == ENODEV  # a matrix of its own
    assert b(dg=A) == EINVAL and b(h=B + 64) == EINVAL and b(dg=C) == EINVAL
    lib = api.load_library()
    lib.ns_ckpt_pitch.restype = lib.ns_ckpt_scale_pitch.restype = ctypes.c_int64
    lib.ns_ckpt_pitch.argtypes = lib.ns_ckpt_scale_pitch.argtypes = [ctypes.c_int64]
    for cols, pitch, scales in [(0, 0, 0), (1, 16, 4), (16, 16, 4), (33, 48, 4), (129, 144, 8), (-1, -1, -1)]:
        assert lib.ns_ckpt_pitch(cols) == pitch and lib.ns_ckpt_scale_pitch(cols) == scales


@NO_GPU
def test_wgrad_refusals(call):
    w = lambda **k: call("ns_ckpt_wgrad", WGRAD, **k)  # noqa: E731
    assert w(off=None) == EINVAL                    # two groups need offsets
    assert w(off=None, groups=1) == ENODEV
    assert w(groups=-1) == EINVAL and w(groups=0) == OK and w(acc=5) == EINVAL and w(gdtype=7) == EINVAL
    assert w(q=B + 4) == EALIGN and w(off=D + 2) == EALIGN and w(dy=A + 1) == EALIGN
    assert w(grad=A + 64) == EINVAL and w(grad=D - 64) == EINVAL and w(grad=None) == EINVAL and w(q=None) == EINVAL
    assert w(rows=0, dy=None, q=None, s=None) == ENODEV    # writes zeros
    assert w(rows=0, dy=None, q=None, s=None, acc=1) == OK
    assert w(n=1 << 22, k=1 << 22, ld=1 << 22) == EINVAL   # a stack beyond 2^42 elements


def test_python_layer_rejects_before_the_library():
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        api.embed_lookup(x, ids)                        # not on a GPU
    with pytest.raises(ValueError):
        api.embed_grad(x, ids, vocab=5)
    with pytest.raises(ValueError):
        api.checkpoint_store(torch.zeros(4))            # not a matrix
    with pytest.raises(ValueError):
        api.Checkpoint8(torch.zeros((4, 15), dtype=torch.int8), torch.zeros((4, 4), dtype=torch.uint8), 15)
    with pytest.raises(ValueError):
        api.Checkpoint8(torch.zeros((4, 16), dtype=torch.int8), torch.zeros((4, 4), dtype=torch.uint8), 16)  # CPU
    with pytest.raises(ValueError):
        api.token_logprobs(x, ids)


@NO_GPU
def test_sides_at_their_limits(call):
    # a row's columns are counted in 32 bits with room for what rounding up adds: at most 2^30 - 1 of them
    most, ld = (1 << 30) - 1, 1 << 30
    far = 1 << 44  # beyond what a row of that length spans
    lookup = lambda dim: call("ns_embed_lookup", LOOKUP, dim=dim, ld=ld, ldo=ld, vocab=2, count=2, ids=far, out=2 * far)  # noqa: E731
    assert lookup(most) == ENODEV and lookup(most + 1) == EINVAL
    logp = lambda v: call("ns_token_logprobs", LOGP, vocab=v, ld=ld, rows=2, y=far, logp=2 * far)  # noqa: E731
    assert logp(most) == ENODEV and logp(most + 1) == EINVAL
    away = {k: far + 4096 * i for i, k in enumerate(("y", "old", "ref", "adv", "w", "loss", "logp", "kl"))}
    loss = lambda v: call("ns_policy_loss", POLICY, vocab=v, ld=ld, ldd=ld, rows=2, d=2 * far, **away)  # noqa: E731
    assert loss(most) == ENODEV and loss(most + 1) == EINVAL
    # the pieces of the table's gradient: (count / 16 + 1) * (dim / 128 + 1) below 2^31, 2^42 values
    grad = lambda n, dim: call("ns_embed_grad", GRAD, count=n, dim=dim, ld=dim, ldg=dim, vocab=2, ids=far * 2, grad=far * 4)  # noqa: E731
    assert grad(1 << 30, 3840) == ENODEV and grad(1 << 30, 3968) == EINVAL and grad((1 << 30) + 1, 64) == EINVAL
    assert grad(1 << 20, 1 << 21) == ENODEV and grad(8, (1 << 24) + 1) == EINVAL


@NO_GPU
def test_columns_of_one_buffer_side_by_side(call):
    # matrices whose rows interleave in one buffer share no element: inputs and outputs may be columns of it
    def both(name, good, inside, outside):
        for change in inside:
            assert call(name, good, **change) == ENODEV, change
        for change in outside:
            assert call(name, good, **change) == EINVAL, change
    wide = dict(ld=256, ldo=256)  # rows of 64 bf16 values, 512 bytes apart
    both("ns_embed_lookup", LOOKUP, [dict(wide, out=A + 128), dict(wide, out=A + 384), dict(wide, out=A - 128), dict(wide, out=A + 5 * 512 + 128)],
         [dict(wide, out=A + 126), dict(wide, out=A + 386), dict(wide, out=A - 126), dict(wide, out=A + 5 * 512 + 126), dict(wide, out=A),
          dict(ld=256, ldo=128, out=A + 128)])
    wide = dict(ld=200, ldd=200)  # 100 values in 400 bytes
    both("ns_policy_loss", POLICY, [dict(wide, d=A + 200), dict(wide, d=A - 200)], [dict(wide, d=A + 198), dict(wide, d=A + 202)])
    wide = dict(ld=192, ldh=192)  # gate, up and h
    both("ns_gated_forward", FORWARD, [dict(wide, h=A + 256)], [dict(wide, h=A + 254), dict(wide, h=A + 258), dict(wide, h=A + 128)])
    wide = dict(ld=256, ldd=256, ldh=256, dh=B + 384)  # dgate, dup, h and dh
    both("ns_gated_backward", BACKWARD, [dict(wide, h=B + 256)], [dict(wide, h=B + 254), dict(wide, h=B + 258), dict(wide, h=B + 384)])
