"""Operators of the training step around the optimizer (C ABI in include/ns.h):
the token embedding and its gradient, the clipped policy loss on logits,
activations held for the backward pass in 8 bits, and the weight gradients
formed from them, which are the matrices ``muon_update_batched`` takes.

As in ``api``: argument checks and marshalling only, every computation runs in
the library's kernels, calls are ordered on ``stream`` (default: torch's
current stream on the tensors' device) and do not synchronise. Matrices are
2-D CUDA tensors with unit column stride and any row stride. Outputs that a
call allocates belong to the stream it runs on.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

import torch

from . import api as _api

_DTYPE = {torch.float32: 0, torch.bfloat16: 1}
_IDTYPE = {torch.int32: 0, torch.int64: 1}

_vp, _i64, _i32, _f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_PROTOTYPES = {
    "ns_embed_lookup": [_vp, _i64, _i64, _i64, _vp, _i32, _i64, _f, _vp, _i64, _i32, _vp],
    "ns_embed_grad": [_vp, _i64, _vp, _i32, _i64, _f, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _vp],
    "ns_token_logprobs": [_vp, _i64, _i64, _i64, _vp, _i32, _f, _vp, _i32, _vp],
    "ns_policy_loss": [_vp, _i64, _i64, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _f, _f, _f, _f, _vp, _vp, _vp, _vp, _i64,
                       _i32, _vp],
    "ns_ckpt_store": [_vp, _i64, _i64, _i64, _vp, _vp, _i32, _vp],
    "ns_ckpt_load": [_vp, _vp, _i64, _i64, _vp, _i64, _i32, _vp],
    "ns_gated_forward": [_vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _vp],
    "ns_gated_backward": [_vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _i32, _vp],
    "ns_ckpt_wgrad": [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _vp, _i32, _i32, _i32, _vp],
}
_functions: dict = {}

# These calls are short: what Python spends around a kernel counts. The raw
# handle of the current stream is had without making a Stream object where
# torch offers that.
_current_device = torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_empty = torch.empty


def _function(name):
    f = getattr(_api.load_library(), name)
    f.restype, f.argtypes = _i32, _PROTOTYPES[name]
    _functions[name] = f
    return f


def _call(name, *args) -> None:
    rc = (_functions.get(name) or _function(name))(*args)
    if rc != 0:
        raise _api.NSError(rc, name)


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """The block in which ``device`` and ``stream`` are torch's current ones, so
    that what a call allocates belongs to the stream it runs on; inside it
    _raw_stream(device.index) is the stream's handle."""
    if stream is None and device.index == _current_device():
        return _HERE
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(device))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(stream))
    return stack


def _matrix(t, what, rows=None, cols=None, dtype=None):
    """The row pitch of a 2-D CUDA tensor of a supported type, checked."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    kind = t.dtype
    if kind not in _DTYPE:
        raise TypeError(f"{what}: unsupported dtype {kind}: use float32 or bfloat16")
    if dtype is not None and kind != dtype:
        raise ValueError(f"{what} must be {dtype}, is {kind}")
    n, m = shape
    if (rows is not None and n != rows) or (cols is not None and m != cols):
        raise ValueError(f"{what} must be {rows if rows is not None else n} x {cols if cols is not None else m}, "
                         f"is {n} x {m}")
    s0, s1 = t.stride()
    if s1 != 1 and m > 1 and n > 0:
        raise ValueError(f"{what} must have unit column stride")
    if n <= 1 or m == 0:
        return m
    if s0 < m:
        raise ValueError(f"{what}: rows must not overlap")
    return s0


def _vector(t, what, n, dtypes, device):
    if t.shape != (n,):
        raise ValueError(f"{what} must be 1-D of length {n}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _same_device(device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("all tensors must be on one device")


# ------------------------------------------------------------------ embedding
def _flat(ids):
    """``ids`` in one dimension. For a view that is not contiguous this is a copy
    by a kernel of its own: made inside _on's block, it runs on the call's
    stream before the call's kernels, and its memory belongs to that stream."""
    return ids if ids.dim() == 1 else ids.reshape(-1)


def embed_lookup(table, ids, scale: float = 1.0, out=None, stream=None):
    """``out[t] = scale * table[ids[t]]`` (ns_embed_lookup). ``table`` is vocab x
    dim; ``ids`` an int32 or int64 tensor of any shape. Ids outside the
    vocabulary are padding: a zero row. Returns ``out``, shaped as ids plus
    dim (given: 2-D, one row per id)."""
    ld = _matrix(table, "table")
    vocab, dim = table.shape
    dev, dt = table.device, table.dtype
    n = ids.numel()
    with _on(dev, stream):
        flat = _flat(ids)
        p_ids = _vector(flat, "ids", n, _IDTYPE, dev)
        if out is None:
            out, ld_out = _empty((*ids.shape, dim), dtype=dt, device=dev), dim
        else:
            _same_device(dev, out)
            ld_out = _matrix(out, "out", n, dim, dt)
        _call("ns_embed_lookup", table.data_ptr(), ld, vocab, dim, p_ids, _IDTYPE[flat.dtype], n, scale, out.data_ptr(),
              ld_out, _DTYPE[dt], _raw_stream(dev.index))
    return out


def embed_grad(dout, ids, vocab: int | None = None, scale: float = 1.0, grad=None, accumulate: bool = False,
               dtype=None, stream=None):
    """Gradient of embed_lookup's table (ns_embed_grad): row v of ``grad`` is
    ``scale`` times the sum of the rows of ``dout`` whose id is v, or has it
    added with ``accumulate``. ``dout`` is 2-D, one row per id. ``grad`` (vocab x
    dim, float32 or bfloat16) is allocated when not given, of ``dtype``
    (default: dout's). Deterministic; returns ``grad``."""
    ld = _matrix(dout, "dout")
    n, dim = dout.shape
    dev = dout.device
    if grad is None:
        if accumulate or vocab is None:
            raise ValueError("without grad, give vocab and do not accumulate")
    else:
        if vocab is not None and vocab != grad.shape[0]:
            raise ValueError("grad has another number of rows than vocab")
        _same_device(dev, grad)
        ld_grad = _matrix(grad, "grad", None, dim, dtype)
    with _on(dev, stream):
        flat = _flat(ids)
        p_ids = _vector(flat, "ids", n, _IDTYPE, dev)
        if grad is None:
            grad = _empty((int(vocab), dim), dtype=dtype or dout.dtype, device=dev)
            ld_grad = _matrix(grad, "grad")
        _call("ns_embed_grad", dout.data_ptr(), ld, p_ids, _IDTYPE[flat.dtype], n, scale, grad.data_ptr(), ld_grad,
              grad.shape[0], dim, _DTYPE[dout.dtype], _DTYPE[grad.dtype], 1 if accumulate else 0,
              _raw_stream(dev.index))
    return grad


# ------------------------------------------------------------------ policy loss
def token_logprobs(logits, targets, temperature: float = 1.0, stream=None):
    """Log probabilities of the target tokens under logits / temperature
    (ns_token_logprobs), float32. ``logits`` is rows x vocab; a row whose
    target is outside the vocabulary (e.g. -100) is masked and gives 0."""
    ld = _matrix(logits, "logits")
    n, vocab = logits.shape
    dev = logits.device
    p_y = _vector(targets, "targets", n, _IDTYPE, dev)
    if not temperature > 0:
        raise ValueError("temperature must be positive")
    with _on(dev, stream):
        logp = _empty(n, dtype=torch.float32, device=dev)
        _call("ns_token_logprobs", logits.data_ptr(), ld, n, vocab, p_y, _IDTYPE[targets.dtype], 1.0 / temperature,
              logp.data_ptr(), _DTYPE[logits.dtype], _raw_stream(dev.index))
    return logp


class PolicyLoss(NamedTuple):
    loss: torch.Tensor      # scalar, float32
    logp: torch.Tensor      # per row, float32 (0 where masked)
    kl: torch.Tensor        # per row, float32 (0 where masked or without reference)
    dlogits: torch.Tensor | None


_F32 = (torch.float32,)


def policy_loss(logits, targets, advantages, weights, old_logp=None, ref_logp=None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0, dlogits=None,
                grad: bool = True, stream=None) -> PolicyLoss:
    """Clipped policy loss with a KL term and the gradient of the logits, in one
    pass (ns_policy_loss): the sum over rows of weights * (kl_coef * k - min(r A,
    clip(r, 1 - clip_low, 1 + clip_high) A)), r = exp(logp - old_logp), k =
    exp(ref_logp - logp) - (ref_logp - logp) - 1. Rows whose target is outside
    the vocabulary or whose weight is 0 are masked; a NaN of any other row reaches
    the loss. With ``kl_coef`` 0 the KL term is only returned, whatever it is.
    ``dlogits`` is where the
    gradient goes; it may be ``logits`` itself; allocated when not given;
    ``grad=False`` computes none."""
    ld = _matrix(logits, "logits")
    n, vocab = logits.shape
    dev = logits.device
    p_y = _vector(targets, "targets", n, _IDTYPE, dev)
    p_adv = _vector(advantages, "advantages", n, _F32, dev)
    p_w = _vector(weights, "weights", n, _F32, dev)
    p_old = _vector(old_logp, "old_logp", n, _F32, dev) if old_logp is not None else None
    p_ref = _vector(ref_logp, "ref_logp", n, _F32, dev) if ref_logp is not None else None
    if not temperature > 0:
        raise ValueError("temperature must be positive")
    if dlogits is not None:
        if not grad:
            raise ValueError("dlogits given, but grad is False")
        _same_device(dev, dlogits)
        _matrix(dlogits, "dlogits", n, vocab, logits.dtype)
    with _on(dev, stream):
        if grad and dlogits is None:
            dlogits = _empty((n, vocab), dtype=logits.dtype, device=dev)
        loss = _empty((), dtype=torch.float32, device=dev)
        logp = _empty(n, dtype=torch.float32, device=dev)
        kl = _empty(n, dtype=torch.float32, device=dev)
        _call("ns_policy_loss", logits.data_ptr(), ld, n, vocab, p_y, _IDTYPE[targets.dtype], p_old, p_ref, p_adv, p_w,
              1.0 / temperature, clip_low, clip_high, kl_coef, loss.data_ptr(), logp.data_ptr(), kl.data_ptr(),
              dlogits.data_ptr() if grad else None, _matrix(dlogits, "dlogits") if grad else 0, _DTYPE[logits.dtype],
              _raw_stream(dev.index))
    return PolicyLoss(loss, logp, kl, dlogits)


# ------------------------------------------------------------------ 8-bit activations
def _pitch(cols):
    return (cols + 15) // 16 * 16


def _scale_pitch(cols):
    return (cols + 127) // 128 * 4


class Checkpoint8:
    """A rows x cols matrix held in 8 bits: ``q`` (int8, rows x cols rounded up to
    16) and ``scales`` (uint8, one per 32 values, rounded up to 4 a row). The
    format is described at ns_ckpt_store in include/ns.h."""

    __slots__ = ("rows", "cols", "device", "_q", "_scales", "_buffer", "_at", "_p_q", "_p_scales")

    def __init__(self, q, scales, cols: int):
        rows = q.shape[0]
        if q.dtype != torch.int8 or q.shape != (rows, _pitch(cols)) or not q.is_contiguous():
            raise ValueError(f"q must be contiguous int8, {rows} x {_pitch(cols)}")
        if scales.dtype != torch.uint8 or scales.shape != (rows, _scale_pitch(cols)) or not scales.is_contiguous():
            raise ValueError(f"scales must be contiguous uint8, {rows} x {_scale_pitch(cols)}")
        if not q.is_cuda or scales.device != q.device:
            raise ValueError("q and scales must be CUDA tensors on one device")
        self.rows, self.cols, self.device = rows, cols, q.device
        self._q, self._scales, self._buffer = q, scales, None
        self._p_q, self._p_scales = q.data_ptr(), scales.data_ptr()

    @classmethod
    def empty(cls, rows: int, cols: int, device):
        """Room for a matrix, in one allocation, uninitialised, on a CUDA device."""
        if not isinstance(device, torch.device):
            device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        if device.type != "cuda":
            raise ValueError("a checkpoint must be on a CUDA device")
        if device.index is None:
            device = torch.device("cuda", _current_device())
        return cls._empties(1, rows, cols, device)[0]

    @classmethod
    def _empties(cls, count, rows, cols, device):
        # `count` of them in one allocation, which lives until the last is dropped
        nq = rows * _pitch(cols)
        each = (nq + rows * _scale_pitch(cols) + 15) // 16 * 16
        buffer = _empty(count * each, dtype=torch.uint8, device=device)
        p = buffer.data_ptr()
        made = []
        for k in range(count):
            self = cls.__new__(cls)
            self.rows, self.cols, self.device = rows, cols, device
            self._q = self._scales = None  # views of the buffer, made when asked for
            self._buffer, self._at = buffer, k * each
            self._p_q = p + k * each
            self._p_scales = self._p_q + nq
            made.append(self)
        return made

    @property
    def q(self):
        if self._q is None:
            n, pitch = self.rows, _pitch(self.cols)
            self._q = self._buffer[self._at:self._at + n * pitch].view(torch.int8).view(n, pitch)
        return self._q

    @property
    def scales(self):
        if self._scales is None:
            n, pitch = self.rows, _scale_pitch(self.cols)
            at = self._at + n * _pitch(self.cols)
            self._scales = self._buffer[at:at + n * pitch].view(n, pitch)
        return self._scales

    def nbytes(self) -> int:
        return self.rows * (_pitch(self.cols) + _scale_pitch(self.cols))


def checkpoint_store(x, stream=None) -> Checkpoint8:
    """Hold a 2-D tensor in 8 bits (ns_ckpt_store)."""
    ld = _matrix(x, "x")
    rows, cols = x.shape
    dev = x.device
    with _on(dev, stream):
        ck, = Checkpoint8._empties(1, rows, cols, dev)
        _call("ns_ckpt_store", x.data_ptr(), ld, rows, cols, ck._p_q, ck._p_scales, _DTYPE[x.dtype],
              _raw_stream(dev.index))
    return ck


def checkpoint_load(ck: Checkpoint8, dtype=torch.bfloat16, out=None, stream=None):
    """The values that a checkpoint holds (ns_ckpt_load)."""
    dev = ck.device
    ld = ck.cols
    if out is not None:
        _same_device(dev, out)
        ld = _matrix(out, "out", ck.rows, ck.cols)
    elif dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype}: use float32 or bfloat16")
    with _on(dev, stream):
        if out is None:
            out = _empty((ck.rows, ck.cols), dtype=dtype, device=dev)
        _call("ns_ckpt_load", ck._p_q, ck._p_scales, ck.rows, ck.cols, out.data_ptr(), ld, _DTYPE[out.dtype],
              _raw_stream(dev.index))
    return out


def gated_forward(gate, up, out=None, stream=None):
    """``h = silu(gate) * up`` with gate and up held in 8 bits for
    gated_backward (ns_gated_forward). gate and up have one shape, type and
    row stride (the two halves of one matrix, or two matrices). Returns (h,
    checkpoint of gate, checkpoint of up)."""
    ld = _matrix(gate, "gate")
    rows, cols = gate.shape
    dev, dt = gate.device, gate.dtype
    if _matrix(up, "up", rows, cols, dt) != ld:
        raise ValueError("gate and up must have the same row stride")
    _same_device(dev, up, out)
    ld_out = cols if out is None else _matrix(out, "out", rows, cols, dt)
    with _on(dev, stream):
        if out is None:
            out = _empty((rows, cols), dtype=dt, device=dev)
        a, b = Checkpoint8._empties(2, rows, cols, dev)
        _call("ns_gated_forward", gate.data_ptr(), up.data_ptr(), ld, rows, cols, out.data_ptr(), ld_out, a._p_q,
              a._p_scales, b._p_q, b._p_scales, _DTYPE[dt], _raw_stream(dev.index))
    return out, a, b


def gated_backward(dh, ck_gate: Checkpoint8, ck_up: Checkpoint8, recompute: bool = True, dgu=None, stream=None):
    """Backward of gated_forward from the 8-bit values (ns_gated_backward).
    Returns (dgu, h): dgu is rows x 2 cols, the gradient of gate in its left
    half and of up in its right one (given or allocated); h is silu(gate) * up
    again, the input of the next layer's weight gradient (None unless
    ``recompute``)."""
    rows, cols = ck_gate.rows, ck_gate.cols
    dev, dt = dh.device, dh.dtype
    ld = _matrix(dh, "dh", rows, cols)
    if ck_up.rows != rows or ck_up.cols != cols:
        raise ValueError("the checkpoints of gate and up must have one shape")
    _same_device(dev, ck_gate, ck_up, dgu)
    ld_d = 2 * cols if dgu is None else _matrix(dgu, "dgu", rows, 2 * cols, dt)
    code = _DTYPE[dt]
    with _on(dev, stream):
        if dgu is None:
            dgu = _empty((rows, 2 * cols), dtype=dt, device=dev)
        h = _empty((rows, cols), dtype=dt, device=dev) if recompute else None
        p = dgu.data_ptr()
        _call("ns_gated_backward", dh.data_ptr(), ld, ck_gate._p_q, ck_gate._p_scales, ck_up._p_q, ck_up._p_scales,
              rows, cols, p, p + cols * (2 if code else 4), ld_d, h.data_ptr() if recompute else None, cols, code,
              _raw_stream(dev.index))
    return dgu, h


def checkpoint_wgrad(dy, ck: Checkpoint8, offsets=None, grad=None, accumulate: bool = False, dtype=None, stream=None):
    """Weight gradients from an input held in 8 bits (ns_ckpt_wgrad): G[e] =
    dy[rows of e]^T @ (values of ck)[rows of e], n_out x n_in, or added to G[e]
    with ``accumulate``. ``offsets`` (int32, on the device, groups + 1 ascending
    row numbers) gives each group of a stack its rows; without it there is one
    group. ``grad`` is groups x n_out x n_in, contiguous, float32 or bfloat16;
    allocated when not given, of ``dtype`` (default: dy's). Returns ``grad``: its
    matrices are what muon_update_batched takes."""
    ld = _matrix(dy, "dy", ck.rows)
    rows, n_out = dy.shape
    dev, dt = dy.device, dy.dtype
    _same_device(dev, ck, offsets, grad)
    groups = 1
    p_off = None
    if offsets is not None:
        groups = offsets.shape[0] - 1
        if groups < 0:
            raise ValueError("offsets must have at least one entry")
        p_off = _vector(offsets, "offsets", groups + 1, (torch.int32,), dev)
    if grad is None:
        if accumulate:
            raise ValueError("accumulate needs grad")
        if dtype is None:
            dtype = dt
        elif dtype not in _DTYPE:
            raise TypeError(f"unsupported dtype {dtype}: use float32 or bfloat16")
    else:
        if grad.shape != (groups, n_out, ck.cols) or not grad.is_contiguous():
            raise ValueError(f"grad must be contiguous, {groups} x {n_out} x {ck.cols}")
        if grad.dtype not in _DTYPE or (dtype is not None and grad.dtype != dtype):
            raise TypeError(f"grad: unsupported dtype {grad.dtype}")
        dtype = grad.dtype
    with _on(dev, stream):
        if grad is None:
            grad = _empty((groups, n_out, ck.cols), dtype=dtype, device=dev)
        _call("ns_ckpt_wgrad", dy.data_ptr(), ld, rows, n_out, ck._p_q, ck._p_scales, ck.cols, p_off, groups,
              grad.data_ptr(), _DTYPE[dt], _DTYPE[dtype], 1 if accumulate else 0, _raw_stream(dev.index))
    return grad
