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


def _function(name):
    f = _functions.get(name)
    if f is None:
        f = getattr(_api.load_library(), name)
        f.restype, f.argtypes = _i32, _PROTOTYPES[name]
        _functions[name] = f
    return f


def _call(name, *args) -> None:
    rc = _function(name)(*args)
    if rc != 0:
        raise _api.NSError(rc, name)


class _On:
    """The device and stream of a call, current inside the ``with`` block when
    they are not already (so that what it allocates belongs to that stream)."""

    __slots__ = ("ptr", "_stack")

    def __init__(self, device, stream):
        self._stack = None
        if stream is not None or device.index != torch.cuda.current_device():
            self._stack = contextlib.ExitStack()
            self._stack.enter_context(torch.cuda.device(device))
            if stream is not None:
                self._stack.enter_context(torch.cuda.stream(stream))
        self.ptr = torch.cuda.current_stream(device).cuda_stream

    def __enter__(self):
        return self.ptr

    def __exit__(self, *exc):
        if self._stack is not None:
            self._stack.close()
        return False


def _matrix(t, what, rows=None, cols=None, dtype=None):
    """The row pitch of a 2-D CUDA tensor of a supported type, checked."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D")
    if t.device.type != "cuda":
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}: use float32 or bfloat16")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, is {t.dtype}")
    n, m = t.shape
    if (rows is not None and n != rows) or (cols is not None and m != cols):
        raise ValueError(f"{what} must be {rows if rows is not None else n} x {cols if cols is not None else m}, "
                         f"is {n} x {m}")
    if n == 0 or m == 0:
        return m
    s0, s1 = t.stride()
    if m > 1 and s1 != 1:
        raise ValueError(f"{what} must have unit column stride")
    if n == 1:
        return m
    if s0 < m:
        raise ValueError(f"{what}: rows must not overlap")
    return s0


def _vector(t, what, n, dtypes, device):
    if t.dim() != 1 or t.shape[0] != n:
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
def embed_lookup(table, ids, scale: float = 1.0, out=None, stream=None):
    """``out[t] = scale * table[ids[t]]`` (ns_embed_lookup). ``table`` is vocab x
    dim; ``ids`` an int32 or int64 tensor of any shape. Ids outside the
    vocabulary are padding: a zero row. Returns ``out``, shaped as ids plus
    dim (given: 2-D, one row per id)."""
    ld = _matrix(table, "table")
    vocab, dim = table.shape
    flat = ids.reshape(-1)
    n = flat.shape[0]
    p_ids = _vector(flat, "ids", n, _IDTYPE, table.device)
    with _On(table.device, stream) as s:
        if out is None:
            res = torch.empty((*ids.shape, dim), dtype=table.dtype, device=table.device)
            p_out, ld_out = res.data_ptr(), dim
        else:
            _same_device(table.device, out)
            res, p_out, ld_out = out, out.data_ptr(), _matrix(out, "out", n, dim, table.dtype)
        _call("ns_embed_lookup", table.data_ptr(), ld, vocab, dim, p_ids, _IDTYPE[flat.dtype], n, scale, p_out, ld_out,
              _DTYPE[table.dtype], s)
    return res


def embed_grad(dout, ids, vocab: int | None = None, scale: float = 1.0, grad=None, accumulate: bool = False,
               dtype=None, stream=None):
    """Gradient of embed_lookup's table (ns_embed_grad): row v of ``grad`` is
    ``scale`` times the sum of the rows of ``dout`` whose id is v, or has it
    added with ``accumulate``. ``dout`` is 2-D, one row per id. ``grad`` (vocab x
    dim, float32 or bfloat16) is allocated when not given, of ``dtype``
    (default: dout's). Deterministic; returns ``grad``."""
    ld = _matrix(dout, "dout")
    n, dim = dout.shape
    flat = ids.reshape(-1)
    p_ids = _vector(flat, "ids", n, _IDTYPE, dout.device)
    if grad is None:
        if accumulate or vocab is None:
            raise ValueError("without grad, give vocab and do not accumulate")
    else:
        if vocab is not None and vocab != grad.shape[0]:
            raise ValueError("grad has another number of rows than vocab")
        _same_device(dout.device, grad)
        ld_grad = _matrix(grad, "grad", None, dim, dtype)
    with _On(dout.device, stream) as s:
        if grad is None:
            grad = torch.empty((int(vocab), dim), dtype=dtype or dout.dtype, device=dout.device)
            ld_grad = _matrix(grad, "grad")
        _call("ns_embed_grad", dout.data_ptr(), ld, p_ids, _IDTYPE[flat.dtype], n, scale, grad.data_ptr(), ld_grad,
              grad.shape[0], dim, _DTYPE[dout.dtype], _DTYPE[grad.dtype], 1 if accumulate else 0, s)
    return grad


# ------------------------------------------------------------------ policy loss
def token_logprobs(logits, targets, temperature: float = 1.0, stream=None):
    """Log probabilities of the target tokens under logits / temperature
    (ns_token_logprobs), float32. ``logits`` is rows x vocab; a row whose
    target is outside the vocabulary (e.g. -100) is masked and gives 0."""
    ld = _matrix(logits, "logits")
    n, vocab = logits.shape
    p_y = _vector(targets, "targets", n, _IDTYPE, logits.device)
    if not temperature > 0:
        raise ValueError("temperature must be positive")
    with _On(logits.device, stream) as s:
        logp = torch.empty(n, dtype=torch.float32, device=logits.device)
        _call("ns_token_logprobs", logits.data_ptr(), ld, n, vocab, p_y, _IDTYPE[targets.dtype], 1.0 / temperature,
              logp.data_ptr(), _DTYPE[logits.dtype], s)
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
    the vocabulary or whose weight is 0 are masked. ``dlogits`` is where the
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
    with _On(dev, stream) as s:
        if grad and dlogits is None:
            dlogits = torch.empty((n, vocab), dtype=logits.dtype, device=dev)
        out = torch.empty(2 * n + 1, dtype=torch.float32, device=dev)
        p = out.data_ptr()
        _call("ns_policy_loss", logits.data_ptr(), ld, n, vocab, p_y, _IDTYPE[targets.dtype], p_old, p_ref, p_adv, p_w,
              1.0 / temperature, clip_low, clip_high, kl_coef, p + 8 * n, p, p + 4 * n,
              dlogits.data_ptr() if grad else None, _matrix(dlogits, "dlogits") if grad else 0, _DTYPE[logits.dtype], s)
    return PolicyLoss(out[2 * n], out[:n], out[n:2 * n], dlogits)


# ------------------------------------------------------------------ 8-bit activations
def _ceil(n, m):
    return (n + m - 1) // m * m


class Checkpoint8:
    """A rows x cols matrix held in 8 bits: ``q`` (int8, rows x cols rounded up to
    16) and ``scales`` (uint8, one per 32 values, rounded up to 4 a row). The
    format is described at ns_ckpt_store in include/ns.h."""

    __slots__ = ("q", "scales", "rows", "cols")

    def __init__(self, q, scales, cols: int):
        rows = q.shape[0]
        if q.dtype != torch.int8 or q.shape != (rows, _ceil(cols, 16)) or not q.is_contiguous():
            raise ValueError(f"q must be contiguous int8, {rows} x {_ceil(cols, 16)}")
        if (scales.dtype != torch.uint8 or scales.shape != (rows, _ceil((cols + 31) // 32, 4))
                or not scales.is_contiguous()):
            raise ValueError(f"scales must be contiguous uint8, {rows} x {_ceil((cols + 31) // 32, 4)}")
        if q.device.type != "cuda" or scales.device != q.device:
            raise ValueError("q and scales must be CUDA tensors on one device")
        self.q, self.scales, self.rows, self.cols = q, scales, rows, cols

    @classmethod
    def empty(cls, rows: int, cols: int, device):
        return cls(torch.empty((rows, _ceil(cols, 16)), dtype=torch.int8, device=device),
                   torch.empty((rows, _ceil((cols + 31) // 32, 4)), dtype=torch.uint8, device=device), cols)

    @property
    def device(self):
        return self.q.device

    def nbytes(self) -> int:
        return self.q.numel() + self.scales.numel()


def checkpoint_store(x, stream=None) -> Checkpoint8:
    """Hold a 2-D tensor in 8 bits (ns_ckpt_store)."""
    ld = _matrix(x, "x")
    rows, cols = x.shape
    with _On(x.device, stream) as s:
        ck = Checkpoint8.empty(rows, cols, x.device)
        _call("ns_ckpt_store", x.data_ptr(), ld, rows, cols, ck.q.data_ptr(), ck.scales.data_ptr(), _DTYPE[x.dtype], s)
    return ck


def checkpoint_load(ck: Checkpoint8, dtype=torch.bfloat16, out=None, stream=None):
    """The values that a checkpoint holds (ns_ckpt_load)."""
    if out is not None:
        _same_device(ck.device, out)
        _matrix(out, "out", ck.rows, ck.cols)
    elif dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype}: use float32 or bfloat16")
    with _On(ck.device, stream) as s:
        if out is None:
            out = torch.empty((ck.rows, ck.cols), dtype=dtype, device=ck.device)
        _call("ns_ckpt_load", ck.q.data_ptr(), ck.scales.data_ptr(), ck.rows, ck.cols, out.data_ptr(),
              _matrix(out, "out"), _DTYPE[out.dtype], s)
    return out


def gated_forward(gate, up, out=None, stream=None):
    """``h = silu(gate) * up`` with gate and up held in 8 bits for
    gated_backward (ns_gated_forward). gate and up have one shape, type and
    row stride (the two halves of one matrix, or two matrices). Returns (h,
    checkpoint of gate, checkpoint of up)."""
    ld = _matrix(gate, "gate")
    rows, cols = gate.shape
    ld_up = _matrix(up, "up", rows, cols, gate.dtype)
    _same_device(gate.device, up, out)
    if ld_up != ld:
        raise ValueError("gate and up must have the same row stride")
    with _On(gate.device, stream) as s:
        if out is None:
            out = torch.empty((rows, cols), dtype=gate.dtype, device=gate.device)
        a, b = Checkpoint8.empty(rows, cols, gate.device), Checkpoint8.empty(rows, cols, gate.device)
        _call("ns_gated_forward", gate.data_ptr(), up.data_ptr(), ld, rows, cols, out.data_ptr(),
              _matrix(out, "out", rows, cols, gate.dtype), a.q.data_ptr(), a.scales.data_ptr(), b.q.data_ptr(),
              b.scales.data_ptr(), _DTYPE[gate.dtype], s)
    return out, a, b


def gated_backward(dh, ck_gate: Checkpoint8, ck_up: Checkpoint8, recompute: bool = True, dgu=None, stream=None):
    """Backward of gated_forward from the 8-bit values (ns_gated_backward).
    Returns (dgu, h): dgu is rows x 2 cols, the gradient of gate in its left
    half and of up in its right one (given or allocated); h is silu(gate) * up
    again, the input of the next layer's weight gradient (None unless
    ``recompute``)."""
    rows, cols = ck_gate.rows, ck_gate.cols
    ld = _matrix(dh, "dh", rows, cols)
    if (ck_up.rows, ck_up.cols) != (rows, cols):
        raise ValueError("the checkpoints of gate and up must have one shape")
    _same_device(dh.device, ck_gate, ck_up, dgu)
    if dgu is not None:
        _matrix(dgu, "dgu", rows, 2 * cols, dh.dtype)
    with _On(dh.device, stream) as s:
        if dgu is None:
            dgu = torch.empty((rows, 2 * cols), dtype=dh.dtype, device=dh.device)
        h = torch.empty((rows, cols), dtype=dh.dtype, device=dh.device) if recompute else None
        p = dgu.data_ptr()
        _call("ns_gated_backward", dh.data_ptr(), ld, ck_gate.q.data_ptr(), ck_gate.scales.data_ptr(),
              ck_up.q.data_ptr(), ck_up.scales.data_ptr(), rows, cols, p, p + cols * dgu.element_size(),
              _matrix(dgu, "dgu"), h.data_ptr() if recompute else None, cols, _DTYPE[dh.dtype], s)
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
    _same_device(dy.device, ck, offsets, grad)
    groups = 1
    p_off = None
    if offsets is not None:
        groups = offsets.shape[0] - 1
        if groups < 0:
            raise ValueError("offsets must have at least one entry")
        p_off = _vector(offsets, "offsets", groups + 1, (torch.int32,), dy.device)
    if grad is None:
        if accumulate:
            raise ValueError("accumulate needs grad")
        if dtype is not None and dtype not in _DTYPE:
            raise TypeError(f"unsupported dtype {dtype}: use float32 or bfloat16")
    else:
        if grad.shape != (groups, n_out, ck.cols) or not grad.is_contiguous():
            raise ValueError(f"grad must be contiguous, {groups} x {n_out} x {ck.cols}")
        if grad.dtype not in _DTYPE or (dtype is not None and grad.dtype != dtype):
            raise TypeError(f"grad: unsupported dtype {grad.dtype}")
    with _On(dy.device, stream) as s:
        if grad is None:
            grad = torch.empty((groups, n_out, ck.cols), dtype=dtype or dy.dtype, device=dy.device)
        _call("ns_ckpt_wgrad", dy.data_ptr(), ld, rows, n_out, ck.q.data_ptr(), ck.scales.data_ptr(), ck.cols, p_off,
              groups, grad.data_ptr(), _DTYPE[dy.dtype], _DTYPE[grad.dtype], 1 if accumulate else 0, s)
    return grad
