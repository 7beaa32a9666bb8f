"""Operators of an expert layer in a training step (C ABI in include/ns.h): the
router with its balance loss, matrices held in 8-bit floating point with a
scale for each block of 128 and their product over a stack of experts, the norms
around a block fused with its gate and residual scale, and dropout whose mask is
never stored.

As in ``training``: argument checks and marshalling only, every computation
runs in the library's kernels, calls are ordered on ``stream`` (default: torch's
current stream on the tensors' device) and do not synchronise. Matrices are 2-D
CUDA tensors with unit column stride and any row stride. What a call allocates,
scratch included, belongs to the stream it runs on.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .training import _DTYPE, _PROTOTYPES, _call, _matrix, _on, _raw_stream, _same_device, _vector

_vp, _i64, _i32, _f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_u64, _size, _d = ctypes.c_uint64, ctypes.c_size_t, ctypes.c_double
_PROTOTYPES.update({
    "ns_route": [_vp, _i64, _i64, _i32, _i32, _vp, _i32, _f, _f, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _size, _i32, _vp],
    "ns_route_backward": [_vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _f, _f, _vp, _i64, _i32, _vp],
    "ns_blocks_store_rows": [_vp, _i64, _i64, _vp, _i32, _i64, _i64, _vp, _vp, _i32, _vp],
    "ns_blocks_store_tiles": [_vp, _i64, _i32, _i64, _i64, _vp, _vp, _i32, _vp],
    "ns_blocks_load": [_vp, _vp, _i32, _i32, _i64, _i64, _vp, _i64, _i32, _vp],
    "ns_blocks_matmul": [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _i32, _vp, _i64, _i32, _vp],
    "ns_block_norm": [_vp, _i64, _vp, _i64, _vp, _i32, _i64, _vp, _vp, _i64, _i64, _f, _f, _f, _vp, _i64, _vp, _i64, _vp, _vp,
                      _i32, _i32, _i32, _i32, _vp],
    "ns_block_norm_backward": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _f,
                               _f, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _size, _i32, _i32, _i32, _i32, _vp],
    "ns_dropout": [_vp, _i64, _vp, _i64, _i64, _i64, _d, _u64, _u64, _vp, _vp, _i64, _i32, _i32, _vp],
})
_empty = torch.empty
_F32, _I32 = torch.float32, torch.int32


def _ptr(t):
    return None if t is None else t.data_ptr()


def _contiguous(t, what, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {dtype} of shape {tuple(shape)} on {device}")
    return t.data_ptr()


# ------------------------------------------------------------------ router
class Routing(NamedTuple):
    experts: torch.Tensor    # rows x top_k int32, largest logit first; -1: none
    weights: torch.Tensor    # rows x top_k float32, 0 where none
    counts: torch.Tensor     # experts, int32
    offsets: torch.Tensor    # experts + 1, int32: their running sum
    order: torch.Tensor      # rows * top_k int32: slots (row * top_k + place) in the experts' order, then -1
    loss: torch.Tensor       # scalar, float32
    logz: torch.Tensor       # per row, float32 (0 for padding)
    live_rows: torch.Tensor  # scalar, int32: rows that are not padding


_MAX_STRETCHES = 152   # of a route call
_MAX_PARTS = 304       # of a block_norm_backward call


def route(logits, top_k: int, live=None, renormalise: bool = True, balance_coef: float = 0.0, z_coef: float = 0.0,
          stream=None) -> Routing:
    """The router (ns_route): the ``top_k`` experts of every row of ``logits``
    (rows x experts), ties to the lower index, with their softmax weights
    (``renormalise``: divided by their sum), counts per expert, the slots in the
    experts' order, and the loss ``balance_coef`` * balance + ``z_coef`` * mean
    logz^2. ``live`` (bool, one per row) marks padding with False: such rows are
    not looked at. ``offsets`` is what blocks_matmul and checkpoint_wgrad take,
    ``order`` what blocks_store(rows=order, per=top_k) takes."""
    ld = _matrix(logits, "logits")
    n, experts = logits.shape
    dev = logits.device
    top_k = int(top_k)
    if not 1 <= top_k <= experts:
        raise ValueError("top_k must be between 1 and the number of experts")
    p_live = None if live is None else _vector(live, "live", n, (torch.bool,), dev)
    slots = n * top_k
    # everything in one allocation: ids, order, counts, offsets, live rows | weights, logz, loss | scratch
    at_f = 2 * slots + 2 * experts + 2
    at_work = at_f + slots + n + 1
    scratch = max(1, min(-(-n // 16), _MAX_STRETCHES)) * (2 * experts + 2)
    with _on(dev, stream):
        floats = _empty(at_work + scratch, dtype=_F32, device=dev)
        p = floats.data_ptr()
        _call("ns_route", logits.data_ptr(), ld, n, experts, top_k, p_live, 1 if renormalise else 0, balance_coef, z_coef,
              p, p + 4 * at_f, p + 4 * (at_f + slots), p + 8 * slots, p + 8 * slots + 4 * experts, p + 4 * slots,
              p + 4 * at_f - 4, p + 4 * at_work - 4, p + 4 * at_work, 4 * scratch, _DTYPE[logits.dtype],
              _raw_stream(dev.index))
    ints = floats.view(_I32)
    part, at = ints.as_strided, 2 * slots
    return Routing(part((n, top_k), (top_k, 1), 0), floats.as_strided((n, top_k), (top_k, 1), at_f),
                   part((experts,), (1,), at), part((experts + 1,), (1,), at + experts), part((slots,), (1,), slots),
                   floats.as_strided((), (), at_work - 1), floats.as_strided((n,), (1,), at_f + slots),
                   part((), (), at_f - 1))


def route_backward(logits, routing: Routing, dweights=None, renormalise: bool = True, balance_coef: float = 0.0,
                   z_coef: float = 0.0, dlogits=None, stream=None):
    """The gradient of route's logits (ns_route_backward) from ``dweights``, the
    gradient of the weights (rows x top_k float32, None: zero), and of the loss with
    the same coefficients. ``dlogits`` is where it goes (it may be ``logits``
    itself); allocated when not given. Returns it."""
    ld = _matrix(logits, "logits")
    n, experts = logits.shape
    dev = logits.device
    if routing.experts.dim() != 2:
        raise ValueError("routing does not belong to logits")
    top_k = routing.experts.shape[1]
    p_ids = _contiguous(routing.experts, "routing.experts", (n, top_k), _I32, dev)
    p_w = _contiguous(routing.weights, "routing.weights", (n, top_k), _F32, dev)
    p_z = _contiguous(routing.logz, "routing.logz", (n,), _F32, dev)
    p_c = _contiguous(routing.counts, "routing.counts", (experts,), _I32, dev)
    p_l = _contiguous(routing.live_rows, "routing.live_rows", (), _I32, dev)
    p_dw = None if dweights is None else _contiguous(dweights, "dweights", (n, top_k), _F32, dev)
    ld_d = experts
    if dlogits is not None:
        _same_device(dev, dlogits)
        ld_d = _matrix(dlogits, "dlogits", n, experts, logits.dtype)
    with _on(dev, stream):
        if dlogits is None:
            dlogits = _empty((n, experts), dtype=logits.dtype, device=dev)
        _call("ns_route_backward", logits.data_ptr(), ld, n, experts, top_k, p_ids, p_w, p_dw, p_z, p_c, p_l,
              1 if renormalise else 0, balance_coef, z_coef, dlogits.data_ptr(), ld_d, _DTYPE[logits.dtype],
              _raw_stream(dev.index))
    return dlogits


# ------------------------------------------------------------------ 8-bit floating point
def _pitch(cols):
    return (cols + 15) // 16 * 16


def _scale_pitch(cols):
    return ((cols + 127) // 128 + 3) // 4 * 4


class Blocks8:
    """A matrix held in e4m3 with power-of-two scales (include/ns.h). Rows form:
    ``q`` (uint8, rows x cols rounded up to 16), ``scales`` (uint8, one per 128
    values, rounded up to 4 a row). Tiles form (a stack of matrices): q groups x
    rows x .., scales groups x ceil(rows / 128) x .., one per 128 x 128 values."""

    __slots__ = ("groups", "rows", "cols", "tiles", "device", "_q", "_scales", "_buffer", "_p_q", "_p_scales")

    def __init__(self, q, scales, cols: int, tiles: bool = False):
        cols, lead = int(cols), 3 if tiles else 2
        if q.dim() != lead or scales.dim() != lead:
            raise ValueError("q and scales must be 3-D for tiles, 2-D for rows")
        self.groups, self.rows, self.cols, self.tiles = (q.shape[0] if tiles else 1), q.shape[-2], cols, bool(tiles)
        self.device = q.device
        want_q, want_s = self._shapes()
        if q.dtype != torch.uint8 or q.shape != want_q or not q.is_contiguous():
            raise ValueError(f"q must be contiguous uint8 of shape {want_q}")
        if scales.dtype != torch.uint8 or scales.shape != want_s or not scales.is_contiguous():
            raise ValueError(f"scales must be contiguous uint8 of shape {want_s}")
        if not q.is_cuda or scales.device != q.device:
            raise ValueError("q and scales must be CUDA tensors on one device")
        self._q, self._scales, self._buffer = q, scales, None
        self._p_q, self._p_scales = q.data_ptr(), scales.data_ptr()

    def _shapes(self):
        pitch, scale_pitch = _pitch(self.cols), _scale_pitch(self.cols)
        if self.tiles:
            return (self.groups, self.rows, pitch), (self.groups, (self.rows + 127) // 128, scale_pitch)
        return (self.rows, pitch), (self.rows, scale_pitch)

    @classmethod
    def _empty(cls, groups, rows, cols, tiles, device):
        self = cls.__new__(cls)
        self.groups, self.rows, self.cols, self.tiles, self.device = groups, rows, cols, tiles, device
        nq = groups * rows * _pitch(cols)  # a multiple of 16
        bands = groups * ((rows + 127) // 128) if tiles else rows
        self._q = self._scales = None  # views of the buffer, made when asked for
        self._buffer = _empty(nq + bands * _scale_pitch(cols), dtype=torch.uint8, device=device)
        self._p_q = self._buffer.data_ptr()
        self._p_scales = self._p_q + nq
        return self

    @property
    def q(self):
        if self._q is None:
            shape = self._shapes()[0]
            self._q = self._buffer[:self.groups * self.rows * shape[-1]].view(shape)
        return self._q

    @property
    def scales(self):
        if self._scales is None:
            q, shape = self._shapes()
            self._scales = self._buffer[self.groups * self.rows * q[-1]:].view(shape)
        return self._scales

    def nbytes(self) -> int:
        bands = self.groups * ((self.rows + 127) // 128) if self.tiles else self.rows
        return self.groups * self.rows * _pitch(self.cols) + bands * _scale_pitch(self.cols)


def blocks_store(x, tiles: bool = False, rows=None, per: int = 1, stream=None) -> Blocks8:
    """Hold a matrix in 8-bit floating point (ns_blocks_store_rows, _tiles).
    Activations: a scale per 128 values of a row; with ``rows`` (int32) row r holds
    ``x[rows[r] // per]``, zeros where rows[r] is negative (with a routing's order and
    per = top_k: every expert's rows in turn). Weights: ``tiles``, a scale per 128 x
    128 values; ``x`` may then be a contiguous stack of matrices."""
    if tiles:
        if rows is not None or per != 1:
            raise ValueError("tiles are not gathered")
        if x.dim() == 3:
            if not x.is_contiguous():
                raise ValueError("a stack of matrices must be contiguous")
            groups, n, cols = x.shape
            if not x.is_cuda:
                raise ValueError("x must be a CUDA tensor")
            if x.dtype not in _DTYPE:
                raise TypeError(f"x: unsupported dtype {x.dtype}: use float32 or bfloat16")
            ld = cols
        else:
            ld, groups = _matrix(x, "x"), 1
            n, cols = x.shape
        dev = x.device
        with _on(dev, stream):
            b = Blocks8._empty(groups, n, cols, True, dev)
            _call("ns_blocks_store_tiles", x.data_ptr(), ld, groups, n, cols, b._p_q, b._p_scales,
                  _DTYPE[x.dtype], _raw_stream(dev.index))
        return b
    ld = _matrix(x, "x")
    n, cols = x.shape
    dev = x.device
    count, p_rows, per = n, None, int(per)
    if rows is not None:
        count = rows.numel()
        p_rows = _vector(rows, "rows", count, (_I32,), dev)
        if not 1 <= per < 1 << 31:  # (an int of the C call, which ctypes would cut short)
            raise ValueError("per must be positive and below 2^31")
    elif per != 1:
        raise ValueError("per needs rows")
    with _on(dev, stream):
        b = Blocks8._empty(1, count, cols, False, dev)
        _call("ns_blocks_store_rows", x.data_ptr(), ld, n, p_rows, per, count, cols, b._p_q, b._p_scales,
              _DTYPE[x.dtype], _raw_stream(dev.index))
    return b


def blocks_load(b: Blocks8, dtype=torch.bfloat16, out=None, stream=None):
    """The values that a Blocks8 holds (ns_blocks_load): rows x cols, a stack of
    matrices for tiles. ``out`` (2-D, all rows) is where they go when given."""
    dev, all_rows, ld = b.device, b.groups * b.rows, b.cols
    if out is not None:
        _same_device(dev, out)
        ld = _matrix(out, "out", all_rows, b.cols)
    elif dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype}: use float32 or bfloat16")
    with _on(dev, stream):
        if out is None:
            out = _empty((b.groups, b.rows, b.cols) if b.tiles else (b.rows, b.cols), dtype=dtype, device=dev)
        _call("ns_blocks_load", b._p_q, b._p_scales, 1 if b.tiles else 0, b.groups, b.rows, b.cols,
              out.data_ptr(), ld, _DTYPE[out.dtype], _raw_stream(dev.index))
    return out


def blocks_matmul(a: Blocks8, w: Blocks8, transpose: bool = False, offsets=None, dtype=torch.bfloat16, out=None,
                  stream=None):
    """``a @ w[e]^T`` (a layer, forward) or with ``transpose`` ``a @ w[e]`` (its
    input's gradient) for the rows of every group e (ns_blocks_matmul). ``a`` is held
    in rows, ``w`` in tiles; ``offsets`` (int32, on the device, groups + 1 ascending row
    numbers, e.g. a routing's) gives each matrix of the stack its rows of a; rows of
    no group become zeros. Without it w is one matrix. Returns rows x n of ``dtype``,
    in ``out`` when given."""
    if a.tiles or not w.tiles:
        raise ValueError("a must be held in rows, w in tiles")
    dev = a.device
    _same_device(dev, w, offsets, out)
    k, n = (w.rows, w.cols) if transpose else (w.cols, w.rows)
    if a.cols != k:
        raise ValueError(f"a has {a.cols} columns, w takes {k}")
    p_off = None
    if offsets is not None:
        p_off = _vector(offsets, "offsets", w.groups + 1, (_I32,), dev)
    elif w.groups != 1:
        raise ValueError("a stack of matrices needs offsets")
    ld = n
    if out is not None:
        ld = _matrix(out, "out", a.rows, n)
    elif dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype}: use float32 or bfloat16")
    with _on(dev, stream):
        if out is None:
            out = _empty((a.rows, n), dtype=dtype, device=dev)
        _call("ns_blocks_matmul", a._p_q, a._p_scales, a.rows, k, w._p_q, w._p_scales, n,
              1 if transpose else 0, p_off, w.groups, out.data_ptr(), ld, _DTYPE[out.dtype], _raw_stream(dev.index))
    return out


# ------------------------------------------------------------------ norms around a block
class BlockNorm(NamedTuple):
    residual: torch.Tensor            # rows x cols, type of x
    normed: torch.Tensor | None       # rows x cols, type of y
    rstd: torch.Tensor                # 2 x rows, float32, for the backward pass: of y, of residual


class BlockNormGrads(NamedTuple):
    dx: torch.Tensor
    dy: torch.Tensor | None
    dgate: torch.Tensor | None
    dpost_weight: torch.Tensor | None
    dpre_weight: torch.Tensor | None


_NONE, _COLS, _ROWS, _FULL = range(4)


def _norm_arguments(x, y, gate, post_weight, pre_weight):
    """What both directions pass on: (rows, cols, device, pitches and codes)."""
    ld_x = _matrix(x, "x")
    n, cols = x.shape
    dev, dt = x.device, x.dtype
    _same_device(dev, y, gate, post_weight, pre_weight)
    ld_y, bt = cols, dt
    if y is not None:
        ld_y, bt = _matrix(y, "y", n, cols), y.dtype
        if dt == torch.bfloat16 and bt != dt:
            raise ValueError("y may not be wider than x")
    elif gate is not None or post_weight is not None:
        raise ValueError("gate and post_weight need y")
    elif pre_weight is None:
        raise ValueError("give y or pre_weight")
    wt = None
    for what, v in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        if v is not None:
            _vector(v, what, cols, tuple(_DTYPE) if wt is None else (wt,), dev)
            wt = v.dtype
    form, ld_g, gt = _NONE, 0, dt
    if gate is not None:
        gt = gate.dtype
        if gate.dim() == 1:
            form = _COLS
            _vector(gate, "gate", cols, tuple(_DTYPE), dev)
        elif gate.shape == (n, 1) and cols != 1:
            form, ld_g = _ROWS, _matrix(gate, "gate")
        else:
            form, ld_g = _FULL, _matrix(gate, "gate", n, cols)
    return n, cols, dev, ld_x, ld_y, form, ld_g, (_DTYPE[dt], _DTYPE[bt], _DTYPE[wt or dt], _DTYPE[gt])


def block_norm(x, y=None, gate=None, post_weight=None, pre_weight=None, residual_scale: float = 1.0,
               block_scale: float = 1.0, eps: float = 1e-6, residual=None, normed=None, stream=None) -> BlockNorm:
    """The norms after and before a block with its gate and the residual scale
    (ns_block_norm): ``residual = residual_scale * x + block_scale * gate * norm(y) *
    post_weight`` and ``normed = norm(residual) * pre_weight``, norm(v) = v /
    sqrt(mean(v^2) + eps) over a row. ``x`` is the residual stream, ``y`` the block's
    output (None: a first norm without a block before it; bfloat16 beside a float32 x
    is allowed). ``gate`` is one value per column (1-D), one per row (rows x 1) or a
    whole matrix; without ``post_weight`` y is not normed, without ``pre_weight``
    there is no ``normed``. ``residual`` (may be x) and ``normed`` (may be y) are where
    the results go; allocated when not given."""
    n, cols, dev, ld_x, ld_y, form, ld_g, codes = _norm_arguments(x, y, gate, post_weight, pre_weight)
    bt = x.dtype if y is None else y.dtype
    ld_r = ld_z = cols
    if residual is not None:
        _same_device(dev, residual)
        ld_r = _matrix(residual, "residual", n, cols, x.dtype)
    if normed is not None:
        if pre_weight is None:
            raise ValueError("normed given, but no pre_weight")
        _same_device(dev, normed)
        ld_z = _matrix(normed, "normed", n, cols, bt)
    with _on(dev, stream):
        if residual is None:
            residual = _empty((n, cols), dtype=x.dtype, device=dev)
        if normed is None and pre_weight is not None:
            normed = _empty((n, cols), dtype=bt, device=dev)
        rstd = _empty((2, n), dtype=_F32, device=dev)
        p_rstd = rstd.data_ptr()
        _call("ns_block_norm", x.data_ptr(), ld_x, _ptr(y), ld_y, _ptr(gate), form, ld_g, _ptr(post_weight),
              _ptr(pre_weight), n, cols, residual_scale, block_scale, eps, residual.data_ptr(), ld_r, _ptr(normed), ld_z,
              p_rstd, p_rstd + 4 * n, *codes, _raw_stream(dev.index))
    return BlockNorm(residual, normed, rstd)


def block_norm_backward(dresidual, dnormed, x, y, saved: BlockNorm, gate=None, post_weight=None, pre_weight=None,
                        residual_scale: float = 1.0, block_scale: float = 1.0, dx=None, dy=None,
                        stream=None) -> BlockNormGrads:
    """Backward of block_norm (ns_block_norm_backward) from the gradients of
    ``residual`` (None: zero) and ``normed`` (None without pre_weight). The other
    arguments are those of the forward call (``x`` and ``y`` as they were before it, where it
    wrote over them), ``saved`` is its result. ``dx`` (may be dresidual) and ``dy`` (may be dnormed) are where those gradients go; allocated when
    not given. Gradients have the types of what they belong to; a gate's has its shape."""
    n, cols, dev, ld_x, ld_y, form, ld_g, codes = _norm_arguments(x, y, gate, post_weight, pre_weight)
    if dresidual is None and pre_weight is None:
        raise ValueError("without pre_weight, give dresidual")
    if (dnormed is None) != (pre_weight is None):
        raise ValueError("dnormed goes with pre_weight")
    _same_device(dev, dresidual, dnormed, dx, dy)
    bt = x.dtype if y is None else y.dtype
    ld_dr = cols if dresidual is None else _matrix(dresidual, "dresidual", n, cols, x.dtype)
    ld_dz = cols if dnormed is None else _matrix(dnormed, "dnormed", n, cols, bt)
    p_rstd = _contiguous(saved.rstd, "saved.rstd", (2, n), _F32, dev)
    ld_dx = cols if dx is None else _matrix(dx, "dx", n, cols, x.dtype)
    if dy is not None and y is None:
        raise ValueError("dy given, but no y")
    ld_dy = cols if dy is None else _matrix(dy, "dy", n, cols, bt)
    scratch = max(1, min(n, _MAX_PARTS)) * 2 * cols
    with _on(dev, stream):
        if dx is None:
            dx = _empty((n, cols), dtype=x.dtype, device=dev)
        if dy is None and y is not None:
            dy = _empty((n, cols), dtype=bt, device=dev)
        dgate = None if gate is None else _empty(gate.shape, dtype=gate.dtype, device=dev)
        dpost = dpre = None
        if post_weight is not None and pre_weight is not None:  # both in one allocation
            dpost, dpre = _empty((2, cols), dtype=pre_weight.dtype, device=dev).unbind()
        elif pre_weight is not None:
            dpre = _empty(cols, dtype=pre_weight.dtype, device=dev)
        elif post_weight is not None:
            dpost = _empty(cols, dtype=post_weight.dtype, device=dev)
        work = _empty(max(scratch, 1), dtype=_F32, device=dev)
        _call("ns_block_norm_backward", _ptr(dresidual), ld_dr, _ptr(dnormed), ld_dz, x.data_ptr(), ld_x, _ptr(y), ld_y,
              _ptr(gate), form, ld_g, _ptr(post_weight), _ptr(pre_weight), p_rstd, p_rstd + 4 * n, n, cols, residual_scale,
              block_scale, dx.data_ptr(), ld_dx, _ptr(dy), ld_dy, _ptr(dgate), 1 if form == _ROWS else cols, _ptr(dpost),
              _ptr(dpre), work.data_ptr(), 4 * max(scratch, 1), *codes, _raw_stream(dev.index))
    return BlockNormGrads(dx, dy, dgate, dpost, dpre)


# ------------------------------------------------------------------ dropout
_U64 = (1 << 64) - 1


def dropout(x, p: float, seed: int, offset: int = 0, residual=None, state=None, out=None, stream=None):
    """``[residual +] x`` with a share ``p`` of its elements dropped and the others
    divided by the share that stays (ns_dropout). The mask is a function of seed,
    offset and place and is not stored: the same call on the gradient, without
    residual, is the backward pass. A call uses rows * ceil(cols / 8) counters from
    ``offset`` on: give the next call that offset. ``state`` (int64, 2, on the device)
    is added to (seed, offset), so that a captured call draws anew. ``residual`` has
    x's type, or float32; the result has its type. ``out`` may be x or residual."""
    ld = _matrix(x, "x")
    n, cols = x.shape
    dev, dt = x.device, x.dtype
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be between 0 and 1")
    _same_device(dev, residual, out)
    ld_r, ot = cols, dt
    if residual is not None:
        ld_r, ot = _matrix(residual, "residual", n, cols), residual.dtype
        if ot != dt and ot != _F32:
            raise ValueError("residual may not be narrower than x")
    p_state = None if state is None else _vector(state, "state", 2, (torch.int64,), dev)
    ld_o = cols if out is None else _matrix(out, "out", n, cols, ot)
    with _on(dev, stream):
        if out is None:
            out = _empty((n, cols), dtype=ot, device=dev)
        _call("ns_dropout", x.data_ptr(), ld, _ptr(residual), ld_r, n, cols, p, int(seed) & _U64, int(offset) & _U64, p_state,
              out.data_ptr(), ld_o, _DTYPE[dt], _DTYPE[ot], _raw_stream(dev.index))
    return out


def dropout_counters(rows: int, cols: int) -> int:
    """Counters that dropout of a rows x cols matrix uses."""
    return rows * ((cols + 7) // 8)
