"""Sequence operators: ``causal_conv``, ``state_scan`` and ``block_norm``.

Together with 1x1 convolutions (``forward`` / ``backward`` on [B, D, 1, L]) they
make up a gated state space block, for training, for prompts and for single
tokens (examples/mixer_block.py runs one).  Activations are channel-first,
[B, D, L] with contiguous positions and any batch and channel strides, float32,
bfloat16 or float16; parameters, scan states and the residual stream are
contiguous float32.  include/sequence_ops.h has the formulas; the C entry
points mirror these names.

Like the convolutions these are plain functions, not autograd nodes: each
gradient is a call of its own.  Calls are asynchronous on ``stream`` (a torch
stream; default: the current one), which the caller orders after whatever
produced the inputs.  Bad arguments raise ValueError or ``Conv2dGiError``
before anything is launched.
"""
from __future__ import annotations

import collections
import ctypes
import struct

import torch

from . import _check, load_library

__all__ = ["causal_conv", "causal_conv_backward", "causal_conv_step", "state_scan",
           "state_scan_backward", "state_scan_step", "block_norm", "block_norm_backward",
           "ScanGrads", "NormGrads", "SCAN_CHECKPOINT"]

#: Positions between two checkpoints of ``state_scan`` (SEQ_SCAN_CHECKPOINT).
SCAN_CHECKPOINT = 128

ScanGrads = collections.namedtuple("ScanGrads", "dx ddt dA dB dC dD dz ddt_bias dstate")
NormGrads = collections.namedtuple("NormGrads", "dy dresidual dgate dscale dweight_post dweight_pre")

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

# The argument structs of sequence_ops.h: int32 fields, then pointers and
# int64 fields (a tensor is its address and two strides).
_CONV = struct.Struct("6i11q")
_CONV_BACKWARD = struct.Struct("6i16q")
_CONV_STEP = struct.Struct("6i10q")
_SCAN = struct.Struct("8i25q")
_SCAN_BACKWARD = struct.Struct("8i41q")
_SCAN_STEP = struct.Struct("8i23q")
_NORM = struct.Struct("4ifi21q")
_NORM_BACKWARD = struct.Struct("4ifi33q")

_NONE = (0, 0, 0)
_entries = {}


def _entry(name):
    fn = _entries.get(name)
    if fn is None:
        fn = getattr(load_library(), name)
        if name.endswith("_workspace"):
            fn.restype = ctypes.c_int64
        else:
            fn.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
            fn.restype = ctypes.c_int
        _entries[name] = fn
    return fn


class _On:
    """Where a call runs: the device, and the stream that the caller named."""

    def __init__(self, t, name, dims, stream):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError("%s must be a tensor on a GPU device" % name)
        if t.dim() != dims:
            raise ValueError("%s must have %d dimensions, has %d" % (name, dims, t.dim()))
        self.dtype = t.dtype
        if self.dtype not in _DTYPES:
            raise ValueError("%s must be float32, bfloat16 or float16" % name)
        self.code = _DTYPES[self.dtype]
        self.device = t.device
        self.index = t.device.index
        current = torch._C._cuda_getCurrentRawStream(self.index)
        # Memory handed between two streams has to be marked for both.
        self.other = stream if stream is not None and stream.cuda_stream != current else None
        self.stream = current if self.other is None else stream.cuda_stream
        self.taken = []

    def act(self, t, name, shape, dtype=None):
        """(address, batch stride, channel stride) of an activation of a shape."""
        if (not isinstance(t, torch.Tensor) or t.device != self.device
                or t.dtype is not (dtype or self.dtype) or t.shape != shape):
            self.refuse(t, name, shape, dtype or self.dtype)
        stride = t.stride()
        if len(shape) == 3 and stride[2] != 1 and shape[2] > 1:
            raise ValueError("%s must have contiguous positions" % name)
        if self.other is not None:
            self.taken.append(t)
        return t.data_ptr(), stride[0], stride[1]

    def states(self, t, name, shape):
        """The same for B and C, [B, G, N] or [B, G, N, L]: the stride between states."""
        if (not isinstance(t, torch.Tensor) or t.device != self.device
                or t.dtype is not self.dtype or t.shape != shape):
            self.refuse(t, name, shape, self.dtype)
        stride = t.stride()
        if len(shape) == 4 and stride[3] != 1 and shape[3] > 1:
            raise ValueError("%s must have contiguous positions" % name)
        step = stride[2] if shape[2] > 1 else stride[1]
        if shape[1] > 1 and shape[2] > 1 and stride[1] != shape[2] * step:
            raise ValueError("the groups of %s must follow each other like its states" % name)
        if self.other is not None:
            self.taken.append(t)
        return t.data_ptr(), stride[0], step

    def dense(self, t, name, shape, dtype=torch.float32):
        """The address of a contiguous tensor of a shape."""
        if (not isinstance(t, torch.Tensor) or t.device != self.device or t.dtype is not dtype
                or t.shape != shape or not t.is_contiguous()):
            self.refuse(t, name, shape, dtype)
        if self.other is not None:
            self.taken.append(t)
        return t.data_ptr()

    def maybe(self, t, name, shape, dtype=torch.float32):
        return 0 if t is None else self.dense(t, name, shape, dtype)

    def refuse(self, t, name, shape, dtype):
        if not isinstance(t, torch.Tensor):
            raise ValueError("%s must be a tensor" % name)
        if t.device != self.device:
            raise ValueError("%s must be on %s like the other tensors" % (name, self.device))
        if t.dtype is not dtype:
            raise ValueError("%s must be %s, is %s" % (name, dtype, t.dtype))
        if tuple(t.shape) != tuple(shape):
            raise ValueError("%s must be %r, is %r" % (name, tuple(shape), tuple(t.shape)))
        raise ValueError("%s must be contiguous" % name)

    def empty(self, shape, dtype=None):
        if self.other is None:
            return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)
        with torch.cuda.stream(self.other):
            t = torch.empty(shape, dtype=dtype or self.dtype, device=self.device)
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def workspace(self, bytes_):
        if bytes_ <= 0:  # none needed; or (-1) sizes that the call itself refuses
            return 0, 0
        t = self.scratch = self.empty((bytes_,), torch.uint8)
        return t.data_ptr(), bytes_

    def call(self, name, packed):
        if torch._C._cuda_getDevice() == self.index:
            code = _entry(name)(packed, self.stream)
        else:
            with torch.cuda.device(self.device):
                code = _entry(name)(packed, self.stream)
        if code:
            _check(code)
        for t in self.taken:
            t.record_stream(self.other)


def causal_conv(x, weight, bias=None, *, silu=True, state=None, lengths=None, want_state=False,
                out=None, stream=None):
    """Depthwise causal convolution of K taps with bias and SiLU: (y, new_state).

    x [B, D, L]; weight [D, K], bias [D] float32.  state [B, D, K-1] (x's dtype):
    the inputs before position 0, zeros by default.  lengths int32 [B]: positions
    of each sequence (y is 0 beyond).  new_state, for the next call or
    ``causal_conv_step``, is None unless want_state.
    """
    on = _On(x, "x", 3, stream)
    shape = x.shape
    B, D, L = shape
    K = weight.shape[-1] if isinstance(weight, torch.Tensor) and weight.dim() else 0
    xs = on.act(x, "x", shape)
    w = on.dense(weight, "weight", (D, K))
    b = on.maybe(bias, "bias", (D,))
    s_in = on.maybe(state, "state", (B, D, K - 1), on.dtype)
    n = on.maybe(lengths, "lengths", (B,), torch.int32)
    if out is None:
        out = on.empty(shape)
    new = on.empty((B, D, max(K - 1, 0))) if want_state else None
    on.call("causal_conv_forward", _CONV.pack(
        on.code, B, D, L, K, bool(silu), *xs, *on.act(out, "out", shape), w, b, s_in,
        0 if new is None else new.data_ptr(), n))
    return out, new


def causal_conv_backward(grad_out, x, weight, bias=None, *, silu=True, lengths=None, want_dx=True,
                         want_dw=True, want_db=None, dx=None, stream=None):
    """The gradients of ``causal_conv`` from a zero state: (dx, dweight, dbias),
    each None when not wanted (dbias by default where there is a bias)."""
    on = _On(x, "x", 3, stream)
    shape = x.shape
    B, D, L = shape
    K = weight.shape[-1] if isinstance(weight, torch.Tensor) and weight.dim() else 0
    gs, xs = on.act(grad_out, "grad_out", shape), on.act(x, "x", shape)
    w = on.dense(weight, "weight", (D, K))
    b = on.maybe(bias, "bias", (D,))
    n = on.maybe(lengths, "lengths", (B,), torch.int32)
    if want_db is None:
        want_db = bias is not None
    if not want_dx:
        dx = None
    elif dx is None:
        dx = on.empty(shape)
    dw = on.empty((D, K), torch.float32) if want_dw else None
    db = on.empty((D,), torch.float32) if want_db else None
    ws = on.workspace(_entry("causal_conv_workspace")(B, D, L, K))
    on.call("causal_conv_backward", _CONV_BACKWARD.pack(
        on.code, B, D, L, K, bool(silu), *gs, *xs, *(_NONE if dx is None else on.act(dx, "dx", shape)),
        w, b, 0 if dw is None else dw.data_ptr(), 0 if db is None else db.data_ptr(), n, *ws))
    return dx, dw, db


def causal_conv_step(x, state, weight, bias=None, *, silu=True, slots=None, out=None, stream=None):
    """One position of ``causal_conv`` for every row: y [B, D] from x [B, D].

    state [lines, D, K-1] (x's dtype, contiguous) is updated in place.  slots
    int32 [B]: the line of each row (row b uses line b without); a slot outside
    the lines marks a padding row, whose y is 0 and which changes no line.
    """
    on = _On(x, "x", 2, stream)
    shape = x.shape
    B, D = shape
    K = weight.shape[-1] if isinstance(weight, torch.Tensor) and weight.dim() else 0
    lines = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0
    xs = on.act(x, "x", shape)
    st = on.dense(state, "state", (lines, D, K - 1), on.dtype)
    w = on.dense(weight, "weight", (D, K))
    b = on.maybe(bias, "bias", (D,))
    sl = on.maybe(slots, "slots", (B,), torch.int32)
    if out is None:
        out = on.empty(shape)
    on.call("causal_conv_step", _CONV_STEP.pack(
        on.code, B, D, K, bool(silu), lines, *xs, *on.act(out, "out", shape), w, b, st, sl))
    return out


def _scan_sizes(A, B):
    """(N, B's shape without batch and positions) from A [D, N] and B."""
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a tensor [D, N]")
    if not isinstance(B, torch.Tensor):
        raise ValueError("B must be a tensor")
    return A.shape[1]


def _grouped(t, name, dims):
    """B or C with its axis of groups: [B, N, ...] has one group."""
    if isinstance(t, torch.Tensor) and t.dim() == dims - 1:
        return t.unsqueeze(1)
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError("%s must be a tensor of %d or %d dimensions" % (name, dims - 1, dims))
    return t


def state_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, softplus=True, state=None,
               lengths=None, want_state=False, want_checkpoints=False, out=None, stream=None):
    """The selective state space scan over a prompt: (y, new_state, checkpoints).

    x, dt, z [B, D, L]; A [D, N] float32; B, C [B, G, N, L] or [B, N, L]; D (the
    skip) and dt_bias [D] float32.  h_t = exp(s_t A) h_{t-1} + s_t x_t B_t,
    y_t = C_t . h_t + D x_t, times silu(z) where z is given, with s = softplus(dt +
    dt_bias).  state [B, D, N] float32: h before position 0.  new_state and the
    checkpoints that ``state_scan_backward`` takes are None unless wanted.
    """
    on = _On(x, "x", 3, stream)
    shape = x.shape
    nB, nD, L = shape
    N = _scan_sizes(A, B)
    B, C = _grouped(B, "B", 4), _grouped(C, "C", 4)
    G = B.shape[1]
    bc = (nB, G, N, L)
    args = (*on.act(x, "x", shape), *on.act(dt, "dt", shape),
            *(_NONE if z is None else on.act(z, "z", shape)),
            *on.states(B, "B", bc), *on.states(C, "C", bc))
    params = (on.dense(A, "A", (nD, N)), on.maybe(D, "D", (nD,)), on.maybe(dt_bias, "dt_bias", (nD,)),
              on.maybe(state, "state", (nB, nD, N)))
    n = on.maybe(lengths, "lengths", (nB,), torch.int32)
    if out is None:
        out = on.empty(shape)
    new = on.empty((nB, nD, N), torch.float32) if want_state else None
    marks = (on.empty((nB, nD, -(-L // SCAN_CHECKPOINT), N), torch.float32)
             if want_checkpoints else None)
    on.call("state_scan_forward", _SCAN.pack(
        on.code, nB, nD, L, N, G, bool(softplus), 0, *args, *on.act(out, "out", shape), *params,
        0 if new is None else new.data_ptr(), 0 if marks is None else marks.data_ptr(), n))
    return out, new, marks


def state_scan_backward(grad_out, x, dt, A, B, C, checkpoints, D=None, z=None, dt_bias=None, *,
                        softplus=True, lengths=None, grad_state=None, want_dstate=False, dx=None,
                        ddt=None, dz=None, stream=None):
    """The gradients of ``state_scan``: a ``ScanGrads``.

    Arguments as the forward call's, with its checkpoints.  grad_state [B, D, N]:
    the gradient of new_state (zeros by default); dstate, that of state, is None
    unless wanted.  dB and dC have B's shape.  dx, ddt, dz: optional outputs.
    """
    on = _On(x, "x", 3, stream)
    shape = x.shape
    nB, nD, L = shape
    N = _scan_sizes(A, B)
    shape_bc = B.shape
    B, C = _grouped(B, "B", 4), _grouped(C, "C", 4)
    G = B.shape[1]
    bc = (nB, G, N, L)
    args = (*on.act(grad_out, "grad_out", shape), *on.act(x, "x", shape), *on.act(dt, "dt", shape),
            *(_NONE if z is None else on.act(z, "z", shape)),
            *on.states(B, "B", bc), *on.states(C, "C", bc))
    params = (on.dense(A, "A", (nD, N)), on.maybe(D, "D", (nD,)), on.maybe(dt_bias, "dt_bias", (nD,)),
              on.dense(checkpoints, "checkpoints", (nB, nD, -(-L // SCAN_CHECKPOINT), N)),
              on.maybe(grad_state, "grad_state", (nB, nD, N)))
    n = on.maybe(lengths, "lengths", (nB,), torch.int32)
    dx = on.empty(shape) if dx is None else dx
    ddt = on.empty(shape) if ddt is None else ddt
    if z is None:
        if dz is not None:
            raise ValueError("dz needs z")
    elif dz is None:
        dz = on.empty(shape)
    f32 = torch.float32
    g = ScanGrads(dx, ddt, on.empty((nD, N), f32), on.empty(shape_bc), on.empty(shape_bc),
                  None if D is None else on.empty((nD,), f32), dz,
                  None if dt_bias is None else on.empty((nD,), f32),
                  on.empty((nB, nD, N), f32) if want_dstate else None)
    ws = on.workspace(_entry("state_scan_workspace")(nB, nD, L, N, G))
    on.call("state_scan_backward", _SCAN_BACKWARD.pack(
        on.code, nB, nD, L, N, G, bool(softplus), 0, *args, *on.act(dx, "dx", shape),
        *on.act(ddt, "ddt", shape), *(_NONE if z is None else on.act(dz, "dz", shape)), *params,
        g.dB.data_ptr(), g.dC.data_ptr(), g.dA.data_ptr(), 0 if g.dD is None else g.dD.data_ptr(),
        0 if g.ddt_bias is None else g.ddt_bias.data_ptr(),
        0 if g.dstate is None else g.dstate.data_ptr(), n, *ws))
    return g


def state_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, *, softplus=True,
                    slots=None, out=None, stream=None):
    """One position of ``state_scan`` for every row: y [B, D].

    x, dt, z [B, D]; B, C [B, G, N] or [B, N]; state [lines, D, N] float32
    (contiguous) is updated in place; slots as in ``causal_conv_step``.
    """
    on = _On(x, "x", 2, stream)
    shape = x.shape
    nB, nD = shape
    N = _scan_sizes(A, B)
    B, C = _grouped(B, "B", 3), _grouped(C, "C", 3)
    G = B.shape[1]
    bc = (nB, G, N)
    lines = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0
    args = (*on.act(x, "x", shape), *on.act(dt, "dt", shape),
            *(_NONE if z is None else on.act(z, "z", shape)),
            *on.states(B, "B", bc), *on.states(C, "C", bc))
    params = (on.dense(A, "A", (nD, N)), on.maybe(D, "D", (nD,)), on.maybe(dt_bias, "dt_bias", (nD,)),
              on.dense(state, "state", (lines, nD, N)), on.maybe(slots, "slots", (nB,), torch.int32))
    if out is None:
        out = on.empty(shape)
    on.call("state_scan_step", _SCAN_STEP.pack(
        on.code, nB, nD, N, G, bool(softplus), lines, 0, *args, *on.act(out, "out", shape), *params))
    return out


def block_norm(y, residual, weight_post=None, weight_pre=None, *, gate=None, scale=None, eps=1e-6,
               lengths=None, residual_out=None, out=None, stream=None):
    """What stands between two residual blocks: (new_residual, u).

    y [B, D, L], the block's output, goes through an RMS norm over the channels
    (weight_post; without it y as it is), times sigmoid(gate) [B, D, L] and scale
    [D], into residual [B, D, L] float32; u, the next block's input in y's dtype,
    is the RMS norm of the sum (weight_pre; None without it).  residual_out may be
    the residual itself.
    """
    on = _On(y, "y", 3, stream)
    shape = y.shape
    B, D, L = shape
    f32 = torch.float32
    args = (*on.act(y, "y", shape), *(_NONE if gate is None else on.act(gate, "gate", shape)),
            *on.act(residual, "residual", shape, f32))
    params = (on.maybe(scale, "scale", (D,)), on.maybe(weight_post, "weight_post", (D,)),
              on.maybe(weight_pre, "weight_pre", (D,)), on.maybe(lengths, "lengths", (B,), torch.int32))
    if residual_out is None:
        residual_out = on.empty(shape, f32)
    if weight_pre is None:
        if out is not None:
            raise ValueError("out needs weight_pre")
    elif out is None:
        out = on.empty(shape)
    ws = on.workspace(_entry("block_norm_workspace")(B, D, L, 0))
    on.call("block_norm_forward", _NORM.pack(
        on.code, B, D, L, eps, 0, *args, *on.act(residual_out, "residual_out", shape, f32),
        *(_NONE if out is None else on.act(out, "out", shape)), *params, *ws))
    return residual_out, out


def block_norm_backward(grad_residual, grad_out, y, residual_out, weight_post=None, weight_pre=None,
                        *, gate=None, scale=None, eps=1e-6, lengths=None, dy=None, dresidual=None,
                        dgate=None, stream=None):
    """The gradients of ``block_norm``: a ``NormGrads`` (None where there is no input).

    grad_residual (float32) is the gradient of new_residual, grad_out that of u;
    either may be None.  residual_out: the forward call's new_residual.
    """
    on = _On(y, "y", 3, stream)
    shape = y.shape
    B, D, L = shape
    f32 = torch.float32
    args = (*(_NONE if grad_residual is None else on.act(grad_residual, "grad_residual", shape, f32)),
            *(_NONE if grad_out is None else on.act(grad_out, "grad_out", shape)),
            *on.act(y, "y", shape), *(_NONE if gate is None else on.act(gate, "gate", shape)),
            *on.act(residual_out, "residual_out", shape, f32))
    params = (on.maybe(scale, "scale", (D,)), on.maybe(weight_post, "weight_post", (D,)),
              on.maybe(weight_pre, "weight_pre", (D,)))
    n = on.maybe(lengths, "lengths", (B,), torch.int32)
    dy = on.empty(shape) if dy is None else dy
    dresidual = on.empty(shape, f32) if dresidual is None else dresidual
    if gate is None:
        if dgate is not None:
            raise ValueError("dgate needs the gate")
    elif dgate is None:
        dgate = on.empty(shape)
    g = NormGrads(dy, dresidual, dgate, *(None if p is None else on.empty((D,), f32)
                                          for p in (scale, weight_post, weight_pre)))
    ws = on.workspace(_entry("block_norm_workspace")(B, D, L, 1))
    on.call("block_norm_backward", _NORM_BACKWARD.pack(
        on.code, B, D, L, eps, 0, *args, *on.act(dy, "dy", shape),
        *on.act(dresidual, "dresidual", shape, f32),
        *(_NONE if gate is None else on.act(dgate, "dgate", shape)), *params,
        *(0 if p is None else p.data_ptr() for p in g[3:]), n, *ws))
    return g
