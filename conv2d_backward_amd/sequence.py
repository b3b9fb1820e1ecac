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
stream of the tensors' device; default: the current one), which the caller
orders after whatever produced the inputs.  Bad arguments raise ValueError or
``Conv2dGiError`` before anything is launched.  torch and the extension module
are loaded at the first call, which raises ``LibraryNotBuilt`` where the module
is missing.
"""
from __future__ import annotations

import collections
import ctypes
import importlib
import os

from . import LibraryNotBuilt, _check, load_library

__all__ = ["causal_conv", "causal_conv_backward", "causal_conv_step", "state_scan",
           "state_scan_backward", "state_scan_step", "state_scan_plan", "block_norm", "block_norm_backward",
           "ScanGrads", "NormGrads", "SCAN_CHECKPOINT"]

#: Positions between two checkpoints of ``state_scan`` (SEQ_SCAN_CHECKPOINT).
SCAN_CHECKPOINT = 128

ScanGrads = collections.namedtuple("ScanGrads", "dx ddt dA dB dC dD dz ddt_bias dstate")
NormGrads = collections.namedtuple("NormGrads", "dy dresidual dgate dscale dweight_post dweight_pre")

torch = _sequence = None  # of the first call
_binding_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_sequence.so")


def _load():
    global torch, _sequence
    if not os.path.exists(_binding_path):
        raise LibraryNotBuilt("%s is missing: build it with `python -m conv2d_backward_amd.build`" % _binding_path)
    torch = importlib.import_module("torch")  # (the extension module links with it)
    _sequence = importlib.import_module("._sequence", __package__)


# Operand kinds and uses of seq_binding.cpp.
_ACT, _ACT32, _STATES, _DENSE, _DENSE32, _INDEX = range(6)
_NEEDED, _OPTIONAL, _OUT = range(3)

#: The entries' operands in the order of their structs in sequence_ops.h.  First
#: the struct's sizes, then sizes that only shapes need; a shape names sizes, "-"
#: after one takes 1 off.
_ENTRIES = {
    "causal_conv_forward": ("B D L K silu", "", "", [
        ("x", _ACT, _NEEDED, "B D L"), ("out", _ACT, _OUT, "B D L"),
        ("weight", _DENSE32, _NEEDED, "D K"), ("bias", _DENSE32, _OPTIONAL, "D"),
        ("state", _DENSE, _OPTIONAL, "B D K-"), ("new_state", _DENSE, _OUT, "B D K-"),
        ("lengths", _INDEX, _OPTIONAL, "B")]),
    "causal_conv_backward": ("B D L K silu", "", "causal_conv_workspace B D L K", [
        ("grad_out", _ACT, _NEEDED, "B D L"), ("x", _ACT, _NEEDED, "B D L"),
        ("dx", _ACT, _OUT, "B D L"), ("weight", _DENSE32, _NEEDED, "D K"),
        ("bias", _DENSE32, _OPTIONAL, "D"), ("dw", _DENSE32, _OUT, "D K"),
        ("db", _DENSE32, _OUT, "D"), ("lengths", _INDEX, _OPTIONAL, "B")]),
    "causal_conv_step": ("B D K silu lines", "", "", [
        ("x", _ACT, _NEEDED, "B D"), ("out", _ACT, _OUT, "B D"),
        ("weight", _DENSE32, _NEEDED, "D K"), ("bias", _DENSE32, _OPTIONAL, "D"),
        ("state", _DENSE, _NEEDED, "lines D K-"), ("slots", _INDEX, _OPTIONAL, "B")]),
    "state_scan_forward": ("B D L N G softplus reserved", "marks", "", [
        ("x", _ACT, _NEEDED, "B D L"), ("dt", _ACT, _NEEDED, "B D L"),
        ("z", _ACT, _OPTIONAL, "B D L"), ("B", _STATES, _NEEDED, "B G N L"),
        ("C", _STATES, _NEEDED, "B G N L"), ("out", _ACT, _OUT, "B D L"),
        ("A", _DENSE32, _NEEDED, "D N"), ("D", _DENSE32, _OPTIONAL, "D"),
        ("dt_bias", _DENSE32, _OPTIONAL, "D"), ("state", _DENSE32, _OPTIONAL, "B D N"),
        ("new_state", _DENSE32, _OUT, "B D N"), ("checkpoints", _DENSE32, _OUT, "B D marks N"),
        ("lengths", _INDEX, _OPTIONAL, "B")]),
    "state_scan_backward": ("B D L N G softplus reserved", "marks", "state_scan_workspace B D L N G", [
        ("grad_out", _ACT, _NEEDED, "B D L"), ("x", _ACT, _NEEDED, "B D L"),
        ("dt", _ACT, _NEEDED, "B D L"), ("z", _ACT, _OPTIONAL, "B D L"),
        ("B", _STATES, _NEEDED, "B G N L"), ("C", _STATES, _NEEDED, "B G N L"),
        ("dx", _ACT, _OUT, "B D L"), ("ddt", _ACT, _OUT, "B D L"), ("dz", _ACT, _OUT, "B D L"),
        ("A", _DENSE32, _NEEDED, "D N"), ("D", _DENSE32, _OPTIONAL, "D"),
        ("dt_bias", _DENSE32, _OPTIONAL, "D"), ("checkpoints", _DENSE32, _NEEDED, "B D marks N"),
        ("grad_state", _DENSE32, _OPTIONAL, "B D N"), ("dB", _DENSE, _OUT, "B G N L"),
        ("dC", _DENSE, _OUT, "B G N L"), ("dA", _DENSE32, _OUT, "D N"), ("dD", _DENSE32, _OUT, "D"),
        ("ddt_bias", _DENSE32, _OUT, "D"), ("dstate", _DENSE32, _OUT, "B D N"),
        ("lengths", _INDEX, _OPTIONAL, "B")]),
    "state_scan_step": ("B D N G softplus lines reserved", "", "", [
        ("x", _ACT, _NEEDED, "B D"), ("dt", _ACT, _NEEDED, "B D"), ("z", _ACT, _OPTIONAL, "B D"),
        ("B", _STATES, _NEEDED, "B G N"), ("C", _STATES, _NEEDED, "B G N"),
        ("out", _ACT, _OUT, "B D"), ("A", _DENSE32, _NEEDED, "D N"), ("D", _DENSE32, _OPTIONAL, "D"),
        ("dt_bias", _DENSE32, _OPTIONAL, "D"), ("state", _DENSE32, _NEEDED, "lines D N"),
        ("slots", _INDEX, _OPTIONAL, "B")]),
    "block_norm_forward": ("B D L eps reserved", "backward", "block_norm_workspace B D L backward", [
        ("y", _ACT, _NEEDED, "B D L"), ("gate", _ACT, _OPTIONAL, "B D L"),
        ("residual", _ACT32, _NEEDED, "B D L"), ("residual_out", _ACT32, _OUT, "B D L"),
        ("out", _ACT, _OUT, "B D L"), ("scale", _DENSE32, _OPTIONAL, "D"),
        ("weight_post", _DENSE32, _OPTIONAL, "D"), ("weight_pre", _DENSE32, _OPTIONAL, "D"),
        ("lengths", _INDEX, _OPTIONAL, "B")]),
    "block_norm_backward": ("B D L eps reserved", "backward", "block_norm_workspace B D L backward", [
        ("grad_residual", _ACT32, _OPTIONAL, "B D L"), ("grad_out", _ACT, _OPTIONAL, "B D L"),
        ("y", _ACT, _NEEDED, "B D L"), ("gate", _ACT, _OPTIONAL, "B D L"),
        ("residual_out", _ACT32, _NEEDED, "B D L"), ("dy", _ACT, _OUT, "B D L"),
        ("dresidual", _ACT32, _OUT, "B D L"), ("dgate", _ACT, _OUT, "B D L"),
        ("scale", _DENSE32, _OPTIONAL, "D"), ("weight_post", _DENSE32, _OPTIONAL, "D"),
        ("weight_pre", _DENSE32, _OPTIONAL, "D"), ("dscale", _DENSE32, _OUT, "D"),
        ("dweight_post", _DENSE32, _OUT, "D"), ("dweight_pre", _DENSE32, _OUT, "D"),
        ("lengths", _INDEX, _OPTIONAL, "B")]),
}

_made = {}


def _make(name):
    if _sequence is None:
        _load()
    header, others, workspace, operands = _ENTRIES[name]
    lib = load_library()

    def address(fn):
        return ctypes.cast(getattr(lib, fn), ctypes.c_void_p).value

    sizes = (header + " " + others).split()
    scratch = workspace.split()
    names = [o[0] for o in operands]
    _made[name] = _sequence.entry(
        address(name), len(header.split()), names.index("x" if "x" in names else "y"),
        address(scratch[0]) if scratch else 0, tuple(sizes.index(s) for s in scratch[1:]),
        tuple((n, kind, use, tuple((sizes.index(d.rstrip("-")), -d.count("-")) for d in dims.split()))
              for n, kind, use, dims in operands))
    return _made[name]


def _call(name, lead, stream, sizes, operands):
    """Runs an entry: its outputs in order (a size None: the operands have it; an
    operand False: an output not wanted)."""
    entry = _made.get(name) or _make(name)
    index = lead.get_device() if isinstance(lead, torch.Tensor) else -1
    if stream is None or index < 0:
        if index < 0:  # refused by name
            out = _sequence.call(entry, 0, sizes, operands)
        elif index == torch._C._cuda_getDevice():
            out = _sequence.call(entry, torch._C._cuda_getCurrentRawStream(index), sizes, operands)
        else:
            with torch.cuda.device(index):
                out = _sequence.call(entry, torch._C._cuda_getCurrentRawStream(index), sizes, operands)
    else:
        if stream.device_index != index:
            raise ValueError("stream is on cuda:%d, the tensors are on cuda:%d" % (stream.device_index, index))
        with torch.cuda.stream(stream):  # outputs and scratch are that stream's memory
            out = _sequence.call(entry, stream.cuda_stream, sizes, operands)
        current = torch.cuda.current_stream(index)
        if stream != current and type(out) is tuple:
            # Memory of either stream is not handed out again before the other is done with it.
            for t in operands:
                if isinstance(t, torch.Tensor):
                    t.record_stream(stream)
            for t in out:
                if t is not None:
                    t.record_stream(current)
    if type(out) is int:
        _check(out)
    return out


def causal_conv(x, weight, bias=None, *, silu=True, state=None, lengths=None, want_state=False,
                out=None, stream=None):
    """Depthwise causal convolution of K taps with bias and SiLU: (y, new_state).

    x [B, D, L]; weight [D, K], bias [D] float32.  state [B, D, K-1] (x's dtype):
    the inputs before position 0, zeros by default.  lengths int32 [B]: positions
    of each sequence (y is 0 beyond).  new_state, for the next call or
    ``causal_conv_step``, is None unless want_state.
    """
    return _call("causal_conv_forward", x, stream, (None, None, None, None, bool(silu)),
                 (x, out, weight, bias, state, None if want_state else False, lengths))


def causal_conv_backward(grad_out, x, weight, bias=None, *, silu=True, lengths=None, want_dx=True,
                         want_dw=True, want_db=None, dx=None, stream=None):
    """The gradients of ``causal_conv`` from a zero state: (dx, dweight, dbias),
    each None when not wanted (dbias by default where there is a bias)."""
    if want_db is None:
        want_db = bias is not None
    return _call("causal_conv_backward", x, stream, (None, None, None, None, bool(silu)),
                 (grad_out, x, dx if want_dx else False, weight, bias, None if want_dw else False,
                  None if want_db else False, lengths))


def causal_conv_step(x, state, weight, bias=None, *, silu=True, slots=None, out=None, stream=None):
    """One position of ``causal_conv`` for every row: y [B, D] from x [B, D].

    state [lines, D, K-1] (x's dtype, contiguous) is updated in place.  slots
    int32 [B]: the line of each row (row b uses line b without); a slot outside
    the lines marks a padding row, whose y is 0 and which changes no line.
    """
    return _call("causal_conv_step", x, stream, (None, None, None, bool(silu), None),
                 (x, out, weight, bias, state, slots))[0]


def _marks(x):
    """Checkpoints of a row."""
    shape = getattr(x, "shape", ())
    if len(shape) != 3:
        raise ValueError("x must be a tensor of 3 dimensions, has %d" % len(shape))
    return -(-shape[2] // SCAN_CHECKPOINT)


def state_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, softplus=True, state=None,
               lengths=None, want_state=False, want_checkpoints=False, out=None, stream=None):
    """The selective state space scan over a prompt: (y, new_state, checkpoints).

    x, dt, z [B, D, L]; A [D, N] float32; B, C [B, G, N, L] or [B, N, L]; D (the
    skip) and dt_bias [D] float32.  h_t = exp(s_t A) h_{t-1} + s_t x_t B_t,
    y_t = C_t . h_t + D x_t, times silu(z) where z is given, with s = softplus(dt +
    dt_bias).  state [B, D, N] float32: h before position 0.  new_state and the
    checkpoints that ``state_scan_backward`` takes are None unless wanted.
    """
    return _call("state_scan_forward", x, stream,
                 (None, None, None, None, None, bool(softplus), 0, _marks(x)),
                 (x, dt, z, B, C, out, A, D, dt_bias, state, None if want_state else False,
                  None if want_checkpoints else False, lengths))


def state_scan_backward(grad_out, x, dt, A, B, C, checkpoints, D=None, z=None, dt_bias=None, *,
                        softplus=True, lengths=None, grad_state=None, want_dstate=False, dx=None,
                        ddt=None, dz=None, stream=None):
    """The gradients of ``state_scan``: a ``ScanGrads``.

    Arguments as the forward call's, with its checkpoints.  grad_state [B, D, N]:
    the gradient of new_state (zeros by default); dstate, that of state, is None
    unless wanted.  dB and dC have B's shape.  dx, ddt, dz: optional outputs.
    """
    if z is None:
        if dz is not None:
            raise ValueError("dz needs z")
        dz = False
    dx, ddt, dz, dB, dC, dA, dD, dbias, dstate = _call(
        "state_scan_backward", x, stream,
        (None, None, None, None, None, bool(softplus), 0, _marks(x)),
        (grad_out, x, dt, z, B, C, dx, ddt, dz, A, D, dt_bias, checkpoints, grad_state, None, None, None,
         False if D is None else None, False if dt_bias is None else None,
         None if want_dstate else False, lengths))
    if B.dim() == 3:
        dB, dC = dB.squeeze(1), dC.squeeze(1)
    return ScanGrads(dx, ddt, dA, dB, dC, dD, dz, dbias, dstate)


def state_scan_plan(B, D, L, N, G=1, backward=False):
    """Host-only: how ``state_scan`` or its backward deals the work of these sizes, as
    text (include/sequence_ops.h)."""
    buf = ctypes.create_string_buffer(256)
    _check(load_library().state_scan_plan(B, D, L, N, G, int(backward), buf, len(buf)))
    return buf.value.decode()


def state_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, *, softplus=True,
                    slots=None, out=None, stream=None):
    """One position of ``state_scan`` for every row: y [B, D].

    x, dt, z [B, D]; B, C [B, G, N] or [B, N]; state [lines, D, N] float32
    (contiguous) is updated in place; slots as in ``causal_conv_step``.
    """
    return _call("state_scan_step", x, stream, (None, None, None, None, bool(softplus), None, 0),
                 (x, dt, z, B, C, out, A, D, dt_bias, state, slots))[0]


def block_norm(y, residual, weight_post=None, weight_pre=None, *, gate=None, scale=None, eps=1e-6,
               lengths=None, residual_out=None, out=None, stream=None):
    """What stands between two residual blocks: (new_residual, u).

    y [B, D, L], the block's output, goes through an RMS norm over the channels
    (weight_post; without it y as it is), times sigmoid(gate) [B, D, L] and scale
    [D], into residual [B, D, L] float32; u, the next block's input in y's dtype,
    is the RMS norm of the sum (weight_pre; None without it).  residual_out may be
    the residual itself.
    """
    if weight_pre is None:
        if out is not None:
            raise ValueError("out needs weight_pre")
        out = False
    return _call("block_norm_forward", y, stream, (None, None, None, float(eps), 0, 0),
                 (y, gate, residual, residual_out, out, scale, weight_post, weight_pre, lengths))


def block_norm_backward(grad_residual, grad_out, y, residual_out, weight_post=None, weight_pre=None,
                        *, gate=None, scale=None, eps=1e-6, lengths=None, dy=None, dresidual=None,
                        dgate=None, stream=None):
    """The gradients of ``block_norm``: a ``NormGrads`` (None where there is no input).

    grad_residual (float32) is the gradient of new_residual, grad_out that of u;
    either may be None.  residual_out: the forward call's new_residual.
    """
    if gate is None:
        if dgate is not None:
            raise ValueError("dgate needs the gate")
        dgate = False
    return NormGrads(*_call(
        "block_norm_backward", y, stream, (None, None, None, float(eps), 0, 1),
        (grad_residual, grad_out, y, gate, residual_out, dy, dresidual, dgate, scale, weight_post,
         weight_pre, False if scale is None else None, False if weight_post is None else None,
         False if weight_pre is None else None, lengths)))
