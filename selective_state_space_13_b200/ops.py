"""Python binding of the C ABI in include/selective_scan_ops.h: the operators around the scan.

The functions carry the C names -- selective_scan_bwd, gated_recurrence_fwd, gated_recurrence_bwd,
selective_scan_step, selective_state_store, selective_state_load -- and only marshal arguments:
they check shapes, dtypes and devices, allocate outputs and workspaces that the caller did not pass
(from PyTorch's allocator, on the current stream) and call the library on the current CUDA stream
of the tensors' device, which has to be the current device.  Outputs, and what is updated in place,
must not overlap inputs.  selective_scan and gated_recurrence wrap forward and gradient for
torch.autograd.  There is no CPU path.

A training step through those two can be captured into a CUDA graph after one eager step.  Nothing
of an eager graph of the same leaves (an output or loss of theirs) may then be alive: PyTorch keeps
a leaf's accumulation node, and with it the eager stream, for as long as such a graph lives, a
captured backward pass would wait for that uncaptured stream, and PyTorch ends the process.  Delete
the eager outputs first, or capture with detached leaves of the same storage.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import scan as _scan
from .scan import (SS_DIR_FWD, SS_DIR_REV, SS_FLAG_PARAMS_PER_DIRECTION, SS_FLAG_U_PER_DIRECTION,
                   SS_MAX_CONV_WIDTH, SS_MAX_DIRS, SS_OK, ScanError, SsDirectionMap, SsLaunchOpts,
                   SsShape, _io_code, make_dirmap, make_opts, make_shape)

SS_GATE_SIGMOID, SS_GATE_EXP = 0, 1
GATE_FORMS = {"sigmoid": SS_GATE_SIGMOID, "exp": SS_GATE_EXP}

EXPORTED = ("gated_recurrence_workspace_size", "gated_recurrence_fwd", "gated_recurrence_bwd",
            "selective_scan_bwd_workspace_size", "selective_scan_bwd", "selective_scan_step",
            "selective_state_store", "selective_state_load")

_F32, _I32, _I8 = torch.float32, torch.int32, torch.int8


class SsRecurrenceOpts(ctypes.Structure):
    _fields_ = [("form", ctypes.c_int32), ("complement", ctypes.c_int32), ("dir", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class SsScanGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("du", "ddelta", "dA", "dB", "dC", "dDskip", "dz",
                                               "ddelta_bias", "dinitial_state")]


_lib = None


def load():
    """The library with the signatures of this header declared."""
    global _lib
    if _lib is None:
        lib = _scan.load()
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        shape, rec = ctypes.POINTER(SsShape), ctypes.POINTER(SsRecurrenceOpts)
        dmap, opts = ctypes.POINTER(SsDirectionMap), ctypes.POINTER(SsLaunchOpts)
        signatures = {
            "gated_recurrence_workspace_size": [shape, rec, i32, ctypes.POINTER(sz)],
            "gated_recurrence_fwd": [shape, rec] + [vp] * 7 + [sz, vp],
            "gated_recurrence_bwd": [shape, rec] + [vp] * 12 + [sz, vp],
            "selective_scan_bwd_workspace_size": [shape, dmap, opts, ctypes.POINTER(sz)],
            "selective_scan_bwd": [shape] + [vp] * 8 + [i32, dmap, vp, vp,
                                                       ctypes.POINTER(SsScanGrads), vp, sz, vp, opts],
            "selective_scan_step": [shape, i64] + [vp] * 8 + [i32] + [vp] * 4 + [i32, vp, vp, vp],
            "selective_state_store": [i64, i64, i64, i32, vp, i64, vp, vp, vp, i64, vp, vp],
            "selective_state_load": [i64, i64, i64, i32, vp, vp, i64, vp, vp, i64, vp, vp],
        }
        for name, args in signatures.items():
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = args
        _lib = lib
    return _lib


def _check(device, *tensors):
    """Each (name, tensor, shape, dtype) is what the C call relies on; a tensor may be None."""
    index = device.index
    for name, t, shape, dtype in tensors:
        if t is None or (t.shape == shape and t.dtype is dtype and t.get_device() == index and
                         t.is_contiguous()):
            continue
        if t.device != device:
            raise ValueError("%s must be a CUDA tensor on %s" % (name, device))
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        if t.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        raise ValueError("%s must be contiguous" % name)


def _device_of(t, name):
    """The device of a CUDA tensor, which has to be the current one: the library launches there."""
    device = t.device
    if device.type != "cuda":
        raise ValueError("%s must be a CUDA tensor" % name)
    if device.index != torch.cuda.current_device():
        raise ValueError("%s is on %s, which is not the current device" % (name, device))
    return device


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    # (the stream object of torch.cuda.current_stream costs 2 us, half of a small call)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _done(status, what):
    if status != SS_OK:
        raise ScanError(status, what)


# ----------------------------------------------------------------------------- gated recurrence

def _recurrence_args(x, gate, gate_bias, initial_state, form, complement, reverse):
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, D]")
    if form not in GATE_FORMS:
        raise ValueError("form must be one of %s, got %r" % (sorted(GATE_FORMS), form))
    if form == "exp" and gate_bias is not None:
        raise ValueError("gate_bias belongs to the sigmoid form")
    io = _io_code(x.dtype)
    device = _device_of(x, "x")
    b, L, D = x.shape
    _check(device, ("x", x, (b, L, D), x.dtype), ("gate", gate, (b, L, D), x.dtype),
           ("gate_bias", gate_bias, (D,), _F32), ("initial_state", initial_state, (b, D), _F32))
    opts = SsRecurrenceOpts(GATE_FORMS[form], 1 if complement else 0,
                            SS_DIR_REV if reverse else SS_DIR_FWD, 0)
    return device, SsShape(b, L, D, 1, io, 0), opts, (b, L, D)


def gated_recurrence_workspace_size(shape: SsShape, opts: SsRecurrenceOpts, backward: bool) -> int:
    n = ctypes.c_size_t(0)
    _done(load().gated_recurrence_workspace_size(ctypes.byref(shape), ctypes.byref(opts),
                                                 int(bool(backward)), ctypes.byref(n)),
          "gated_recurrence_workspace_size")
    return n.value


@functools.lru_cache(maxsize=1024)
def _recurrence_workspace(b, L, D, io, form, backward):
    """The size goes by the sizes alone: asked once for each."""
    return gated_recurrence_workspace_size(SsShape(b, L, D, 1, io, 0),
                                           SsRecurrenceOpts(form, 0, SS_DIR_FWD, 0), backward)


def _workspace(nbytes, device):
    """Scratch of one call, from the caching allocator: freed into the current stream's pool, so
    calls on other streams and captured graphs never share it while it is in use."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def gated_recurrence_fwd(x, gate, gate_bias=None, initial_state=None, form="sigmoid",
                         complement=False, reverse=False, out=None, last_state=None,
                         return_last_state=False):
    """h_t = a_t h_{t-1} + c_t x_t along the sequence, elementwise per channel.

    x, gate: [batch, L, D] float32 or bfloat16.  form "sigmoid": a = sigmoid(gate + gate_bias),
    gate_bias [D] float32 or None; form "exp": a = exp(gate).  complement: c = 1 - a (a leaky
    average), else c = 1.  reverse: from the last step to the first.  initial_state: [batch, D]
    float32 (None = zero).  Returns out [batch, L, D] (every state, in x's dtype), or (out,
    last_state [batch, D] float32) with return_last_state.
    """
    device, shape, opts, (b, L, D) = _recurrence_args(x, gate, gate_bias, initial_state, form,
                                                      complement, reverse)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check(device, ("out", out, (b, L, D), x.dtype))
    if last_state is not None:
        _check(device, ("last_state", last_state, (b, D), _F32))
    elif return_last_state:
        last_state = torch.empty((b, D), dtype=_F32, device=device)
    n = _recurrence_workspace(b, L, D, shape.io_dtype, opts.form, False)
    ws = _workspace(n, device)
    _done(load().gated_recurrence_fwd(ctypes.byref(shape), ctypes.byref(opts), x.data_ptr(),
                                      gate.data_ptr(), _ptr(gate_bias), _ptr(initial_state),
                                      out.data_ptr(), _ptr(last_state), _ptr(ws), n,
                                      _stream(device)), "gated_recurrence_fwd")
    return (out, last_state) if return_last_state else out


def gated_recurrence_bwd(dout, x, gate, out, gate_bias=None, initial_state=None, dlast_state=None,
                         form="sigmoid", complement=False, reverse=False):
    """Gradients through gated_recurrence_fwd: (dx, dgate, dgate_bias, dinitial_state), the last
    two None where their input is.  out is the forward call's output; dout [batch, L, D] in x's
    dtype; dlast_state [batch, D] float32 or None, the gradient of the last state."""
    device, shape, opts, (b, L, D) = _recurrence_args(x, gate, gate_bias, initial_state, form,
                                                      complement, reverse)
    _check(device, ("out", out, (b, L, D), x.dtype), ("dout", dout, (b, L, D), x.dtype),
           ("dlast_state", dlast_state, (b, D), _F32))
    dx, dgate = torch.empty_like(x), torch.empty_like(x)
    dbias = None if gate_bias is None else torch.empty_like(gate_bias)
    dinit = None if initial_state is None else torch.empty_like(initial_state)
    n = _recurrence_workspace(b, L, D, shape.io_dtype, opts.form, True)
    ws = _workspace(n, device)
    _done(load().gated_recurrence_bwd(ctypes.byref(shape), ctypes.byref(opts), x.data_ptr(),
                                      gate.data_ptr(), _ptr(gate_bias), _ptr(initial_state),
                                      out.data_ptr(), dout.data_ptr(), _ptr(dlast_state),
                                      dx.data_ptr(), dgate.data_ptr(), _ptr(dbias), _ptr(dinit),
                                      _ptr(ws), n, _stream(device)), "gated_recurrence_bwd")
    return dx, dgate, dbias, dinit


# ----------------------------------------------------------------------------- gradient of the scan

def selective_scan_bwd_workspace_size(shape: SsShape, dmap: SsDirectionMap | None = None,
                                      opts: SsLaunchOpts | None = None) -> int:
    n = ctypes.c_size_t(0)
    _done(load().selective_scan_bwd_workspace_size(
        ctypes.byref(shape), ctypes.byref(dmap) if dmap is not None else None,
        ctypes.byref(opts) if opts is not None else None, ctypes.byref(n)),
        "selective_scan_bwd_workspace_size")
    return n.value


@functools.lru_cache(maxsize=1024)
def _bwd_workspace(batch, L, D, N, io, dirs, H, W, segments, flags, initial):
    """The size goes by the sizes and options alone (of the initial state only whether there is
    one): asked once for each."""
    return selective_scan_bwd_workspace_size(make_shape(batch, L, D, N, io), make_dirmap(dirs, H, W),
                                             make_opts(segments, flags, None, 16 if initial else 0))


def selective_scan_bwd(dout, u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                       dirs=(SS_DIR_FWD,), H=0, W=0, initial_state=None, dlast_state=None,
                       segments=0, flags=0):
    """Gradients through selective_scan_fwd of the same arguments.

    dout: [batch, L, D] in u's dtype; dlast_state: [K, batch, D, N] float32 or None, the gradient of
    last_state.  Returns a dict of du, ddelta, dA, dB, dC, dD, dz, ddelta_bias, dinitial_state, each
    with the shape and dtype of its input and None where the input is None.  The exact ZOH, int8
    delta and the fused convolution have no gradient here.
    """
    K = len(dirs)
    # (the C call refuses int8 delta with its flag)
    _scan._check_flags(int(flags) & ~_scan.SS_FLAG_DELTA_INT8, K, u, delta, A)
    device = _device_of(u, "u")
    if not 1 <= K <= SS_MAX_DIRS:
        raise ValueError("1 to %d directions, got %d" % (SS_MAX_DIRS, K))
    if u.dim() == 4 and u.shape[0] == K:
        flags = int(flags) | SS_FLAG_U_PER_DIRECTION
    elif u.dim() != 3:
        raise ValueError("u must be [batch, L, D] or [K, batch, L, D]")
    batch, L, Dm = u.shape[-3:]
    N = A.shape[-1]
    lead = (K,) if delta.dim() == 4 else ()
    if K > 1 and not lead:
        raise ValueError("delta must be [K, batch, L, D]")
    leadB, leadC = (K,) if B.dim() == 4 else (), (K,) if C.dim() == 4 else ()
    if K > 1 and not (leadB and leadC):
        raise ValueError("B and C must be [K, batch, L, N]")
    pshape = (Dm,)
    if A.dim() == 3:
        flags = int(flags) | SS_FLAG_PARAMS_PER_DIRECTION
        pshape = (K, Dm)
    io = u.dtype
    code = _io_code(io)
    rows = (batch, L, Dm)
    _check(device, ("u", u, u.shape, io), ("delta", delta, lead + rows, io),
           ("B", B, leadB + (batch, L, N), io), ("C", C, leadC + (batch, L, N), io),
           ("z", z, rows, io), ("dout", dout, rows, io), ("A", A, pshape + (N,), _F32),
           ("D", D, pshape, _F32), ("delta_bias", delta_bias, pshape, _F32),
           ("initial_state", initial_state, (K, batch, Dm, N), _F32),
           ("dlast_state", dlast_state, (K, batch, Dm, N), _F32))

    def like(t):
        return None if t is None else torch.empty_like(t)

    r = dict(du=like(u), ddelta=like(delta), dA=like(A), dB=like(B), dC=like(C), dD=like(D),
             dz=like(z), ddelta_bias=like(delta_bias), dinitial_state=like(initial_state))
    grads = SsScanGrads(*(_ptr(t) for t in r.values()))
    shape = make_shape(batch, L, Dm, N, code)
    dmap = make_dirmap(dirs, H, W)
    opts = make_opts(segments, flags, None, _ptr(initial_state) or 0)
    n = _bwd_workspace(batch, L, Dm, N, code, tuple(dirs), H, W, segments, flags,
                       initial_state is not None)
    ws = _workspace(n, device)
    _done(load().selective_scan_bwd(
        ctypes.byref(shape), u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(),
        C.data_ptr(), _ptr(D), _ptr(z), _ptr(delta_bias), int(bool(softplus)), ctypes.byref(dmap),
        dout.data_ptr(), _ptr(dlast_state), ctypes.byref(grads), _ptr(ws), n, _stream(device),
        ctypes.byref(opts)), "selective_scan_bwd")
    return r


# ----------------------------------------------------------------------------- single-token step

def selective_scan_step(u, delta, A, B, C, state, D=None, z=None, delta_bias=None, softplus=True,
                        slots=None, conv_weight=None, conv_bias=None, conv_state=None, out=None):
    """One token of the forward scan per row, on states in a pool that is updated in place.

    u, delta, z: [batch, D]; B, C: [batch, N] (one dtype, float32 or bfloat16); A: [D, N], D and
    delta_bias: [D] float32.  state: [num_slots, D, N] float32.  slots: [batch] int32 or None (row r
    uses slot r); a row whose slot is outside the pool is padding and changes nothing, and of rows
    that name one slot the lowest takes it.  conv_weight: [D, width] float32 (width <= 4) with
    conv_bias [D] or None and conv_state [num_slots, width - 1, D], the last inputs, oldest first,
    shifted in place.  Returns out [batch, D]; rows that are padding keep what out held (zero when
    it is allocated here).
    """
    device = _device_of(u, "u")
    if u.dim() != 2:
        raise ValueError("u must be [batch, D]")
    batch, Dm = u.shape
    N = A.shape[-1]
    io = u.dtype
    code = _io_code(io)
    if state.dim() != 3:
        raise ValueError("state must be [num_slots, D, N]")
    num_slots = state.shape[0]
    row, group, channel = (batch, Dm), (batch, N), (Dm,)
    _check(device, ("u", u, row, io), ("delta", delta, row, io), ("B", B, group, io),
           ("C", C, group, io), ("z", z, row, io), ("A", A, (Dm, N), _F32), ("D", D, channel, _F32),
           ("delta_bias", delta_bias, channel, _F32), ("state", state, (num_slots, Dm, N), _F32),
           ("slots", slots, (batch,), _I32), ("out", out, row, io))
    width = 0
    if conv_weight is not None:
        width = conv_weight.shape[-1]
        if not 1 <= width <= SS_MAX_CONV_WIDTH:
            raise ValueError("conv_weight must be [D, width] with 1 to %d taps" % SS_MAX_CONV_WIDTH)
        if conv_state is None and width > 1:
            raise ValueError("conv_weight needs conv_state")
        _check(device, ("conv_weight", conv_weight, (Dm, width), _F32),
               ("conv_bias", conv_bias, channel, _F32),
               ("conv_state", conv_state, (num_slots, width - 1, Dm), io))
    elif conv_bias is not None or conv_state is not None:
        raise ValueError("conv_bias and conv_state need conv_weight")
    if out is None:
        out = torch.zeros_like(u) if slots is not None else torch.empty_like(u)
    _done(load().selective_scan_step(
        ctypes.byref(SsShape(batch, 1, Dm, N, code, 0)), num_slots, u.data_ptr(), delta.data_ptr(),
        A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z), _ptr(delta_bias),
        1 if softplus else 0, state.data_ptr(), _ptr(slots), _ptr(conv_weight), _ptr(conv_bias),
        width, _ptr(conv_state), out.data_ptr(), _stream(device)), "selective_scan_step")
    return out


# ----------------------------------------------------------------------------- parked states

def _state_args(state, codes, scales, bits, src_slots, dst_slots, src_pool, dst_pool):
    device = _device_of(state, "state")
    if bits not in (4, 8):
        raise ValueError("bits must be 8 or 4, got %r" % (bits,))
    if state.dim() != 3 or codes.dim() != 3:
        raise ValueError("state and codes must be [slots, D, ...]")
    slots, Dm, N = state.shape
    parked = codes.shape[0]
    _check(device, ("state", state, (slots, Dm, N), _F32), ("scales", scales, (parked, Dm), _F32),
           ("codes", codes, (parked, Dm, N if bits == 8 else (N + 1) // 2), _I8))
    rows = None
    for t, name in ((src_slots, "src_slots"), (dst_slots, "dst_slots")):
        if t is not None:
            if t.dim() != 1:
                raise ValueError("%s must be [rows]" % name)
            if rows is not None and t.shape[0] != rows:
                raise ValueError("src_slots and dst_slots must have one length")
            rows = t.shape[0]
            _check(device, (name, t, (rows,), _I32))
    if rows is None:
        rows = src_pool.shape[0]
    return device, rows, Dm, N, slots, parked


def selective_state_store(state, codes, scales, bits=8, src_slots=None, dst_slots=None):
    """Park states in 8 or 4 bits: row r quantises state[src_slots[r]] into codes[dst_slots[r]] and
    scales[dst_slots[r]], one scale per channel.

    state: [state_slots, D, N] float32; codes: [cache_slots, D, N] int8 (bits 8) or
    [cache_slots, D, (N + 1) // 2] int8 (bits 4, two codes a byte); scales: [cache_slots, D] float32;
    slots: [rows] int32 or None (row r uses slot r; rows then is the other list's length, or all
    source slots).  Rows with a slot outside its pool are skipped; of rows with one destination the
    lowest is taken.
    """
    device, rows, Dm, N, slots, parked = _state_args(state, codes, scales, bits, src_slots,
                                                     dst_slots, state, codes)
    _done(load().selective_state_store(rows, Dm, N, bits, state.data_ptr(), slots, _ptr(src_slots),
                                       codes.data_ptr(), scales.data_ptr(), parked,
                                       _ptr(dst_slots), _stream(device)), "selective_state_store")


def selective_state_load(codes, scales, state, bits=8, src_slots=None, dst_slots=None):
    """Read parked states back: row r writes codes[src_slots[r]] * scales[src_slots[r]] to
    state[dst_slots[r]].  Arguments as in selective_state_store."""
    device, rows, Dm, N, slots, parked = _state_args(state, codes, scales, bits, src_slots,
                                                     dst_slots, codes, state)
    _done(load().selective_state_load(rows, Dm, N, bits, codes.data_ptr(), scales.data_ptr(), parked,
                                      _ptr(src_slots), state.data_ptr(), slots, _ptr(dst_slots),
                                      _stream(device)), "selective_state_load")


# ----------------------------------------------------------------------------- autograd

def _incoming(grad):
    """A gradient as the library reads it: dense, from a 16-byte border on (autograd hands out views
    that may start anywhere)."""
    if grad is None:
        return None
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, initial_state, softplus, dirs, H, W):
        out, last = _scan.selective_scan_fwd(
            u, delta, A, B, C, D=D, z=z, delta_bias=delta_bias, softplus=softplus, dirs=dirs, H=H,
            W=W, initial_state=initial_state, return_last_state=True)
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, initial_state)
        ctx.set_materialize_grads(False)
        ctx.call = dict(softplus=softplus, dirs=dirs, H=H, W=W)
        return out, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dlast):
        u, delta, A, B, C, D, z, delta_bias, initial_state = ctx.saved_tensors
        if dout is None and dlast is None:
            return (None,) * 13
        dout = u.new_zeros(u.shape[-3:]) if dout is None else _incoming(dout)
        g = selective_scan_bwd(dout, u, delta, A, B, C, D=D, z=z, delta_bias=delta_bias,
                               initial_state=initial_state, dlast_state=_incoming(dlast),
                               **ctx.call)
        return tuple(g[n] for n in ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias",
                                    "dinitial_state")) + (None,) * 4


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                   dirs=(SS_DIR_FWD,), H=0, W=0, initial_state=None):
    """selective_scan_fwd with a gradient: (out, last_state), differentiable in every tensor."""
    return _SelectiveScan.apply(u, delta, A, B, C, D, z, delta_bias, initial_state, softplus,
                                tuple(dirs), H, W)


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, gate_bias, initial_state, form, complement, reverse):
        out, last = gated_recurrence_fwd(x, gate, gate_bias=gate_bias, initial_state=initial_state,
                                         form=form, complement=complement, reverse=reverse,
                                         return_last_state=True)
        ctx.save_for_backward(x, gate, gate_bias, initial_state, out)
        ctx.set_materialize_grads(False)
        ctx.call = dict(form=form, complement=complement, reverse=reverse)
        return out, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dlast):
        x, gate, gate_bias, initial_state, out = ctx.saved_tensors
        if dout is None and dlast is None:
            return (None,) * 7
        dout = torch.zeros_like(x) if dout is None else _incoming(dout)
        return gated_recurrence_bwd(dout, x, gate, out, gate_bias=gate_bias,
                                    initial_state=initial_state, dlast_state=_incoming(dlast),
                                    **ctx.call) + (None,) * 3


def gated_recurrence(x, gate, gate_bias=None, initial_state=None, form="sigmoid", complement=False,
                     reverse=False):
    """gated_recurrence_fwd with a gradient: (out, last_state), differentiable in every tensor."""
    return _GatedRecurrence.apply(x, gate, gate_bias, initial_state, form, complement, reverse)
