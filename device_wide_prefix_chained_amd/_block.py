"""ctypes binding of the state space block's operators (``include/dwps.h``):
causal convolution, selective scan, norms around the block, with their
backward and single-token forms.  Argument marshalling only, as in
``_binding``; tensors are checked against one another, results are allocated
on the call's stream.

Activations are bfloat16, float16 or float32 tensors ``[tokens, ...]`` whose
rows may be strided (a slice of a wider projection) but are packed within;
parameters, scan states and their gradients are float32.  ``offsets`` (int32
or uint32, ``num_seqs + 1`` entries) cuts the packed tokens into sequences;
without it all tokens are one sequence.  Rows that no sequence holds are not
written, in results allocated here too.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from ._binding import (_check, _dev_tensor, _ptr, _stream, _torch_stream, _U32_DTYPES, _workspace, lib)

PS_BF16, PS_F16 = 3, 4
_TYPES = {torch.float32: 1, torch.bfloat16: PS_BF16, torch.float16: PS_F16}
_VP, _I64, _U64, _U32, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int


class _ConvInput(ctypes.Structure):
    _fields_ = [("x", _VP), ("x_stride", _I64), ("weight", _VP), ("bias", _VP), ("offsets", _VP), ("initial", _VP),
                ("tokens", _U64), ("channels", _U32), ("width", _U32), ("num_seqs", _U32), ("dtype", _I32)]


class _ScanInput(ctypes.Structure):
    _fields_ = [("x", _VP), ("dt", _VP), ("z", _VP), ("B", _VP), ("C", _VP),
                ("x_stride", _I64), ("dt_stride", _I64), ("z_stride", _I64), ("b_stride", _I64), ("c_stride", _I64),
                ("A", _VP), ("D", _VP), ("dt_bias", _VP), ("offsets", _VP), ("initial", _VP),
                ("tokens", _U64), ("channels", _U32), ("groups", _U32), ("states", _U32), ("num_seqs", _U32),
                ("dtype", _I32)]


class _ScanGrads(ctypes.Structure):
    _fields_ = [(n, _VP) for n in ("dx", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dinitial")]


class _NormInput(ctypes.Structure):
    _fields_ = [("y", _VP), ("gate", _VP), ("residual", _VP),
                ("y_stride", _I64), ("gate_stride", _I64), ("residual_stride", _I64),
                ("scale", _VP), ("post_weight", _VP), ("pre_weight", _VP),
                ("tokens", _U64), ("channels", _U32), ("dtype", _I32), ("residual_dtype", _I32), ("eps", ctypes.c_float)]


class _NormGrads(ctypes.Structure):
    _fields_ = [(n, _VP) for n in ("dy", "dgate", "dresidual", "dscale", "dpost_weight", "dpre_weight")]


class ConvGrads(NamedTuple):
    dx: torch.Tensor
    dweight: torch.Tensor
    dbias: Optional[torch.Tensor]
    dinitial: Optional[torch.Tensor]


class ScanGrads(NamedTuple):
    dx: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]
    dinitial: Optional[torch.Tensor]


class NormGrads(NamedTuple):
    dy: torch.Tensor
    dresidual: torch.Tensor
    dgate: Optional[torch.Tensor]
    dscale: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]
    dpre_weight: Optional[torch.Tensor]


_lib_ready = None


def _lib():
    global _lib_ready
    if _lib_ready is None:
        L = lib()
        P, sz = ctypes.POINTER, ctypes.POINTER(ctypes.c_size_t)
        sigs = {
            "ps_causal_conv": [P(_ConvInput), _VP, _VP, _VP],
            "ps_causal_conv_bwd": [_VP, sz, P(_ConvInput), _VP, _VP, _VP, _VP, _VP, _VP],
            "ps_causal_conv_step": [P(_ConvInput), _VP, _VP, _VP, _U32, _VP, _VP],
            "ps_selective_scan": [_VP, sz, P(_ScanInput), _VP, _VP, _VP, _VP],
            "ps_selective_scan_bwd": [_VP, sz, P(_ScanInput), _VP, _VP, P(_ScanGrads), _VP],
            "ps_selective_scan_step": [P(_ScanInput), _VP, _VP, _VP, _U32, _VP, _VP],
            "ps_block_norm": [P(_NormInput), _VP, _VP, _VP],
            "ps_block_norm_bwd": [_VP, sz, P(_NormInput), _VP, _VP, P(_NormGrads), _VP],
        }
        for name, args in sigs.items():
            getattr(L, name).argtypes = args
            getattr(L, name).restype = _I32
        L.ps_selective_scan_checkpoint_rows.argtypes = [_U64, _U32]
        L.ps_selective_scan_checkpoint_rows.restype = _U64
        _lib_ready = L
    return _lib_ready


# A call checks ten tensors or more; each check is one expression where
# nothing is wrong, and only then does _refuse look for what is.
def _refuse(name, t, like, shape, dtype):
    """Raises for a tensor that is not of like's device, `shape` and `dtype`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() != like.get_device():
        raise ValueError("%s must be on the device of the other tensors" % name)


def _row_stride(name, t):
    """Elements from row to row of an activation, packed within its rows."""
    if t.is_contiguous() and t.shape[0]:
        return t.numel() // t.shape[0]
    step = 1
    for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if s != step and n > 1:
            raise ValueError("%s must be packed within its rows" % name)
        step *= n
    # the stride of a single row (or none) says nothing
    if t.shape[0] <= 1:
        return step
    if t.stride(0) < step:
        raise ValueError("%s has rows that overlap" % name)
    return t.stride(0)


def _shape(name, t, dims, of):
    """The shape of a tensor that gives the call sizes: `dims` dimensions, `of`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != dims:
        raise ValueError("%s must be %s" % (name, of))
    return t.shape


def _first(name, t):
    """The activation the others are compared with ([tokens, channels])."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be [tokens, channels]" % name)
    return _row_stride(name, t)


def _same(name, t, like, shape, dtype=None):
    """An activation shaped `shape` of like's type and device: its row stride."""
    if dtype is None:
        dtype = like.dtype
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == like.get_device():
            return _row_stride(name, t)
    except AttributeError:
        pass
    _refuse(name, t, like, shape, dtype)


def _packed(name, t, like, shape, dtype):
    """A packed tensor (parameter, state, result) or None: its address."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == like.get_device() and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, like, shape, dtype)
    raise ValueError("%s must be contiguous" % name)


def _type_of(name, t):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s has dtype %s, expected bfloat16, float16 or float32" % (name, t.dtype))
    return code


def _sequences(offsets, like):
    """Address and number of sequences."""
    if offsets is None:
        return None, 1
    _dev_tensor("offsets", offsets, _U32_DTYPES)
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets needs num_seqs + 1 >= 1 entries")
    if offsets.get_device() != like.get_device():
        raise ValueError("offsets must be on the device of the other tensors")
    return offsets.data_ptr(), offsets.numel() - 1


def _slots(slots, like, batch, pool):
    if slots is None:
        if batch > pool:
            raise ValueError("a batch of %d rows needs slots in a pool of %d" % (batch, pool))
        return None
    _dev_tensor("slots", slots, (torch.int32,))
    if slots.dim() != 1 or slots.numel() != batch:
        raise ValueError("slots needs one entry for each row")
    if slots.get_device() != like.get_device():
        raise ValueError("slots must be on the device of the other tensors")
    return slots.data_ptr()


class _Results:
    """Allocates results on the call's stream."""

    def __init__(self, device, stream):
        self.device, self.stream = device, stream

    def __call__(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(_torch_stream(self.device, self.stream)):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def like(self, t):
        """A packed tensor of t's shape and type, or None for None."""
        if t is None:
            return None
        if self.stream is None and t.is_contiguous():
            return torch.empty_like(t)
        return self(t.shape, t.dtype)


def _addr(t):
    return None if t is None else t.data_ptr()


def _with_workspace(fn, call, like, workspace, stream):
    ws, have = _workspace(fn, call, like, workspace, stream)
    _check(fn, call(_ptr(ws), ctypes.byref(have)))


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------
def _conv_input(x, weight, bias, offsets, initial):
    f32 = torch.float32
    stride = _first("x", x)
    code = _type_of("x", x)
    tokens, channels = x.shape
    width = _shape("weight", weight, 2, "[channels, width]")[1]
    w = _packed("weight", weight, x, (channels, width), f32)
    b = _packed("bias", bias, x, (channels,), f32)
    off, seqs = _sequences(offsets, x)
    init = _packed("initial", initial, x, (seqs, width - 1, channels), x.dtype)
    return _ConvInput(x.data_ptr(), stride, w, b, off, init, tokens, channels, width, seqs, code)


def ps_causal_conv(x, weight, bias=None, *, offsets=None, initial=None, out=None, final=None, stream=None):
    """out = silu(bias + causal convolution of x with weight [channels,
    width] over each channel's past); ``initial`` and ``final`` are the width
    - 1 rows before and at the end of each sequence."""
    a = _conv_input(x, weight, bias, offsets, initial)
    o = _Results(x.device, stream).like(x) if out is None else out
    _check("ps_causal_conv", _lib().ps_causal_conv(
        a, _packed("out", o, x, x.shape, x.dtype),
        _packed("final", final, x, (a.num_seqs, a.width - 1, a.channels), x.dtype), _stream(x, stream)))
    return o


def ps_causal_conv_bwd(x, weight, dout, bias=None, *, offsets=None, initial=None, workspace=None, stream=None):
    """Gradients of ps_causal_conv's out: ConvGrads(dx, dweight, dbias,
    dinitial), the last two where there is a bias and an initial."""
    a = _conv_input(x, weight, bias, offsets, initial)
    g = _packed("dout", dout, x, x.shape, x.dtype)
    new = _Results(x.device, stream)
    r = ConvGrads(*(new.like(t) for t in (x, weight, bias, initial)))
    s, f = _stream(x, stream), _lib().ps_causal_conv_bwd
    call = lambda ws, wsb: f(ws, wsb, a, g, _addr(r.dx), _addr(r.dweight), _addr(r.dbias),  # noqa: E731
                             _addr(r.dinitial), s)
    _with_workspace("ps_causal_conv_bwd", call, x, workspace, stream)
    return r


def ps_causal_conv_step(x, state, weight, bias=None, *, slots=None, new_state=None, out=None, stream=None):
    """One token for each row of x [batch, channels]; ``state`` [pool, width
    - 1, channels] holds each sequence's last rows, row i's in slot slots[i].
    The rows after the token go to ``new_state`` (default: state itself)."""
    a = _conv_input(x, weight, bias, None, None)
    pool = _shape("state", state, 3, "[pool, width - 1, channels]")[0]
    shape = (pool, a.width - 1, a.channels)
    old = _packed("state", state, x, shape, x.dtype)
    new = old if new_state is None else _packed("new_state", new_state, x, shape, x.dtype)
    o = _Results(x.device, stream).like(x) if out is None else out
    _check("ps_causal_conv_step", _lib().ps_causal_conv_step(
        a, old, new, _slots(slots, x, a.tokens, pool), pool, _packed("out", o, x, x.shape, x.dtype),
        _stream(x, stream)))
    return o


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------
def _scan_input(x, dt, A, B, C, D, z, dt_bias, offsets, initial):
    f32 = torch.float32
    xs = _first("x", x)
    code = _type_of("x", x)
    tokens, channels = x.shape
    _, groups, states = _shape("B", B, 3, "[tokens, groups, states]")
    bc = (tokens, groups, states)
    dts = _same("dt", dt, x, x.shape)
    zs = 0 if z is None else _same("z", z, x, x.shape)
    bs, cs = _same("B", B, x, bc), _same("C", C, x, bc)
    _shape("A", A, 2, "[channels, states]")
    a = _packed("A", A, x, (channels, states), f32)
    d = _packed("D", D, x, (channels,), f32)
    db = _packed("dt_bias", dt_bias, x, (channels,), f32)
    off, seqs = _sequences(offsets, x)
    init = _packed("initial", initial, x, (seqs, channels, states), f32)
    return _ScanInput(x.data_ptr(), dt.data_ptr(), _addr(z), B.data_ptr(), C.data_ptr(), xs, dts, zs, bs, cs, a, d, db,
                      off, init, tokens, channels, groups, states, seqs, code)


def ps_selective_scan_checkpoint_rows(tokens: int, states: int) -> int:
    """Rows of the ``checkpoints`` [rows, channels, states] of a forward call
    that a backward call follows."""
    return int(_lib().ps_selective_scan_checkpoint_rows(int(tokens), int(states)))


def ps_selective_scan(x, dt, A, B, C, *, D=None, z=None, dt_bias=None, offsets=None, initial=None, out=None, final=None,
                      checkpoints=None, workspace=None, stream=None):
    """The selective scan of x with steps softplus(dt + dt_bias): out (and
    ``final`` [num_seqs, channels, states], the states after each sequence;
    ``checkpoints``, what ps_selective_scan_bwd starts from)."""
    a = _scan_input(x, dt, A, B, C, D, z, dt_bias, offsets, initial)
    f32 = torch.float32
    o = _Results(x.device, stream).like(x) if out is None else out
    to = _packed("out", o, x, x.shape, x.dtype)
    fin = _packed("final", final, x, (a.num_seqs, a.channels, a.states), f32)
    kept = None
    if checkpoints is not None:
        rows = ps_selective_scan_checkpoint_rows(a.tokens, a.states)
        kept = _packed("checkpoints", checkpoints, x, (rows, a.channels, a.states), f32)
    s, f = _stream(x, stream), _lib().ps_selective_scan
    _with_workspace("ps_selective_scan", lambda ws, wsb: f(ws, wsb, a, to, fin, kept, s), x, workspace, stream)
    return o


def ps_selective_scan_bwd(x, dt, A, B, C, dout, checkpoints, *, D=None, z=None, dt_bias=None, offsets=None, initial=None,
                          workspace=None, stream=None):
    """Gradients of ps_selective_scan's out, from the checkpoints that it wrote
    for these inputs: ScanGrads, with None for the inputs that are not given."""
    a = _scan_input(x, dt, A, B, C, D, z, dt_bias, offsets, initial)
    f32 = torch.float32
    g = _packed("dout", dout, x, x.shape, x.dtype)
    rows = ps_selective_scan_checkpoint_rows(a.tokens, a.states)
    kept = _packed("checkpoints", checkpoints, x, (rows, a.channels, a.states), f32)
    new = _Results(x.device, stream)
    r = ScanGrads(*(new.like(t) for t in (x, dt, A, B, C, D, z, dt_bias, initial)))
    grads = _ScanGrads(_addr(r.dx), _addr(r.ddt), _addr(r.dz), _addr(r.dB), _addr(r.dC), _addr(r.dA), _addr(r.dD),
                       _addr(r.ddt_bias), _addr(r.dinitial))
    s, f = _stream(x, stream), _lib().ps_selective_scan_bwd
    _with_workspace("ps_selective_scan_bwd", lambda ws, wsb: f(ws, wsb, a, g, kept, grads, s), x, workspace, stream)
    return r


def ps_selective_scan_step(x, state, dt, A, B, C, *, D=None, z=None, dt_bias=None, slots=None, new_state=None, out=None,
                           stream=None):
    """One token for each row of x [batch, channels]; ``state`` [pool,
    channels, states] in float32, row i's in slot slots[i].  The states after
    the token go to ``new_state`` (default: state itself)."""
    a = _scan_input(x, dt, A, B, C, D, z, dt_bias, None, None)
    f32 = torch.float32
    pool = _shape("state", state, 3, "[pool, channels, states]")[0]
    shape = (pool, a.channels, a.states)
    old = _packed("state", state, x, shape, f32)
    new = old if new_state is None else _packed("new_state", new_state, x, shape, f32)
    o = _Results(x.device, stream).like(x) if out is None else out
    _check("ps_selective_scan_step", _lib().ps_selective_scan_step(
        a, old, new, _slots(slots, x, a.tokens, pool), pool, _packed("out", o, x, x.shape, x.dtype), _stream(x, stream)))
    return o


# ---------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------
def _norm_input(y, residual, gate, scale, post_weight, pre_weight, eps):
    f32 = torch.float32
    ys = _first("y", y)
    code = _type_of("y", y)
    tokens, channels = y.shape
    _shape("residual", residual, 2, "[tokens, channels]")
    rt = residual.dtype
    if rt != y.dtype and rt != f32:
        raise TypeError("residual has dtype %s, expected %s or %s" % (rt, y.dtype, f32))
    rs = _same("residual", residual, y, y.shape, rt)
    gs = 0 if gate is None else _same("gate", gate, y, y.shape)
    w = (channels,)
    return _NormInput(y.data_ptr(), _addr(gate), residual.data_ptr(), ys, gs, rs, _packed("scale", scale, y, w, f32),
                      _packed("post_weight", post_weight, y, w, f32), _packed("pre_weight", pre_weight, y, w, f32),
                      tokens, channels, code, _TYPES[rt], eps)


def ps_block_norm(y, residual, *, gate=None, scale=None, post_weight=None, pre_weight=None, eps=1e-6, residual_out=None,
                  out=None, stream=None):
    """(residual + scale * sigmoid(gate) * norm(y) * post_weight, its norm *
    pre_weight): the residual stream after a block and the input of the next."""
    a = _norm_input(y, residual, gate, scale, post_weight, pre_weight, eps)
    new = _Results(y.device, stream)
    r = new.like(residual) if residual_out is None else residual_out
    o = new.like(y) if out is None else out
    _check("ps_block_norm", _lib().ps_block_norm(
        a, _packed("residual_out", r, y, y.shape, residual.dtype), _packed("out", o, y, y.shape, y.dtype),
        _stream(y, stream)))
    return r, o


def ps_block_norm_bwd(y, residual_out, dout, dresidual_out=None, *, gate=None, scale=None, post_weight=None,
                      pre_weight=None, eps=1e-6, workspace=None, stream=None):
    """Gradients of ps_block_norm from its residual_out: NormGrads, with None
    for the inputs that are not given."""
    a = _norm_input(y, residual_out, gate, scale, post_weight, pre_weight, eps)
    g = _packed("dout", dout, y, y.shape, y.dtype)
    dr = _packed("dresidual_out", dresidual_out, y, y.shape, residual_out.dtype)
    new = _Results(y.device, stream)
    r = NormGrads(*(new.like(t) for t in (y, residual_out, gate, scale, post_weight, pre_weight)))
    grads = _NormGrads(_addr(r.dy), _addr(r.dgate), _addr(r.dresidual), _addr(r.dscale), _addr(r.dpost_weight),
                       _addr(r.dpre_weight))
    s, f = _stream(y, stream), _lib().ps_block_norm_bwd
    _with_workspace("ps_block_norm_bwd", lambda ws, wsb: f(ws, wsb, a, g, dr, grads, s), y, workspace, stream)
    return r
