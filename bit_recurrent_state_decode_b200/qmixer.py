"""Thin ctypes binding of the C ABI in include/qmixer.h (libqmixer.so): the
operators around the recurrent state of a Mamba2 layer.

    conv, conv_step      the short causal convolution of a prompt / of one token
    scan, scan_step      the selective scan of a prompt / of one token, binary32 states
    load                 a prompt's binary32 states into a low-bit ``qstate.QState``
    step                 the selective step of one token on a ``qstate.QState``
    norm                 root-mean-square norm, with a residual or a gate, and 8-bit output

Argument checks and marshalling only: the arithmetic runs in the CUDA kernels
of the library.  Calls are asynchronous on the current stream of the tensors'
device, or on `stream`; tensors of another stream have to be ordered before
the call by the caller, as for any PyTorch operator.  The library must have
been built; there is no CPU fallback and no autograd: inputs that require a
gradient are refused while gradients are recorded.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import qstate as Q
from .qstate import QStateError

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqmixer.so")

INITIAL, SILU, SOFTPLUS = 1, 2, 4
BEFORE_NONE, BEFORE_RESIDUAL, BEFORE_GATE = 0, 1, 2
OUT_SAME, OUT_INT8, OUT_E4M3 = 0, 1, 2

# every symbol include/qmixer.h declares
EXPORTS = ("qmixer_conv", "qmixer_conv_step", "qmixer_scan", "qmixer_scan_workspace", "qmixer_scan_step",
           "qmixer_step_operands", "qmixer_step_output", "qmixer_norm", "qmixer_quantize")

_lib = None


def lib():
    """Load libqmixer.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_recurrent_state_decode_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, L64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        row = [P, L64]
        L.qmixer_conv.argtypes = row + [P, P, P] + row + [P, I, L64, I, I, I, I, P]
        L.qmixer_conv_step.argtypes = row + [P, P, P] + row + [I, I, I, I, I, P]
        ops = row + row + [P] + row + row
        L.qmixer_scan.argtypes = ops + [P, P, P] + row + [P, I, L64, I, I, I, I, I, I, I, P, L64, P]
        L.qmixer_scan_workspace.argtypes = [I, L64, I, I, I, I, I]
        L.qmixer_scan_step.argtypes = ops + [P, P, P] + row + [I, I, I, I, I, I, I, I, P]
        L.qmixer_step_operands.argtypes = ops + [P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, P]
        L.qmixer_step_output.argtypes = [P] + row + [P] + row + [I, I, I, I, P]
        L.qmixer_norm.argtypes = row + row + [P] + row + [P, L64, I, I, F, I, I, I, P]
        L.qmixer_quantize.argtypes = [P, P, P, P, L64, I, I, I, I, P, I, I, I, P]
        for name in EXPORTS:
            getattr(L, name).restype = I
        L.qmixer_scan_workspace.restype = L64
        _lib = L
    return _lib


def _check(fn, rc):
    if rc != Q.OK:
        raise QStateError(fn, rc)


# ---------------------------------------------------------------- argument checks
_CODE = {torch.float32: Q.F32, torch.bfloat16: Q.BF16}


def _tensor(fn, name, t, like=None, dtype=None, shape=None):
    """A CUDA tensor of the given device, type and shape that no gradient is wanted for."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor")
    if like is not None and t.device != like.device:
        raise ValueError(f"{fn}: {name} is on {t.device}, not on {like.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{fn}: {name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {shape}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{fn}: {name} requires a gradient, and {fn} has no backward pass")
    return t


def _dense(fn, name, t, like, dtype, shape):
    _tensor(fn, name, t, like, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous")
    return t


def _rows(fn, name, t, inner):
    """(address, stride between rows) of a tensor whose last `inner` dimensions are
    contiguous and whose leading ones, where there are two, walk in one stride."""
    step = 1
    for d in range(t.dim() - 1, t.dim() - 1 - inner, -1):
        if t.shape[d] != 1 and t.stride(d) != step:
            raise ValueError(f"{fn}: the elements of a row of {name} must be contiguous")
        step *= t.shape[d]
    lead = t.dim() - inner
    n = t.shape[lead - 1]
    stride = t.stride(lead - 1) if n > 1 else step
    if lead == 2 and t.shape[0] > 1:
        if n == 1:
            stride = t.stride(0)
        elif n and t.stride(0) != n * stride:
            raise ValueError(f"{fn}: the sequences of {name} must lie one behind the other")
    return t.data_ptr(), max(stride, step) if t.numel() == 0 or lead == 0 else stride


def _overlap(fn, name, a, other, b):
    """Refuse an output that shares memory with an input."""
    if a.numel() and b.numel():
        a0, b0 = a.data_ptr(), b.data_ptr()
        if a0 < b0 + _span(b) and b0 < a0 + _span(a):
            # rows of one buffer may interleave without sharing an element
            if not _interleaved(a, b):
                raise ValueError(f"{fn}: {name} overlaps {other}")


def _span(t):
    return (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))) * t.element_size()


def _interleaved(a, b):
    """Two views of rows of one pitch whose columns are apart."""
    pa, pb = a.stride(0) * a.element_size(), b.stride(0) * b.element_size()
    if pa != pb or a.dim() < 2 or b.dim() < 2:
        return False
    wa = _span(a[0]) if a.shape[0] else 0
    wb = _span(b[0]) if b.shape[0] else 0
    off = (b.data_ptr() - a.data_ptr()) % pa if pa else 0
    return off >= wa and off + wb <= pa


def _code(fn, t):
    c = _CODE.get(t.dtype)
    if c is None:
        raise ValueError(f"{fn}: dtype {t.dtype} is not float32 or bfloat16")
    return c


def _ptr(t):
    return None if t is None else t.data_ptr()


class _On:
    """The device of `t` and the stream to launch on; allocations inside belong to that stream."""

    def __init__(self, t, stream):
        i = t.device.index
        self.guard = self.side = None
        if i != torch.cuda.current_device():
            self.guard = torch.cuda.device(i)
        if stream is None:
            self.stream = None
        else:
            if stream.device.index != i:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
            self.side = torch.cuda.stream(stream)
        self.index = i

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        if self.side is not None:
            self.side.__enter__()
        return torch.cuda.current_stream(self.index).cuda_stream

    def __exit__(self, *a):
        if self.side is not None:
            self.side.__exit__(*a)
        if self.guard is not None:
            self.guard.__exit__(*a)


def _sequences(fn, lead, seq_starts, like):
    """(sequences, tokens, address of seq_starts) of a prompt's leading dimensions."""
    if len(lead) == 2:
        if seq_starts is not None:
            raise ValueError(f"{fn}: seq_starts goes with tokens in one axis, not with a batch of equal sequences")
        return lead[0], lead[0] * lead[1], None
    if seq_starts is None:
        return 1, lead[0], None
    _tensor(fn, "seq_starts", seq_starts, like, torch.int32)
    if seq_starts.dim() != 1 or seq_starts.numel() < 1 or not seq_starts.is_contiguous():
        raise ValueError(f"{fn}: seq_starts must be a contiguous vector of the sequences' first tokens and their end")
    return seq_starts.numel() - 1, lead[0], seq_starts.data_ptr()


def _out(fn, out, like, shape, dtype, inputs):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _tensor(fn, "out", out, like, dtype, tuple(shape))
    for name, t in inputs:
        if t is not None:
            _overlap(fn, "out", out, name, t)
    return out


# ---------------------------------------------------------------- convolution
def conv(x, weight, bias=None, *, state=None, initial=False, seq_starts=None, activation=True, out=None,
         stream=None):
    """Causal convolution of a prompt, channel by channel, and its SiLU.

    x [batch, length, channels], or [tokens, channels] with the sequences one
    behind the other from seq_starts (int32 [n + 1], on the device; None: one
    sequence).  weight [channels, width], width 2 to 4; bias [channels].  state
    [n, width - 1, channels], oldest token first: each sequence continues from
    its row with initial=True, else from zeros, and leaves its last rows there.
    Tokens behind the last sequence stay as they are in `out` (undefined where
    `out` is not given).  Returns out, shaped like x."""
    fn = "conv"
    _tensor(fn, "x", x)
    if x.dim() not in (2, 3):
        raise ValueError(f"{fn}: x must be [batch, length, channels] or [tokens, channels]")
    code = _code(fn, x)
    n, tokens, starts = _sequences(fn, x.shape[:-1], seq_starts, x)
    channels = x.shape[-1]
    width = _taps(fn, x, weight, bias, state, n)
    if initial and state is None:
        raise ValueError(f"{fn}: initial=True needs the state to continue from")
    xp, xs = _rows(fn, "x", x, 1)
    with _On(x, stream) as st:
        y = _out(fn, out, x, x.shape, x.dtype, (("x", x), ("state", state), ("weight", weight), ("bias", bias)))
        yp, ys = _rows(fn, "out", y, 1)
        _check("qmixer_conv", lib().qmixer_conv(
            xp, xs, weight.data_ptr(), _ptr(bias), _ptr(state), yp, ys, starts, n, tokens, channels, width, code,
            (INITIAL if initial else 0) | (SILU if activation else 0), st))
    return y


def conv_step(x, weight, bias=None, *, state, activation=True, out=None, stream=None):
    """The same for one token of each sequence: x [batch, channels]; state
    [batch, width - 1, channels] moves on by one token."""
    fn = "conv_step"
    _tensor(fn, "x", x)
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be [batch, channels]")
    code = _code(fn, x)
    if state is None:
        raise ValueError(f"{fn}: state is required")
    width = _taps(fn, x, weight, bias, state, x.shape[0])
    xp, xs = _rows(fn, "x", x, 1)
    with _On(x, stream) as st:
        y = _out(fn, out, x, x.shape, x.dtype, (("x", x), ("state", state), ("weight", weight), ("bias", bias)))
        yp, ys = _rows(fn, "out", y, 1)
        _check("qmixer_conv_step", lib().qmixer_conv_step(
            xp, xs, weight.data_ptr(), _ptr(bias), _ptr(state), yp, ys, x.shape[0], x.shape[1], width, code,
            SILU if activation else 0, st))
    return y


def _taps(fn, x, weight, bias, state, n):
    channels = x.shape[-1]
    _tensor(fn, "weight", weight, x, x.dtype)
    if weight.dim() != 2 or weight.shape[0] != channels or not weight.is_contiguous():
        raise ValueError(f"{fn}: weight must be contiguous [channels, width]")
    width = weight.shape[1]
    if bias is not None:
        _dense(fn, "bias", bias, x, x.dtype, (channels,))
    if state is not None:
        _dense(fn, "state", state, x, x.dtype, (n, width - 1, channels))
        _overlap(fn, "state", state, "x", x)
    return width


# ---------------------------------------------------------------- selective scan
def _selective(fn, x, dt, A, B, C, D, dt_bias):
    _tensor(fn, "x", x)
    code = _code(fn, x)
    lead, (heads, d_v) = tuple(x.shape[:-2]), x.shape[-2:]
    _tensor(fn, "dt", dt, x, None, lead + (heads,))
    dt_code = _code(fn, dt)
    _tensor(fn, "B", B, x, x.dtype)
    if B.dim() != x.dim() or tuple(B.shape[:-2]) != lead:
        raise ValueError(f"{fn}: B has shape {tuple(B.shape)}, expected {lead} + (groups, d_k)")
    groups, d_k = B.shape[-2:]
    _tensor(fn, "C", C, x, x.dtype, tuple(B.shape))
    if groups == 0 or heads % groups:
        raise ValueError(f"{fn}: {heads} heads do not divide into {groups} groups")
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias)):
        if t is not None or name == "A":
            _dense(fn, name, t, x, torch.float32, (heads,))
    rows = (*_rows(fn, "x", x, 2), *_rows(fn, "dt", dt, 1), A.data_ptr(), *_rows(fn, "B", B, 2), *_rows(fn, "C", C, 2))
    return rows, code, dt_code, heads, groups, d_k, d_v


def scan(x, dt, A, B, C, D=None, *, dt_bias=None, softplus=True, state=None, initial=False, seq_starts=None,
         out=None, stream=None):
    """Selective scan of a prompt: S <- exp(dt A) S + dt B x^T, y = S^T C + D x.

    x [batch, length, heads, d_v], or [tokens, heads, d_v] with the sequences
    one behind the other from seq_starts (int32 [n + 1], on the device; None:
    one sequence); dt [.., heads] (float32 or bfloat16; softplus(dt + dt_bias)
    is the time step, or dt + dt_bias with softplus=False); B, C
    [.., groups, d_k] of x's type; A, D, dt_bias [heads] float32.  d_k and d_v
    64 or 128.  state [n, heads, d_k, d_v] float32: each sequence continues
    from its row with initial=True, else from zeros, and leaves its state
    there.  Rows may be views into wider ones, on 16-byte boundaries.  Tokens
    behind the last sequence stay as they are in `out` (undefined where `out`
    is not given).  Returns out, shaped like x."""
    fn = "scan"
    if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4):
        raise ValueError(f"{fn}: x must be [batch, length, heads, d_v] or [tokens, heads, d_v]")
    rows, code, dt_code, heads, groups, d_k, d_v = _selective(fn, x, dt, A, B, C, D, dt_bias)
    n, tokens, starts = _sequences(fn, x.shape[:-2], seq_starts, x)
    if initial and state is None:
        raise ValueError(f"{fn}: initial=True needs the state to continue from")
    if state is not None:
        _dense(fn, "state", state, x, torch.float32, (n, heads, d_k, d_v))
    with _On(x, stream) as st:
        y = _out(fn, out, x, x.shape, x.dtype, (("x", x), ("B", B), ("C", C), ("dt", dt), ("state", state)))
        yp, ys = _rows(fn, "out", y, 2)
        size = lib().qmixer_scan_workspace(n, tokens, heads, groups, d_k, d_v, code)
        if size < 0:
            raise QStateError("qmixer_scan", size)
        work = torch.empty(size, dtype=torch.uint8, device=x.device) if size else None
        _check("qmixer_scan", lib().qmixer_scan(
            *rows, _ptr(D), _ptr(dt_bias), _ptr(state), yp, ys, starts, n, tokens, heads, groups, d_k, d_v, code,
            dt_code, (INITIAL if initial else 0) | (SOFTPLUS if softplus else 0), _ptr(work), size, st))
    return y


def scan_step(x, dt, A, B, C, D=None, *, dt_bias=None, softplus=True, state, out=None, stream=None):
    """The same for one token of each sequence: x [batch, heads, d_v]; state
    [batch, heads, d_k, d_v] float32 moves on by one token."""
    fn = "scan_step"
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{fn}: x must be [batch, heads, d_v]")
    rows, code, dt_code, heads, groups, d_k, d_v = _selective(fn, x, dt, A, B, C, D, dt_bias)
    n = x.shape[0]
    _dense(fn, "state", state, x, torch.float32, (n, heads, d_k, d_v))
    with _On(x, stream) as st:
        y = _out(fn, out, x, x.shape, x.dtype, (("x", x), ("B", B), ("C", C), ("dt", dt), ("state", state)))
        yp, ys = _rows(fn, "out", y, 2)
        _check("qmixer_scan_step", lib().qmixer_scan_step(
            *rows, _ptr(D), _ptr(dt_bias), state.data_ptr(), yp, ys, n, heads, groups, d_k, d_v, code, dt_code,
            SOFTPLUS if softplus else 0, st))
    return y


# ---------------------------------------------------------------- the low-bit state
def load(obj, S, *, stream=None):
    """Quantise binary32 states S [layers * batch * heads, d_k, d_v] (or
    [.., heads, d_k, d_v], as scan leaves them) into a ``qstate.QState`` of any
    kind, width, group, scale mode or rotation: scales from the state itself, as
    the dynamic rule does.  A yoked object's reference becomes S; a bypass or a
    window is emptied.  Objects with row x column scales are refused."""
    fn = "load"
    if getattr(obj, "rowcol", False):
        raise ValueError(f"{fn}: an object with row x column scales fits them in its own steps only")
    _tensor(fn, "S", S, None, torch.float32)
    if S.device.index != obj.device:
        raise ValueError(f"{fn}: S is on {S.device}, the object on cuda:{obj.device}")
    if S.numel() != obj.tiles * obj.d_k * obj.d_v or tuple(S.shape[-2:]) != (obj.d_k, obj.d_v):
        raise ValueError(f"{fn}: S has shape {tuple(S.shape)}, the object {obj.tiles} tiles of {obj.d_k} x {obj.d_v}")
    if not S.is_contiguous():
        raise ValueError(f"{fn}: S must be contiguous")
    if obj.tiles == 0:
        return
    z = obj.sizes
    hb = None if obj.head_bits is None else (ctypes.c_uint8 * obj.heads)(*obj.head_bits)
    with _On(S, stream) as st:
        codes = torch.empty(z["code_bytes"], dtype=torch.uint8, device=S.device)
        scales = torch.empty(max(z["scale_bytes"], 4), dtype=torch.uint8, device=S.device)
        ref = torch.empty_like(S) if z["ref_bytes"] else None
        _check("qmixer_quantize", lib().qmixer_quantize(
            S.data_ptr(), codes.data_ptr(), scales.data_ptr(), _ptr(ref), obj.layers * obj.batch, obj.heads, obj.d_k,
            obj.d_v, 0 if hb is not None else obj.bits, hb, obj.group, obj.scale_dtype, obj.rotation, st))
        obj.import_(codes, scales, ref, stream=torch.cuda.current_stream())


def step(obj, x, dt, A, B, C, D=None, *, dt_bias=None, softplus=True, out=None, stream=None):
    """One token of each sequence on a low-bit state: scan_step with a one-layer
    ``qstate.QState`` of kind MAMBA2 in the place of the binary32 states.
    x [batch, heads, d_v]; returns y, shaped like x."""
    fn = "step"
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{fn}: x must be [batch, heads, d_v]")
    if obj.kind != Q.MAMBA2 or obj.layers != 1:
        raise ValueError(f"{fn}: the object must be of kind MAMBA2 and hold one layer")
    rows, code, dt_code, heads, groups, d_k, d_v = _selective(fn, x, dt, A, B, C, D, dt_bias)
    n = x.shape[0]
    if (n, heads, d_k, d_v) != (obj.batch, obj.heads, obj.d_k, obj.d_v):
        raise ValueError(f"{fn}: the operands are {n} x {heads} tiles of {d_k} x {d_v}, the object "
                         f"{obj.batch} x {obj.heads} of {obj.d_k} x {obj.d_v}")
    if x.device.index != obj.device:
        raise ValueError(f"{fn}: x is on {x.device}, the object on cuda:{obj.device}")
    with _On(x, stream) as st:
        y = _out(fn, out, x, x.shape, x.dtype, (("x", x), ("B", B), ("C", C), ("dt", dt)))
        yp, ys = _rows(fn, "out", y, 2)
        if n == 0:
            return y
        q, k, v, gates, o = obj.alloc_inputs(x.device)
        _check("qmixer_step_operands", lib().qmixer_step_operands(
            *rows, _ptr(dt_bias), q.data_ptr(), k.data_ptr(), v.data_ptr(), gates.data_ptr(), n, heads, groups, d_k,
            d_v, code, dt_code, obj.qkv_dtype, obj.gate_dtype, SOFTPLUS if softplus else 0, st))
        obj.step(q, k, v, gates, o, torch.cuda.current_stream())
        _check("qmixer_step_output", lib().qmixer_step_output(
            o.data_ptr(), rows[0], rows[1], _ptr(D), yp, ys, n, heads, d_v, code, st))
    return y


# ---------------------------------------------------------------- norm
_OUT = {None: OUT_SAME, torch.int8: OUT_INT8, torch.float8_e4m3fn: OUT_E4M3}


def norm(x, weight, *, residual=None, gate=None, eps=1e-5, dtype=None, group=0, out=None, scales=None, stream=None):
    """Root-mean-square norm of the rows of x [.., columns].

    residual: x is added to it in place and the unrounded sum is normalised;
    gate: x * silu(gate) is normalised.  dtype None: returns y of x's type.
    torch.int8 or torch.float8_e4m3fn: returns (codes, scales), y = codes *
    scales, with float32 scales [.., columns / group] of `group` consecutive
    columns (a power of two from 8 to 256), or [.., 1] of whole rows for 0; a
    row or group without a finite maximum gets the scale NaN."""
    fn = "norm"
    _tensor(fn, "x", x)
    code = _code(fn, x)
    if x.dim() < 1:
        raise ValueError(f"{fn}: x must have rows")
    columns = x.shape[-1]
    _dense(fn, "weight", weight, x, x.dtype, (columns,))
    if residual is not None and gate is not None:
        raise ValueError(f"{fn}: residual or gate, not both")
    if dtype not in _OUT:
        raise ValueError(f"{fn}: dtype {dtype} is not None, torch.int8 or torch.float8_e4m3fn")
    if dtype is None and (group or scales is not None):
        raise ValueError(f"{fn}: group and scales go with 8-bit output")
    if group and (group < 0 or columns % group):
        raise ValueError(f"{fn}: groups of {group} do not divide {columns} columns")
    other = residual if residual is not None else gate
    shape = tuple(x.shape)
    x2 = _flat(fn, "x", x)
    if other is not None:
        _tensor(fn, "residual" if other is residual else "gate", other, x, x.dtype, shape)
        o2 = _flat(fn, "residual" if other is residual else "gate", other)
        if other is residual:
            _overlap(fn, "residual", o2, "x", x2)
    before = BEFORE_NONE if other is None else BEFORE_RESIDUAL if other is residual else BEFORE_GATE
    rows = x2.shape[0]
    with _On(x, stream) as st:
        y = _out(fn, out, x, shape, dtype or x.dtype, (("x", x), ("residual or gate", other), ("weight", weight)))
        y2 = _flat(fn, "out", y)
        if dtype is not None:
            want = shape[:-1] + (columns // group if group else 1,)
            if scales is None:
                scales = torch.empty(want, dtype=torch.float32, device=x.device)
            else:
                _dense(fn, "scales", scales, x, torch.float32, want)
        _check("qmixer_norm", lib().qmixer_norm(
            *_rows(fn, "x", x2, 1), *(_rows(fn, "residual or gate", o2, 1) if other is not None else (None, 0)),
            weight.data_ptr(), *_rows(fn, "out", y2, 1), _ptr(scales), rows, columns, group, eps, code, before,
            _OUT[dtype], st))
    return y if dtype is None else (y, scales)


def _flat(fn, name, t):
    """[rows, columns] without a copy."""
    if t.dim() == 2:
        return t
    try:
        return t.view(-1, t.shape[-1]) if t.shape[-1] else t.reshape(-1, 0)
    except RuntimeError:
        raise ValueError(f"{fn}: the rows of {name} must lie in one stride") from None
