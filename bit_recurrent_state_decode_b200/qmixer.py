"""Thin ctypes binding of the C ABI in include/qmixer.h (libqmixer.so): the
operators around the recurrent state of a Mamba2 layer.

    conv, conv_step      the short causal convolution of a prompt / of one token
    scan, scan_step      the selective scan of a prompt / of one token, binary32 states
    load                 a prompt's binary32 states into a low-bit ``qstate.QState``
    step                 the selective step of one token on a ``qstate.QState``
    norm                 root-mean-square norm, with a residual or a gate, and 8-bit output

    scan_timeouts        blocks of prompt scans that gave up a bounded wait

Argument checks and marshalling only: the arithmetic runs in the CUDA kernels
of the library.  A usual call (its own output, the current stream) is checked and
launched by the compiled module _qmixer_usual; what that leaves takes the way below.
Calls are asynchronous on the current stream of the tensors' device, or on
`stream`, to which an output made by the call then belongs; tensors of another
stream have to be ordered before the call by the caller and kept until it has run
(Tensor.record_stream), as for any PyTorch operator.  What is written may not share
memory with what is read.  The library must have been built; there is no CPU fallback
and no autograd: inputs that require a gradient are refused while gradients are
recorded, inputs with a forward-mode tangent always, and what a call writes in place
counts as a new version of the tensor.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch
from torch.autograd import forward_ad

from . import qstate as Q
from .qstate import QStateError

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqmixer.so")

INITIAL, SILU, SOFTPLUS = 1, 2, 4
BEFORE_NONE, BEFORE_RESIDUAL, BEFORE_GATE = 0, 1, 2
OUT_SAME, OUT_INT8, OUT_E4M3 = 0, 1, 2

# every function include/qmixer.h declares, with the fields of its argument
# structure in the notation of the struct module (native alignment)
_FIELDS = {"qmixer_conv": "PqPPPPqPiqiiii", "qmixer_conv_step": "PqPPPPqiiiii",
           "qmixer_scan": "PqPqPPqPqPPPPqPiqiiiiiiiPq", "qmixer_scan_step": "PqPqPPqPqPPPPqiiiiiiii",
           "qmixer_step_operands": "PqPqPPqPqPPPPPiiiiiiiiii", "qmixer_step_output": "PPqPPqiiii",
           "qmixer_norm": "PqPqPPqPqiifiii", "qmixer_quantize": "PPPPqiiiiPiii"}
EXPORTS = tuple(_FIELDS) + ("qmixer_scan_workspace", "qmixer_scan_timeouts", "qmixer_debug_set")

_lib = None


class _Load:
    """Stands for _qmixer_usual until the first call of one of its functions."""

    def __getattr__(self, name):
        global _usual
        from . import build
        lib()
        if not os.path.exists(build.USUAL):
            raise RuntimeError(f"{build.USUAL} is missing: build it with "
                               "`python -m bit_recurrent_state_decode_b200.build`")
        if not build.usual_built_for(build.usual_versions()):
            # of another binary interface: loading it could do anything
            raise RuntimeError(f"{build.USUAL} was built for other versions of Python or PyTorch: build it again with "
                               "`python -m bit_recurrent_state_decode_b200.build`")
        from . import _qmixer_usual
        _usual = _qmixer_usual
        return getattr(_usual, name)


_usual = _Load()


def lib():
    """Load libqmixer.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_recurrent_state_decode_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name in _FIELDS:
            f = getattr(L, name)
            f.argtypes, f.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
        L.qmixer_scan_workspace.argtypes = [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 5
        L.qmixer_scan_workspace.restype = ctypes.c_int64
        L.qmixer_scan_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint64), ctypes.c_void_p]
        L.qmixer_debug_set.argtypes = [ctypes.c_int32, ctypes.c_uint32]
        _lib = L
    return _lib


def _entry(name):
    """The C call `name` of an argument structure's fields (addresses as integers, 0
    for NULL) and a stream.  The structure is packed into bytes in one go: a
    ctypes conversion of each field would cost as much as a small kernel."""
    pack = struct.Struct(_FIELDS[name]).pack

    def call(stream, *fields):
        rc = getattr(_lib or lib(), name)(pack(*fields), stream)
        if rc:
            raise QStateError(name, rc)
    return call


_conv, _conv_step, _scan, _scan_step, _step_operands, _step_output, _norm, _quantize = map(_entry, _FIELDS)


# ---------------------------------------------------------------- argument checks
_CODE = {torch.float32: Q.F32, torch.bfloat16: Q.BF16}
_F32 = torch.float32
# the current device and the address of its current stream (a tensor was seen, so
# CUDA is initialised; torch.cuda's own calls check that and build an object first)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _tensor(fn, name, t, index, dtype=None, shape=None):
    """Refuse what is not a CUDA tensor of this device (None: any), type and shape
    (None: any), whose memory does not hold its values (negated views, sparse
    layouts), or that carries or wants a gradient, in either direction."""
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{fn}: {name} is on {t.device}, not on cuda:{index}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{fn}: {name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.layout is not torch.strided or t.is_neg() or t.is_conj():
        raise ValueError(f"{fn}: {name} is a view whose memory does not hold its values (resolve_neg() gives one)")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{fn}: {name} requires a gradient, and {fn} has no backward pass")
    if getattr(forward_ad, "_current_level", 0) >= 0 and forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{fn}: {name} carries a tangent, and {fn} has no forward-mode derivative")


def _dense(fn, name, t, index, dtype, shape):
    """The same for a contiguous tensor; returns its address."""
    _tensor(fn, name, t, index, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous")
    return t.data_ptr()


def _rows(fn, name, t, inner):
    """Stride between the rows of a tensor whose last `inner` dimensions are a row:
    contiguous, the leading ones (one or two) walking in one stride."""
    shape, strides = t.shape, t.stride()
    step = 1
    for d in range(len(shape) - 1, len(shape) - 1 - inner, -1):
        if strides[d] != step and shape[d] != 1:
            raise ValueError(f"{fn}: the elements of a row of {name} must be contiguous")
        step *= shape[d]
    at = len(shape) - inner - 1
    n = shape[at]
    stride = strides[at] if n > 1 else step
    if at == 1 and shape[0] > 1:
        if n == 1:
            stride = strides[0]
        elif n > 1 and strides[0] != n * stride:
            raise ValueError(f"{fn}: the sequences of {name} must lie one behind the other")
    if n and stride < step:
        raise ValueError(f"{fn}: the rows of {name} overlap")
    return stride


def _span(t):
    if t.is_contiguous():
        return t.nbytes
    return (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))) * t.element_size() if t.numel() else 0


def _pitch(t):
    """(bytes from one row to the next, bytes of a row) of a tensor of rows with gaps;
    None for one without."""
    row = 1
    for n, stride in zip(reversed(t.shape), reversed(t.stride())):
        if n == 1:
            continue
        if stride != row:
            return stride * t.element_size(), row * t.element_size()
        row *= n
    return None


def _apart(fn, name, a, other, b):
    """Refuse an output that shares memory with an input; columns of one buffer's
    rows may interleave."""
    if b is None:
        return
    pa, pb = a.data_ptr(), b.data_ptr()
    if pa >= pb + _span(b) or pb >= pa + _span(a):
        return
    ra, rb = _pitch(a), _pitch(b)
    if ra and rb and ra[0] == rb[0]:
        off = (pb - pa) % ra[0]
        if off >= ra[1] and off + rb[1] <= ra[0]:
            return
    raise ValueError(f"{fn}: {name} overlaps {other}")


def _code(fn, t):
    c = _CODE.get(t.dtype)
    if c is None:
        raise ValueError(f"{fn}: dtype {t.dtype} is not float32 or bfloat16")
    return c


def _launch(fn, t, stream, body):
    """body(address of the stream) with the tensors' device current, and, on a
    stream of the caller's, its allocations belonging to that stream."""
    index = t.get_device()
    if stream is None and index == _current_device():
        return body(_raw_stream(index))
    if stream is not None and stream.device.index != index:
        raise ValueError(f"{fn}: the stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.device(index):
        if stream is None:
            return body(_raw_stream(index))
        with torch.cuda.stream(stream):
            return body(stream.cuda_stream)


def _sequences(fn, lead, seq_starts, index):
    """(sequences, tokens, address of seq_starts) of a prompt's leading dimensions."""
    if len(lead) == 2:
        if seq_starts is not None:
            raise ValueError(f"{fn}: seq_starts goes with tokens in one axis, not with a batch of equal sequences")
        return lead[0], lead[0] * lead[1], 0
    if seq_starts is None:
        return 1, lead[0], 0
    _tensor(fn, "seq_starts", seq_starts, index, torch.int32)
    if seq_starts.dim() != 1 or seq_starts.numel() < 1 or not seq_starts.is_contiguous():
        raise ValueError(f"{fn}: seq_starts must be a contiguous vector of the sequences' first tokens and their end")
    return seq_starts.numel() - 1, lead[0], seq_starts.data_ptr()


def _fresh(like, dtype):
    """A contiguous output of `like`'s shape."""
    if dtype is like.dtype:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)


def _given(fn, out, like, shape, dtype, inputs):
    """The caller's `out`, apart from the inputs {name: tensor or None}."""
    _tensor(fn, "out", out, like.get_device(), dtype, shape)
    _alone(fn, "out", out, inputs)
    return out


def _written(*tensors):
    """What a call has written in place, autograd learns by its version: an operation that
    saved the former values for its backward pass must not go on with these."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _alone(fn, name, a, inputs):
    """_apart of each of the inputs {name: tensor or None}, by bounds first."""
    if a is None:
        return
    at = a.data_ptr()
    end = at + _span(a)
    for other, b in inputs.items():
        if b is not None:
            first = b.data_ptr()
            if first < end and at < first + _span(b):
                _apart(fn, name, a, other, b)


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
    if out is None and stream is None:
        y = _usual.conv(x, weight, bias, state, bool(activation), bool(initial), seq_starts)
        if y is not None:
            return y
    fn = "conv"
    _tensor(fn, "x", x, None)
    if x.dim() not in (2, 3):
        raise ValueError(f"{fn}: x must be [batch, length, channels] or [tokens, channels]")
    shape, index, code = x.shape, x.get_device(), _code(fn, x)
    n, tokens, starts = _sequences(fn, shape[:-1], seq_starts, index)
    inputs = {"x": x, "weight": weight, "bias": bias, "seq_starts": seq_starts}
    width, wp, bp, sp = _taps(fn, x, weight, bias, state, n, index, inputs)
    if initial and state is None:
        raise ValueError(f"{fn}: initial=True needs the state to continue from")
    xs = _rows(fn, "x", x, 1)

    def body(st):
        if out is None:
            y, ys = _fresh(x, x.dtype), shape[-1]
        else:
            y = _given(fn, out, x, shape, x.dtype, {**inputs, "state": state})
            ys = _rows(fn, "out", y, 1)
        _conv(st, x.data_ptr(), xs, wp, bp, sp, y.data_ptr(), ys, starts, n, tokens, shape[-1],
              width, code, (INITIAL if initial else 0) | (SILU if activation else 0))
        _written(state, out)
        return y
    return _launch(fn, x, stream, body)


def conv_step(x, weight, bias=None, *, state, activation=True, out=None, stream=None):
    """The same for one token of each sequence: x [batch, channels]; state
    [batch, width - 1, channels] moves on by one token."""
    if out is None and stream is None:
        y = _usual.conv_step(x, weight, bias, state, bool(activation))
        if y is not None:
            return y
    fn = "conv_step"
    _tensor(fn, "x", x, None)
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be [batch, channels]")
    if state is None:
        raise ValueError(f"{fn}: state is required")
    shape, code = x.shape, _code(fn, x)
    inputs = {"x": x, "weight": weight, "bias": bias}
    width, wp, bp, sp = _taps(fn, x, weight, bias, state, shape[0], x.get_device(), inputs)
    xs = _rows(fn, "x", x, 1)

    def body(st):
        if out is None:
            y, ys = _fresh(x, x.dtype), shape[1]
        else:
            y = _given(fn, out, x, shape, x.dtype, {**inputs, "state": state})
            ys = _rows(fn, "out", y, 1)
        _conv_step(st, x.data_ptr(), xs, wp, bp, sp, y.data_ptr(), ys, shape[0], shape[1], width,
                   code, SILU if activation else 0)
        _written(state, out)
        return y
    return _launch(fn, x, stream, body)


def _taps(fn, x, weight, bias, state, n, index, inputs):
    channels, dtype = x.shape[-1], x.dtype
    _tensor(fn, "weight", weight, index, dtype)
    if weight.dim() != 2 or weight.shape[0] != channels or not weight.is_contiguous():
        raise ValueError(f"{fn}: weight must be contiguous [channels, width]")
    width = weight.shape[1]
    bp = 0 if bias is None else _dense(fn, "bias", bias, index, dtype, (channels,))
    sp = 0
    if state is not None:
        sp = _dense(fn, "state", state, index, dtype, (n, width - 1, channels))
        _alone(fn, "state", state, inputs)
    return width, weight.data_ptr(), bp, sp


# ---------------------------------------------------------------- selective scan
def _selective(fn, x, dt, A, B, C, D, dt_bias):
    """The fields x, dt, A, B, C and D, dt_bias of a call, then (dtype, dt's dtype,
    heads, groups, d_k, d_v) and the device."""
    _tensor(fn, "x", x, None)
    code, index, xsh, dtype = _code(fn, x), x.get_device(), x.shape, x.dtype
    lead, heads, d_v = xsh[:-2], xsh[-2], xsh[-1]
    per_head = (heads,)
    _tensor(fn, "B", B, index, dtype)
    bsh = B.shape
    if len(bsh) != len(xsh) or bsh[:-2] != lead:
        raise ValueError(f"{fn}: B has shape {tuple(bsh)}, expected {tuple(lead)} + (groups, d_k)")
    groups, d_k = bsh[-2], bsh[-1]
    if groups == 0 or heads % groups:
        raise ValueError(f"{fn}: {heads} heads do not divide into {groups} groups")
    _tensor(fn, "dt", dt, index, None, lead + per_head)
    _tensor(fn, "C", C, index, dtype, bsh)
    ap = _dense(fn, "A", A, index, _F32, per_head)
    dp, biasp = (0 if t is None else _dense(fn, name, t, index, _F32, per_head)
                 for name, t in (("D", D), ("dt_bias", dt_bias)))
    rows = (x.data_ptr(), _rows2(fn, "x", x, d_v, heads * d_v), dt.data_ptr(), _rows(fn, "dt", dt, 1), ap,
            B.data_ptr(), _rows2(fn, "B", B, d_k, groups * d_k), C.data_ptr(), _rows2(fn, "C", C, d_k, groups * d_k))
    if (rows[0] | rows[5] | rows[7] | (rows[1] | rows[6] | rows[8]) * x.element_size()) & 15:
        raise ValueError(f"{fn}: the rows of x, B and C must start on 16-byte boundaries")
    return rows, dp, biasp, (heads, groups, d_k, d_v, code, _code(fn, dt)), index


def _rows2(fn, name, t, inner, row):
    """_rows of tokens of [heads, d]: the common case first, one axis of tokens whose
    rows are whole."""
    s = t.stride()
    if len(s) == 3 and s[2] == 1 and s[1] == inner:
        if t.shape[0] <= 1:
            return row
        if s[0] >= row:
            return s[0]
    return _rows(fn, name, t, 2)


@functools.lru_cache(maxsize=256)
def _workspace(index, *sizes):
    """qmixer_scan_workspace of a device, which has to be the current one."""
    size = lib().qmixer_scan_workspace(*sizes)
    if size < 0:
        raise QStateError("qmixer_scan", size)
    return size


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
    if out is None and stream is None:
        y = _usual.scan(x, dt, A, B, C, D, dt_bias, state, bool(softplus), bool(initial), seq_starts)
        if y is not None:
            return y
    fn = "scan"
    if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4):
        raise ValueError(f"{fn}: x must be [batch, length, heads, d_v] or [tokens, heads, d_v]")
    rows, dp, biasp, sizes, index = _selective(fn, x, dt, A, B, C, D, dt_bias)
    n, tokens, starts = _sequences(fn, x.shape[:-2], seq_starts, index)
    if initial and state is None:
        raise ValueError(f"{fn}: initial=True needs the state to continue from")
    heads, groups, d_k, d_v = sizes[:4]
    inputs = {"x": x, "dt": dt, "A": A, "B": B, "C": C, "D": D, "dt_bias": dt_bias, "seq_starts": seq_starts}
    sp = 0
    if state is not None:
        sp = _dense(fn, "state", state, index, _F32, (n, heads, d_k, d_v))
        _alone(fn, "state", state, inputs)

    def body(st):
        if out is None:
            y, ys = _fresh(x, x.dtype), sizes[0] * sizes[3]
        else:
            y = _given(fn, out, x, x.shape, x.dtype, {**inputs, "state": state})
            ys = _rows(fn, "out", y, 2)
        size = _workspace(index, n, tokens, *sizes[:5])
        work = x.new_empty(size, dtype=torch.uint8) if size else None
        _scan(st, *rows, dp, biasp, sp, y.data_ptr(), ys, starts, n, tokens, *sizes,
              (INITIAL if initial else 0) | (SOFTPLUS if softplus else 0), work.data_ptr() if size else 0, size)
        _written(state, out)
        return y
    return _launch(fn, x, stream, body)


def scan_timeouts(device=None):
    """Thread blocks of prompt scans on `device` (None: the current one) that gave up a
    bounded wait so far (qmixer_scan_timeouts); their outputs and states are NaN.
    Waits for the device's current stream."""
    count = ctypes.c_uint64()
    with torch.cuda.device(device):
        rc = lib().qmixer_scan_timeouts(ctypes.byref(count), torch.cuda.current_stream().cuda_stream)
    if rc:
        raise QStateError("qmixer_scan_timeouts", rc)
    return count.value


def debug_set(drop_from_chunk=-1, wait_polls=1 << 24):
    """Fault injection for the bounded waits of the prompt scans that follow
    (qmixer_debug_set)."""
    rc = lib().qmixer_debug_set(int(drop_from_chunk), int(wait_polls))
    if rc:
        raise QStateError("qmixer_debug_set", rc)


def scan_step(x, dt, A, B, C, D=None, *, dt_bias=None, softplus=True, state, out=None, stream=None):
    """The same for one token of each sequence: x [batch, heads, d_v]; state
    [batch, heads, d_k, d_v] float32 moves on by one token."""
    if out is None and stream is None:
        y = _usual.scan_step(x, dt, A, B, C, D, dt_bias, state, bool(softplus))
        if y is not None:
            return y
    fn = "scan_step"
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{fn}: x must be [batch, heads, d_v]")
    rows, dp, biasp, sizes, index = _selective(fn, x, dt, A, B, C, D, dt_bias)
    shape = x.shape
    n = shape[0]
    sp = _dense(fn, "state", state, index, _F32, (n, sizes[0], sizes[2], sizes[3]))
    inputs = {"x": x, "dt": dt, "A": A, "B": B, "C": C, "D": D, "dt_bias": dt_bias}
    _alone(fn, "state", state, inputs)

    def body(st):
        if out is None:
            y, ys = _fresh(x, x.dtype), sizes[0] * sizes[3]
        else:
            y = _given(fn, out, x, shape, x.dtype, {**inputs, "state": state})
            ys = _rows(fn, "out", y, 2)
        _scan_step(st, *rows, dp, biasp, sp, y.data_ptr(), ys, n, *sizes,
                   SOFTPLUS if softplus else 0)
        _written(state, out)
        return y
    return _launch(fn, x, stream, body)


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
    _tensor(fn, "S", S, None, _F32)
    if S.get_device() != obj.device:
        raise ValueError(f"{fn}: S is on {S.device}, the object on cuda:{obj.device}")
    if S.numel() != obj.tiles * obj.d_k * obj.d_v or S.shape[-2:] != (obj.d_k, obj.d_v):
        raise ValueError(f"{fn}: S has shape {tuple(S.shape)}, the object {obj.tiles} tiles of {obj.d_k} x {obj.d_v}")
    if not S.is_contiguous():
        raise ValueError(f"{fn}: S must be contiguous")
    if obj.tiles == 0:
        return
    z = obj.sizes

    def body(st):
        # an object's own buffers are reached by qstate_import alone
        at = (z["code_bytes"] + 255) // 256 * 256
        codes = torch.empty(at + z["scale_bytes"], dtype=torch.uint8, device=S.device)
        cp, scales = codes.data_ptr(), codes.data_ptr() + at
        ref = torch.empty_like(S) if z["ref_bytes"] else None
        mixed = obj.head_bits is not None
        hb = (ctypes.c_uint8 * obj.heads)(*obj.head_bits) if mixed else None
        _quantize(st, S.data_ptr(), cp, scales, 0 if ref is None else ref.data_ptr(),
                  obj.layers * obj.batch, obj.heads, obj.d_k, obj.d_v, 0 if mixed else obj.bits,
                  ctypes.addressof(hb) if mixed else 0, obj.group, obj.scale_dtype, obj.rotation)
        rc = Q.lib().qstate_import(obj._h, cp, scales, None if ref is None else ref.data_ptr(), st)
        if rc:
            raise QStateError("qstate_import", rc)
    _launch(fn, S, stream, body)


def step(obj, x, dt, A, B, C, D=None, *, dt_bias=None, softplus=True, out=None, stream=None):
    """One token of each sequence on a low-bit state: scan_step with a one-layer
    ``qstate.QState`` of kind MAMBA2 in the place of the binary32 states.
    x [batch, heads, d_v]; returns y, shaped like x."""
    fn = "step"
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{fn}: x must be [batch, heads, d_v]")
    if obj.kind != Q.MAMBA2 or obj.layers != 1:
        raise ValueError(f"{fn}: the object must be of kind MAMBA2 and hold one layer")
    rows, dp, biasp, sizes, index = _selective(fn, x, dt, A, B, C, D, dt_bias)
    n = x.shape[0]
    if (n, sizes[0], sizes[2], sizes[3]) != (obj.batch, obj.heads, obj.d_k, obj.d_v):
        raise ValueError(f"{fn}: the operands are {n} x {sizes[0]} tiles of {sizes[2]} x {sizes[3]}, the object "
                         f"{obj.batch} x {obj.heads} of {obj.d_k} x {obj.d_v}")
    if index != obj.device:
        raise ValueError(f"{fn}: x is on {x.device}, the object on cuda:{obj.device}")

    def body(st):
        if out is None:
            y, ys = _fresh(x, x.dtype), sizes[0] * sizes[3]
        else:
            y = _given(fn, out, x, x.shape, x.dtype,
                       {"x": x, "dt": dt, "A": A, "B": B, "C": C, "D": D, "dt_bias": dt_bias})
            ys = _rows(fn, "out", y, 2)
        if n == 0:
            return y
        q, k, v, gates, o = obj.alloc_inputs(x.device)
        _step_operands(st, *rows, biasp, q.data_ptr(), k.data_ptr(), v.data_ptr(), gates.data_ptr(), n, *sizes,
                       obj.qkv_dtype, obj.gate_dtype, SOFTPLUS if softplus else 0)
        obj.step(q, k, v, gates, o, torch.cuda.current_stream())
        _step_output(st, o.data_ptr(), rows[0], rows[1], dp, y.data_ptr(), ys, n, sizes[0],
                     sizes[3], sizes[4])
        _written(out)
        return y
    return _launch(fn, x, stream, body)


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
    kind = _OUT.get(dtype)
    if out is None and stream is None and scales is None and kind is not None and (residual is None or gate is None):
        y = _usual.norm(x, weight, residual if gate is None else gate,
                        BEFORE_RESIDUAL if residual is not None else BEFORE_GATE if gate is not None else BEFORE_NONE,
                        eps, kind, group)
        if y is not None:
            return y
    fn = "norm"
    _tensor(fn, "x", x, None)
    code, index, shape, xd = _code(fn, x), x.get_device(), x.shape, x.dtype
    if len(shape) < 1:
        raise ValueError(f"{fn}: x must have rows")
    columns = shape[-1]
    wp = _dense(fn, "weight", weight, index, xd, (columns,))
    if residual is not None and gate is not None:
        raise ValueError(f"{fn}: residual or gate, not both")
    if kind is None:
        raise ValueError(f"{fn}: dtype {dtype} is not None, torch.int8 or torch.float8_e4m3fn")
    if kind == OUT_SAME and (group or scales is not None):
        raise ValueError(f"{fn}: group and scales go with 8-bit output")
    if group and (group < 0 or columns % group):
        raise ValueError(f"{fn}: groups of {group} do not divide {columns} columns")
    x2 = _flat(fn, "x", x)
    xs = _rows(fn, "x", x2, 1)
    before, name, other = ((BEFORE_RESIDUAL, "residual", residual) if residual is not None else
                           (BEFORE_GATE, "gate", gate) if gate is not None else (BEFORE_NONE, None, None))
    op, ostride = 0, 0
    if before:
        _tensor(fn, name, other, index, xd, shape)
        o2 = _flat(fn, name, other)
        op, ostride = o2.data_ptr(), _rows(fn, name, o2, 1)
        if before == BEFORE_RESIDUAL:
            _alone(fn, name, o2, {"x": x2, "weight": weight})

    def body(st):
        if out is None:
            y = y2 = _fresh(x, dtype or xd)
            ys = columns
        else:
            y = _given(fn, out, x, shape, dtype or xd, {"x": x, name: other, "weight": weight})
            y2 = _flat(fn, "out", y)
            ys = _rows(fn, "out", y2, 1)
        scale, sp = scales, 0
        if kind:
            want = shape[:-1] + (columns // group if group else 1,)
            if scale is None:
                scale = x.new_empty(want, dtype=_F32)
            else:
                _dense(fn, "scales", scale, index, _F32, want)
                _alone(fn, "scales", scale, {"x": x2, name: other, "weight": weight, "out": y2})
            sp = scale.data_ptr()
        _norm(st, x2.data_ptr(), xs, op, ostride, wp, y2.data_ptr(), ys, sp, x2.shape[0],
              columns, group, eps, code, before, kind)
        _written(residual, out, scales)
        return (y, scale) if kind else y
    return _launch(fn, x, stream, body)


def _flat(fn, name, t):
    """[rows, columns] without a copy."""
    if t.dim() == 2:
        return t
    try:
        return t.view(-1, t.shape[-1]) if t.shape[-1] else t.reshape(0, 0)
    except RuntimeError:
        raise ValueError(f"{fn}: the rows of {name} must lie in one stride") from None
