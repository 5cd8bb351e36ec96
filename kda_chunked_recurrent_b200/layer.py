"""The layer operators around the KDA recurrence on device tensors (include/kda_layer.h):
short causal convolution, selective state space scan and root-mean-square norm.

Like ``prefill`` and ``decode`` these functions only check and marshal arguments and allocate
outputs; all arithmetic is in the library's kernels.  A call is one launch on ``stream`` (the
tensors' device's current stream by default), reads nothing back and can be captured in a
CUDA graph.  Wrong types, shapes, strides or devices raise ValueError, what the library
refuses raises KDAError.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import KDAError, capi

_DTYPE = {torch.bfloat16: capi.KDA_DTYPE_BF16, torch.float16: capi.KDA_DTYPE_F16,
          torch.float32: capi.KDA_DTYPE_F32}
_byref, _lib = ctypes.byref, capi.lib
# handle of a device's current stream, without making a Stream object where torch allows it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _fail(what):
    raise ValueError(what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _device(x):
    """Index of the GPU that x is on."""
    d = x.get_device()
    if d < 0:
        _fail(f"CUDA tensors expected, got one on {x.device}")
    return d


def _dtype(x, name):
    code = _DTYPE.get(x.dtype)
    if code is None:
        _fail(f"{name}: bfloat16, float16 or float32 expected, got {x.dtype}")
    return code


# The checks of a call are on the path of every token: each looks at what it needs once and
# returns what the launch takes (an address, a stride); the messages are made on failure only.
def _like(name, t, dtype, shape, dev):
    """Address of a contiguous tensor of this type, shape and device; None for None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _fail(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on GPU {dev} expected, "
          f"got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _vector(name, t, dtypes, n, dev):
    """Address of n contiguous values of one of these types; None for None."""
    if t is None:
        return None
    if t.dtype in dtypes and t.numel() == n and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _fail(f"{name}: {n} contiguous values of {dtypes} on GPU {dev} expected, got {t.numel()} of "
          f"{t.dtype} on {t.device}")


_INT32, _BYTES = (torch.int32,), (torch.bool, torch.uint8)


def _rows(name, t, dtype, shape, dev, tail=1):
    """Elements between rows of a tensor [..., row] whose last ``tail`` dimensions are a
    contiguous row and whose leading dimensions step through rows at one stride."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _fail(f"{name}: a {dtype} tensor of shape {tuple(shape)} on GPU {dev} expected, got "
              f"{t.dtype} {tuple(t.shape)} on {t.device}")
    st = t.stride()
    if tail == 1 and st[-1] == 1 and st[-2] >= shape[-1]:    # the usual layouts
        if len(st) == 2 or st[0] == st[1] * shape[1]:
            return st[-2]
    n = 1
    for i in range(1, tail + 1):
        if shape[-i] != 1 and st[-i] != n:
            _fail(f"{name}: the elements of a row must be adjacent, strides {st}")
        n *= shape[-i]
    row, step = None, 1
    for i in range(len(st) - tail - 1, -1, -1):
        if shape[i] == 1:
            continue
        if row is None:
            row = st[i]
        if st[i] != row * step:
            _fail(f"{name}: rows must lie at one distance, strides {st}")
        step *= shape[i]
    if row is None or 0 in shape:
        return n
    if row < n:
        _fail(f"{name}: rows must not overlap, strides {st}")
    return row


def _seqs(rows, cu_seqlens, num_seqs, state, state_indices, has_state, device_status, dev):
    """Number of sequences, the flag of the offsets' type, and the addresses of offsets,
    slots, state marks and status word."""
    flags, cu = 0, None
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        if cu_seqlens.dtype is torch.int64:
            flags = capi.KDA_LAYER_CU_SEQLENS_I64
        if N < 1:
            _fail("cu_seqlens: at least two offsets expected")
        cu = _vector("cu_seqlens", cu_seqlens, (torch.int32, torch.int64), N + 1, dev)
        if num_seqs is not None and num_seqs != N:
            _fail("num_seqs does not agree with cu_seqlens")
    else:
        N = 1 if num_seqs is None else int(num_seqs)
        if N < 1 or rows % N:
            _fail("without cu_seqlens the rows are num_seqs sequences of one length")
    if state is None and (state_indices is not None or has_state is not None):
        _fail("state_indices and has_state need a state")
    return (N, flags, cu, _vector("state_indices", state_indices, _INT32, N, dev),
            _vector("has_state", has_state, _BYTES, N, dev),
            _vector("device_status", device_status, _INT32, 1, dev))


def _call(fn, where, dev, stream, *args):
    """Launch on the tensors' device: its current stream unless one is given."""
    s = _current_stream(dev) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == dev:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc != capi.KDA_OK:
        raise KDAError(rc, where)


def _conv_weight(weight, bias, C, dev):
    if weight.dim() != 2:
        _fail("weight: [channels, width] expected")
    W = weight.shape[1]
    return (W, _like("weight", weight, torch.float32, (C, W), dev),
            _like("bias", bias, torch.float32, (C,), dev))


def _parts_shape(lead, C, parts):
    if parts < 1 or C % parts:
        _fail("parts must divide the channels")
    return lead + (C,) if parts == 1 else (parts,) + lead + (C // parts,)


def conv_prefill(x, weight, *, bias=None, state=None, state_indices=None, has_state=None,
                 cu_seqlens=None, num_seqs: Optional[int] = None, parts: int = 1,
                 silu: bool = True, out=None, device_status=None, stream=None):
    """Short causal convolution over packed prompts (kda_conv_prefill).

    x: [T, C] bf16 / fp16 / fp32, rows at any distance; weight: [C, W] fp32, W = 2, 3 or 4;
    bias: [C] fp32.  ``state``: [P, W - 1, C] pool of x's type, updated in place: sequence n
    continues from slot ``state_indices[n]`` (n without indices) where ``has_state[n]`` (all,
    when None) and leaves its last W - 1 rows there.  ``cu_seqlens``: int32 or int64 [N + 1];
    without it ``num_seqs`` (default 1) sequences of equal length.
    Returns out [T, C], or with ``parts`` [parts, T, C / parts], each part contiguous (3 gives
    q, k and v for ``prefill``).
    """
    if x.dim() != 2:
        _fail("x: [T, C] expected")
    (T, C), t, dev = x.shape, x.dtype, _device(x)
    code = _dtype(x, "x")
    W, pw, pb = _conv_weight(weight, bias, C, dev)
    N, flags, pcu, pslot, phas, pstatus = _seqs(T, cu_seqlens, num_seqs, state, state_indices,
                                                has_state, device_status, dev)
    P = 0 if state is None else state.shape[0]
    pstate = _like("state", state, t, (P, W - 1, C), dev)
    oshape = _parts_shape((T,), C, parts)
    if out is None:
        out = x.new_empty(oshape)
    pout = _like("out", out, t, oshape, dev)
    shape = capi.kda_conv_shape_t(N, T, C, W, parts, P, code, 0, _rows("x", x, t, (T, C), dev))
    _call(_lib.kda_conv_prefill, "kda_conv_prefill", dev, stream, x.data_ptr(), pw, pb, pstate,
          pslot, phas, pcu, _byref(shape), pout, pstatus,
          flags | (capi.KDA_CONV_SILU if silu else 0))
    return out


def conv_decode(x, weight, state, *, bias=None, state_indices=None, parts: int = 1,
                silu: bool = True, out=None, step_states=None, return_step_states: bool = False,
                keep_state: bool = False, device_status=None, stream=None):
    """Short causal convolution of new tokens over a state pool (kda_conv_decode).

    x: [N, T, C], T new tokens of every sequence; weight, bias, state as in conv_prefill;
    state_indices: [N] int32 (negative = padding row: zero output) or None (slot n).
    Returns (out, step_states): out [N, T, C] or [parts, N, T, C / parts]; step_states
    [N, T, W - 1, C], the state after every token, when requested.  ``keep_state`` leaves the
    pool as it was.
    """
    if x.dim() != 3:
        _fail("x: [N, T, C] expected")
    (N, T, C), t, dev = x.shape, x.dtype, _device(x)
    code = _dtype(x, "x")
    W, pw, pb = _conv_weight(weight, bias, C, dev)
    P = state.shape[0]
    pstate = _like("state", state, t, (P, W - 1, C), dev)
    pslot = _vector("state_indices", state_indices, _INT32, N, dev)
    pstatus = _vector("device_status", device_status, _INT32, 1, dev)
    oshape = _parts_shape((N, T), C, parts)
    if out is None:
        out = x.new_empty(oshape)
    pout = _like("out", out, t, oshape, dev)
    if step_states is None and return_step_states:
        step_states = x.new_empty((N, T, W - 1, C))
    psteps = _like("step_states", step_states, t, (N, T, W - 1, C), dev)
    shape = capi.kda_conv_shape_t(N, T, C, W, parts, P, code, 0, _rows("x", x, t, (N, T, C), dev))
    _call(_lib.kda_conv_decode, "kda_conv_decode", dev, stream, x.data_ptr(), pw, pb, pstate,
          pslot, _byref(shape), pout, psteps, pstatus,
          (capi.KDA_CONV_SILU if silu else 0) | (capi.KDA_LAYER_KEEP_STATE if keep_state else 0))
    return out, step_states


def _scan_args(x, dt, A_log, B, C, D, z, dt_bias, state, rows, dev):
    """Check the operands that both forms share: their addresses in the entry points' order
    and the shape struct without its sequences.  rows: the shape of x."""
    t, ch = x.dtype, rows[-1]
    code = _dtype(x, "x")
    if A_log.dim() != 2 or B.dim() != len(rows) + 1:
        _fail("A_log: [D, N] and B, C: [..., G, N] expected")
    size, groups = A_log.shape[1], B.shape[-2]
    P = 0 if state is None else state.shape[0]
    bc = (*rows[:-1], groups, size)
    shape = capi.kda_scan_shape_t(
        0, 0, ch, size, groups, P, code, 0, _rows("x", x, t, rows, dev),
        _rows("dt", dt, t, rows, dev), 0 if z is None else _rows("z", z, t, rows, dev),
        _rows("B", B, t, bc, dev, 2), _rows("C", C, t, bc, dev, 2))
    f32 = torch.float32
    ptrs = (x.data_ptr(), dt.data_ptr(), _like("A_log", A_log, f32, (ch, size), dev),
            B.data_ptr(), C.data_ptr(), _like("D", D, f32, (ch,), dev), _ptr(z),
            _like("dt_bias", dt_bias, f32, (ch,), dev),
            _like("state", state, f32, (P, ch, size), dev))
    return ptrs, shape


def scan_prefill(x, dt, A_log, B, C, *, D=None, z=None, dt_bias=None, state=None,
                 state_indices=None, has_state=None, cu_seqlens=None,
                 num_seqs: Optional[int] = None, max_seqlen: int = 0, softplus: bool = True,
                 out=None, device_status=None, stream=None):
    """Selective state space scan over packed prompts (kda_scan_prefill).

    x, dt, z: [T, D] bf16 / fp16 / fp32 (z, the gate, may be None); A_log: [D, N] fp32 (the
    decay rates are -exp(A_log)); B, C: [T, G, N], channels dealt to the groups in equal runs;
    D, dt_bias: [D] fp32 or None; N at most 128.  The rows of each may lie at any distance.
    ``softplus``: the step is softplus(dt + dt_bias), else dt + dt_bias.  ``state``: [P, D, N]
    fp32 pool, updated in place; state_indices, has_state, cu_seqlens, num_seqs as in
    conv_prefill.  ``max_seqlen``: an upper bound on the lengths, a hint (0: not known).
    Returns out [T, D].
    """
    if x.dim() != 2:
        _fail("x: [T, D] expected")
    rows, dev = x.shape, _device(x)
    N, flags, pcu, pslot, phas, pstatus = _seqs(rows[0], cu_seqlens, num_seqs, state,
                                                state_indices, has_state, device_status, dev)
    ptrs, shape = _scan_args(x, dt, A_log, B, C, D, z, dt_bias, state, rows, dev)
    shape.num_seqs, shape.tokens, shape.max_seqlen = N, rows[0], max_seqlen
    if out is None:
        out = x.new_empty(rows)
    pout = _like("out", out, x.dtype, rows, dev)
    _call(_lib.kda_scan_prefill, "kda_scan_prefill", dev, stream, *ptrs, pslot, phas, pcu,
          _byref(shape), pout, pstatus, flags | (capi.KDA_SCAN_SOFTPLUS if softplus else 0))
    return out


def scan_decode(x, dt, A_log, B, C, state, *, D=None, z=None, dt_bias=None, state_indices=None,
                softplus: bool = True, out=None, step_states=None,
                return_step_states: bool = False, keep_state: bool = False, device_status=None,
                stream=None):
    """Selective state space scan of new tokens over a state pool (kda_scan_decode).

    x, dt, z: [N, T, D]; B, C: [N, T, G, N_state]; the rest as in scan_prefill;
    state_indices: [N] int32 (negative = padding row: zero output) or None (slot n).
    Returns (out, step_states): step_states [N, T, D, N_state] fp32, the state after every
    token, when requested.  ``keep_state`` leaves the pool as it was.
    """
    if x.dim() != 3:
        _fail("x: [N, T, D] expected")
    rows, dev = x.shape, _device(x)
    N, T, ch = rows
    ptrs, shape = _scan_args(x, dt, A_log, B, C, D, z, dt_bias, state, rows, dev)
    shape.num_seqs, shape.tokens = N, T
    pslot = _vector("state_indices", state_indices, _INT32, N, dev)
    pstatus = _vector("device_status", device_status, _INT32, 1, dev)
    if out is None:
        out = x.new_empty(rows)
    pout = _like("out", out, x.dtype, rows, dev)
    if step_states is None and return_step_states:
        step_states = state.new_empty((N, T, ch, shape.state_size))
    psteps = _like("step_states", step_states, torch.float32, (N, T, ch, shape.state_size), dev)
    _call(_lib.kda_scan_decode, "kda_scan_decode", dev, stream, *ptrs, pslot, _byref(shape), pout,
          psteps, pstatus, (capi.KDA_SCAN_SOFTPLUS if softplus else 0)
          | (capi.KDA_LAYER_KEEP_STATE if keep_state else 0))
    return out, step_states


_GATES = {"silu": 0, "sigmoid": capi.KDA_NORM_GATE_SIGMOID}


def rms_norm(x, weight=None, *, eps: float = 1e-6, residual=None, gate=None,
             gate_activation: str = "silu", out_dtype=None, group: int = 0, out=None,
             residual_out=None, scales=None, stream=None):
    """Root-mean-square norm of rows (kda_rms_norm).

    x: [T, W], or [T, H, W] for H rows a token (the heads of a KDA output); bf16 / fp16 / fp32,
    tokens at any distance.  weight: [W] fp32 or None.  ``residual`` is added before the norm;
    the sum is returned, rounded, in ``residual_out`` (new by default; may be residual or x
    itself).  ``gate`` multiplies the result by silu(gate) or sigmoid(gate).  With
    ``out_dtype=torch.float8_e4m3fn`` the output is in 8 bits with one fp32 scale per row
    (``group=0``) or per 128 elements (``group=128``): out * scale is the value.
    Returns (out, residual_out, scales); scales [T, (H,) ceil(W / group)].
    """
    full, t, dev = x.shape, x.dtype, _device(x)
    dims = len(full)
    if dims not in (2, 3):
        _fail("x: [T, W] or [T, H, W] expected")
    code, tail = _dtype(x, "x"), dims - 1
    T, W, H = full[0], full[-1], (full[1] if dims == 3 else 1)
    pw = _like("weight", weight, torch.float32, (W,), dev)
    gate_flag = _GATES.get(gate_activation)
    if gate_flag is None:
        _fail("gate_activation: 'silu' or 'sigmoid'")
    bits8 = out_dtype is torch.float8_e4m3fn
    if not bits8 and out_dtype not in (None, t):
        _fail("out_dtype: x's type or float8_e4m3fn")
    if group not in (0, 128) or (group and not bits8):
        _fail("group: 0, or 128 with an 8-bit output")
    if not bits8 and scales is not None:
        _fail("scales belong to an 8-bit output")
    otype = out_dtype if bits8 else t
    if out is None:
        out = x.new_empty(full, dtype=otype)
    pout = _like("out", out, otype, full, dev)
    xs = _rows("x", x, t, full, dev, tail)
    rs = ros = gs = 0
    if residual is not None:
        rs = _rows("residual", residual, t, full, dev, tail)
        if residual_out is None:
            residual_out = x.new_empty(full)
        ros = _rows("residual_out", residual_out, t, full, dev, tail)
    elif residual_out is not None:
        _fail("residual_out needs a residual")
    if gate is not None:
        gs = _rows("gate", gate, t, full, dev, tail)
    psc = None
    if bits8:
        sshape = (*full[:-1], -(-W // 128) if group else 1)
        if scales is None:
            scales = x.new_empty(sshape, dtype=torch.float32)
        psc = _like("scales", scales, torch.float32, sshape, dev)
    shape = capi.kda_norm_shape_t(T, H, W, group, code, capi.KDA_DTYPE_E4M3 if bits8 else code,
                                  xs, rs, ros, gs, eps, 0)
    _call(_lib.kda_rms_norm, "kda_rms_norm", dev, stream, x.data_ptr(), pw, _ptr(residual),
          _ptr(gate), _byref(shape), pout, _ptr(residual_out), psc, gate_flag)
    return out, residual_out, scales
