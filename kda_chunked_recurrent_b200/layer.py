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
_byref = ctypes.byref


def _fail(what):
    raise ValueError(what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dtype(x, name):
    code = _DTYPE.get(x.dtype)
    if code is None:
        _fail(f"{name}: bfloat16, float16 or float32 expected, got {x.dtype}")
    return code


def _like(name, t, dtype, shape, dev):
    """A contiguous tensor of this type, shape and device, or None."""
    if t is None:
        return
    if t.dtype != dtype or tuple(t.shape) != shape or t.device != dev or not t.is_contiguous():
        _fail(f"{name}: a contiguous {dtype} tensor of shape {shape} on {dev} expected, got "
              f"{t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _rows(name, t, dtype, shape, dev, tail):
    """Elements between rows of a tensor [..., row] whose last ``tail`` dimensions are a
    contiguous row and whose leading dimensions step through rows at one stride."""
    if t.dtype != dtype or tuple(t.shape) != shape or t.device != dev:
        _fail(f"{name}: a {dtype} tensor of shape {shape} on {dev} expected, got {t.dtype} "
              f"{tuple(t.shape)} on {t.device}")
    st, n = t.stride(), 1
    for i in range(1, tail + 1):
        if shape[-i] != 1 and st[-i] != n:
            _fail(f"{name}: the elements of a row must be adjacent, strides {st}")
        n *= shape[-i]
    lead, row = shape[:-tail], None
    step = 1
    for i in range(len(lead) - 1, -1, -1):
        if lead[i] == 1:
            continue
        if row is None:
            row = st[i] // step if st[i] % step == 0 else -1
        if st[i] != row * step:
            _fail(f"{name}: rows must lie at one distance, strides {st}")
        step *= lead[i]
    if row is None:
        return n
    if row < n:
        if 0 in shape:
            return n
        _fail(f"{name}: rows must not overlap, strides {st}")
    return row


def _index(name, t, n, dev):
    if t is not None and (t.dtype != torch.int32 or t.numel() != n or t.device != dev
                          or not t.is_contiguous()):
        _fail(f"{name}: {n} contiguous int32 values on {dev} expected")


def _seqs(rows, cu_seqlens, num_seqs, state, state_indices, has_state, device_status, dev):
    """Number of sequences and the flag of the offsets' type."""
    flags = 0
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        if (cu_seqlens.dtype not in (torch.int32, torch.int64) or N < 1
                or cu_seqlens.device != dev or not cu_seqlens.is_contiguous()):
            _fail(f"cu_seqlens: at least two contiguous int32 or int64 offsets on {dev} expected")
        if num_seqs is not None and num_seqs != N:
            _fail("num_seqs does not agree with cu_seqlens")
        if cu_seqlens.dtype == torch.int64:
            flags = capi.KDA_LAYER_CU_SEQLENS_I64
    else:
        N = 1 if num_seqs is None else int(num_seqs)
        if N < 1 or rows % N:
            _fail("without cu_seqlens the rows are num_seqs sequences of one length")
    if state is None and (state_indices is not None or has_state is not None):
        _fail("state_indices and has_state need a state")
    _index("state_indices", state_indices, N, dev)
    _index("device_status", device_status, 1, dev)
    if has_state is not None and (has_state.dtype not in (torch.bool, torch.uint8)
                                  or has_state.numel() != N or has_state.device != dev
                                  or not has_state.is_contiguous()):
        _fail(f"has_state: {N} contiguous bool or uint8 values on {dev} expected")
    return N, flags


def _call(fn, where, dev, stream, *args):
    """Launch on the tensors' device: its current stream unless one is given."""
    if dev.type != "cuda":
        _fail(f"{where}: CUDA tensors expected, got {dev}")
    if torch.cuda.current_device() == dev.index:
        s = torch.cuda.current_stream(dev) if stream is None else stream
        rc = fn(*args, s.cuda_stream)
    else:
        with torch.cuda.device(dev):
            s = torch.cuda.current_stream(dev) if stream is None else stream
            rc = fn(*args, s.cuda_stream)
    if rc != capi.KDA_OK:
        raise KDAError(rc, where)


def _conv_weight(weight, bias, C, dev):
    if weight.dim() != 2:
        _fail("weight: [channels, width] expected")
    W = weight.shape[1]
    _like("weight", weight, torch.float32, (C, W), dev)
    _like("bias", bias, torch.float32, (C,), dev)
    return W


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
    dev, (T, C) = x.device, x.shape
    code = _dtype(x, "x")
    W = _conv_weight(weight, bias, C, dev)
    N, flags = _seqs(T, cu_seqlens, num_seqs, state, state_indices, has_state, device_status, dev)
    P = 0
    if state is not None:
        P = state.shape[0]
        _like("state", state, x.dtype, (P, W - 1, C), dev)
    oshape = _parts_shape((T,), C, parts)
    if out is None:
        out = torch.empty(oshape, dtype=x.dtype, device=dev)
    else:
        _like("out", out, x.dtype, oshape, dev)
    shape = capi.kda_conv_shape_t(N, T, C, W, parts, P, code, 0,
                                  _rows("x", x, x.dtype, (T, C), dev, 1))
    _call(capi.kda_conv_prefill, "kda_conv_prefill", dev, stream, x.data_ptr(),
          weight.data_ptr(), _ptr(bias), _ptr(state), _ptr(state_indices), _ptr(has_state),
          _ptr(cu_seqlens), _byref(shape), out.data_ptr(), _ptr(device_status),
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
    dev, (N, T, C) = x.device, x.shape
    code = _dtype(x, "x")
    W = _conv_weight(weight, bias, C, dev)
    P = state.shape[0]
    _like("state", state, x.dtype, (P, W - 1, C), dev)
    _index("state_indices", state_indices, N, dev)
    _index("device_status", device_status, 1, dev)
    oshape = _parts_shape((N, T), C, parts)
    if out is None:
        out = torch.empty(oshape, dtype=x.dtype, device=dev)
    else:
        _like("out", out, x.dtype, oshape, dev)
    if step_states is None and return_step_states:
        step_states = torch.empty(N, T, W - 1, C, dtype=x.dtype, device=dev)
    elif step_states is not None:
        _like("step_states", step_states, x.dtype, (N, T, W - 1, C), dev)
    shape = capi.kda_conv_shape_t(N, T, C, W, parts, P, code, 0,
                                  _rows("x", x, x.dtype, (N, T, C), dev, 1))
    _call(capi.kda_conv_decode, "kda_conv_decode", dev, stream, x.data_ptr(), weight.data_ptr(),
          _ptr(bias), state.data_ptr(), _ptr(state_indices), _byref(shape), out.data_ptr(),
          _ptr(step_states), _ptr(device_status),
          (capi.KDA_CONV_SILU if silu else 0) | (capi.KDA_LAYER_KEEP_STATE if keep_state else 0))
    return out, step_states


def _scan_args(x, dt, A_log, B, C, D, z, dt_bias, state, lead):
    """Check the operands that both forms share; the shape struct without its sequences."""
    dev, ch = x.device, x.shape[-1]
    code = _dtype(x, "x")
    if A_log.dim() != 2 or B.dim() != len(lead) + 2:
        _fail("A_log: [D, N] and B, C: [..., G, N] expected")
    size, groups = A_log.shape[1], B.shape[-2]
    _like("A_log", A_log, torch.float32, (ch, size), dev)
    _like("D", D, torch.float32, (ch,), dev)
    _like("dt_bias", dt_bias, torch.float32, (ch,), dev)
    P = 0
    if state is not None:
        P = state.shape[0]
        _like("state", state, torch.float32, (P, ch, size), dev)
    rows, bc = lead + (ch,), lead + (groups, size)
    shape = capi.kda_scan_shape_t(
        0, 0, ch, size, groups, P, code, 0, _rows("x", x, x.dtype, rows, dev, 1),
        _rows("dt", dt, x.dtype, rows, dev, 1),
        0 if z is None else _rows("z", z, x.dtype, rows, dev, 1),
        _rows("B", B, x.dtype, bc, dev, 2), _rows("C", C, x.dtype, bc, dev, 2))
    return shape


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
    dev, (T, ch) = x.device, x.shape
    N, flags = _seqs(T, cu_seqlens, num_seqs, state, state_indices, has_state, device_status, dev)
    shape = _scan_args(x, dt, A_log, B, C, D, z, dt_bias, state, (T,))
    shape.num_seqs, shape.tokens, shape.max_seqlen = N, T, max_seqlen
    if out is None:
        out = torch.empty(T, ch, dtype=x.dtype, device=dev)
    else:
        _like("out", out, x.dtype, (T, ch), dev)
    _call(capi.kda_scan_prefill, "kda_scan_prefill", dev, stream, x.data_ptr(), dt.data_ptr(),
          A_log.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z), _ptr(dt_bias),
          _ptr(state), _ptr(state_indices), _ptr(has_state), _ptr(cu_seqlens), _byref(shape),
          out.data_ptr(), _ptr(device_status),
          flags | (capi.KDA_SCAN_SOFTPLUS if softplus else 0))
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
    dev, (N, T, ch) = x.device, x.shape
    shape = _scan_args(x, dt, A_log, B, C, D, z, dt_bias, state, (N, T))
    shape.num_seqs, shape.tokens = N, T
    _index("state_indices", state_indices, N, dev)
    _index("device_status", device_status, 1, dev)
    if out is None:
        out = torch.empty(N, T, ch, dtype=x.dtype, device=dev)
    else:
        _like("out", out, x.dtype, (N, T, ch), dev)
    size = shape.state_size
    if step_states is None and return_step_states:
        step_states = torch.empty(N, T, ch, size, dtype=torch.float32, device=dev)
    elif step_states is not None:
        _like("step_states", step_states, torch.float32, (N, T, ch, size), dev)
    _call(capi.kda_scan_decode, "kda_scan_decode", dev, stream, x.data_ptr(), dt.data_ptr(),
          A_log.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z), _ptr(dt_bias),
          state.data_ptr(), _ptr(state_indices), _byref(shape), out.data_ptr(),
          _ptr(step_states), _ptr(device_status),
          (capi.KDA_SCAN_SOFTPLUS if softplus else 0)
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
    if x.dim() not in (2, 3):
        _fail("x: [T, W] or [T, H, W] expected")
    dev, full = x.device, tuple(x.shape)
    code = _dtype(x, "x")
    T, W, H = full[0], full[-1], (full[1] if len(full) == 3 else 1)
    tail = len(full) - 1
    _like("weight", weight, torch.float32, (W,), dev)
    if gate_activation not in _GATES:
        _fail("gate_activation: 'silu' or 'sigmoid'")
    bits8 = out_dtype == torch.float8_e4m3fn
    if not bits8 and out_dtype not in (None, x.dtype):
        _fail("out_dtype: x's type or float8_e4m3fn")
    if group not in (0, 128) or (group and not bits8):
        _fail("group: 0, or 128 with an 8-bit output")
    if not bits8 and scales is not None:
        _fail("scales belong to an 8-bit output")
    otype = torch.float8_e4m3fn if bits8 else x.dtype
    if out is None:
        out = torch.empty(full, dtype=otype, device=dev)
    else:
        _like("out", out, otype, full, dev)
    rs = ros = gs = 0
    if residual is not None:
        rs = _rows("residual", residual, x.dtype, full, dev, tail)
        if residual_out is None:
            residual_out = torch.empty(full, dtype=x.dtype, device=dev)
        ros = _rows("residual_out", residual_out, x.dtype, full, dev, tail)
    elif residual_out is not None:
        _fail("residual_out needs a residual")
    if gate is not None:
        gs = _rows("gate", gate, x.dtype, full, dev, tail)
    if bits8:
        sshape = full[:-1] + (-(-W // 128) if group else 1,)
        if scales is None:
            scales = torch.empty(sshape, dtype=torch.float32, device=dev)
        else:
            _like("scales", scales, torch.float32, sshape, dev)
    shape = capi.kda_norm_shape_t(T, H, W, group, code,
                                  capi.KDA_DTYPE_E4M3 if bits8 else code,
                                  _rows("x", x, x.dtype, full, dev, tail), rs, ros, gs, eps, 0)
    _call(capi.kda_rms_norm, "kda_rms_norm", dev, stream, x.data_ptr(), _ptr(weight),
          _ptr(residual), _ptr(gate), _byref(shape), out.data_ptr(), _ptr(residual_out),
          _ptr(scales), _GATES[gate_activation])
    return out, residual_out, scales
