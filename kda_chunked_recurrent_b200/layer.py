"""The layer operators around the KDA recurrence on device tensors (include/kda_layer.h):
short causal convolution, selective state space scan and root-mean-square norm.

Like ``prefill`` and ``decode`` these functions only check and marshal arguments and allocate
outputs (in the native binding, csrc/kda_layer_bind.cpp); all arithmetic is in the library's
kernels.  A call is one launch on ``stream`` (the tensors' device's current stream by
default), reads nothing back and can be captured in a CUDA graph.  New outputs are allocated on
the same stream, as under ``torch.cuda.stream(stream)``.  Wrong types, shapes, strides or devices
raise ValueError, what the library refuses raises KDAError.
"""
from __future__ import annotations

import os
from typing import Optional

import torch

from . import KDAError, capi

_PKG = os.path.dirname(os.path.abspath(__file__))
if not os.path.exists(os.path.join(_PKG, "_layer_bind.so")):
    raise ImportError(f"{_PKG}/_layer_bind.so is missing: build it with `python -m "
                      "kda_chunked_recurrent_b200.build` (there is no fallback implementation)")
from . import _layer_bind as _bind  # noqa: E402


def _fail(code, where):
    raise KDAError(code, where)


_bind.set_fail(_fail)


def _handle(stream):
    return None if stream is None else stream.cuda_stream


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
    return _bind.conv_prefill(x, weight, bias, state, state_indices, has_state, cu_seqlens,
                              num_seqs, parts, silu, out, device_status, _handle(stream))


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
    return _bind.conv_decode(x, weight, bias, state, state_indices, parts, silu, out, step_states,
                             return_step_states, keep_state, device_status, _handle(stream))


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
    return _bind.scan_prefill(x, dt, A_log, B, C, D, z, dt_bias, state, state_indices, has_state,
                              cu_seqlens, num_seqs, max_seqlen, softplus, out, device_status,
                              _handle(stream))


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
    return _bind.scan_decode(x, dt, A_log, B, C, D, z, dt_bias, state, state_indices, softplus, out,
                             step_states, return_step_states, keep_state, device_status,
                             _handle(stream))


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
    flags = _GATES.get(gate_activation)
    if flags is None:
        raise ValueError("gate_activation: 'silu' or 'sigmoid'")
    bits8 = out_dtype is torch.float8_e4m3fn
    if not bits8 and out_dtype is not None and out_dtype is not x.dtype:
        raise ValueError("out_dtype: x's type or float8_e4m3fn")
    return _bind.rms_norm(x, weight, eps, residual, gate, flags, bits8, group, out, residual_out,
                          scales, _handle(stream))
