"""The layer operators' refusals, on the host: the C entry points check their arguments
before any CUDA call, and the Python functions check types, shapes, strides and devices."""
import ctypes
import os
import re

import pytest
import torch

import kda_chunked_recurrent_b200 as K
from kda_chunked_recurrent_b200 import capi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE, MB = 0x7F0000000000, 1 << 20
NO_GPU = not torch.cuda.is_available()


def test_every_declared_entry_point_is_exported():
    src = open(os.path.join(ROOT, "include", "kda_layer.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(kda_[a-z_]+)\s*\(", src)))
    assert names == ["kda_conv_decode", "kda_conv_prefill", "kda_rms_norm", "kda_scan_decode",
                     "kda_scan_prefill"]
    lib = ctypes.CDLL(capi.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(capi.kda_conv_shape_t) == 40
    assert ctypes.sizeof(capi.kda_scan_shape_t) == 72
    assert ctypes.sizeof(capi.kda_norm_shape_t) == 64


# ---- C entry points with addresses that are never read --------------------------------
def conv(decode=False, shape=None, **over):
    s = dict(num_seqs=4, tokens=1 if decode else 64, channels=96, width=4, parts=3, pool_size=8,
             dtype=0, reserved=0, x_stride=96)
    s.update(shape or {})
    a = dict(x=BASE, weight=BASE + MB, bias=BASE + 2 * MB, state=BASE + 3 * MB,
             idx=BASE + 4 * MB, has=BASE + 5 * MB, cu=BASE + 6 * MB, out=BASE + 7 * MB,
             steps=None, status=BASE + 9 * MB, flags=capi.KDA_CONV_SILU)
    a.update(over)
    sh = capi.kda_conv_shape_t(**s)
    if decode:
        return capi.kda_conv_decode(a["x"], a["weight"], a["bias"], a["state"], a["idx"], sh,
                                    a["out"], a["steps"], a["status"], a["flags"], None)
    return capi.kda_conv_prefill(a["x"], a["weight"], a["bias"], a["state"], a["idx"], a["has"],
                                 a["cu"], sh, a["out"], a["status"], a["flags"], None)


def scan(decode=False, shape=None, **over):
    s = dict(num_seqs=4, tokens=1 if decode else 64, channels=96, state_size=16, groups=2,
             pool_size=8, dtype=0, max_seqlen=0, x_stride=96, dt_stride=96, z_stride=96,
             b_stride=64, c_stride=64)
    s.update(shape or {})
    a = dict(x=BASE, dt=BASE + MB, A=BASE + 2 * MB, B=BASE + 3 * MB, C=BASE + 4 * MB,
             D=BASE + 5 * MB, z=BASE + 6 * MB, bias=BASE + 7 * MB, state=BASE + 8 * MB,
             idx=BASE + 9 * MB, has=BASE + 10 * MB, cu=BASE + 11 * MB, out=BASE + 12 * MB,
             steps=None, status=BASE + 14 * MB, flags=capi.KDA_SCAN_SOFTPLUS)
    a.update(over)
    sh = capi.kda_scan_shape_t(**s)
    if decode:
        return capi.kda_scan_decode(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"],
                                    a["bias"], a["state"], a["idx"], sh, a["out"], a["steps"],
                                    a["status"], a["flags"], None)
    return capi.kda_scan_prefill(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"],
                                 a["bias"], a["state"], a["idx"], a["has"], a["cu"], sh,
                                 a["out"], a["status"], a["flags"], None)


def norm(shape=None, **over):
    s = dict(tokens=16, heads=2, width=128, group=0, dtype=0, out_dtype=0, x_stride=256,
             residual_stride=256, residual_out_stride=256, gate_stride=256, eps=1e-6, reserved=0)
    s.update(shape or {})
    a = dict(x=BASE, weight=BASE + MB, res=BASE + 2 * MB, gate=BASE + 3 * MB, out=BASE + 4 * MB,
             res_out=BASE + 5 * MB, scales=None, flags=0)
    a.update(over)
    return capi.kda_rms_norm(a["x"], a["weight"], a["res"], a["gate"], capi.kda_norm_shape_t(**s),
                             a["out"], a["res_out"], a["scales"], a["flags"], None)


@pytest.mark.skipif(not NO_GPU, reason="would launch on addresses that are none")
def test_valid_arguments_reach_the_device_check():
    dev = capi.KDA_ERR_UNSUPPORTED_DEVICE
    assert conv() == dev and conv(True) == dev and scan() == dev and scan(True) == dev
    assert conv(bias=None, state=None, idx=None, has=None, status=None, cu=None) == dev
    assert conv(True, steps=BASE + 8 * MB, flags=capi.KDA_LAYER_KEEP_STATE) == dev
    assert conv(flags=capi.KDA_LAYER_CU_SEQLENS_I64) == dev
    assert scan(D=None, z=None, bias=None, state=None, idx=None, has=None, cu=None) == dev
    assert scan(True, steps=BASE + 20 * MB, flags=capi.KDA_LAYER_KEEP_STATE) == dev
    e4 = dict(out_dtype=capi.KDA_DTYPE_E4M3, group=128)
    assert norm() == dev and norm(e4, scales=BASE + 6 * MB) == dev
    assert norm(weight=None, res=None, gate=None, res_out=None) == dev
    # in place: out over x, the residual over itself or x
    assert norm(out=BASE, res=None, res_out=None) == dev
    assert norm(res_out=BASE + 2 * MB) == dev and norm(res_out=BASE) == dev


@pytest.mark.parametrize("decode", [False, True])
def test_null_pointers_refused(decode):
    for f in ("x", "weight", "out"):
        assert conv(decode, **{f: None}) == capi.KDA_ERR_NULL_ARG
    for f in ("x", "dt", "A", "B", "C", "out"):
        assert scan(decode, **{f: None}) == capi.KDA_ERR_NULL_ARG
    # indices without a pool, and decode without one
    assert conv(decode, state=None) == capi.KDA_ERR_NULL_ARG
    assert scan(decode, state=None) == capi.KDA_ERR_NULL_ARG


def test_null_pointers_of_the_norm_refused():
    assert norm(x=None) == capi.KDA_ERR_NULL_ARG and norm(out=None) == capi.KDA_ERR_NULL_ARG
    assert norm(res=None) == capi.KDA_ERR_NULL_ARG                       # residual_out without
    assert norm(dict(out_dtype=capi.KDA_DTYPE_E4M3)) == capi.KDA_ERR_NULL_ARG     # no scales


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("bad", [dict(num_seqs=0), dict(tokens=-1), dict(channels=0),
                                 dict(width=1), dict(width=5), dict(parts=0), dict(parts=5),
                                 dict(x_stride=95), dict(pool_size=0), dict(channels=1 << 25)])
def test_conv_bad_shapes_refused(decode, bad):
    if "channels" in bad:
        bad = dict(bad, parts=1, x_stride=1 << 26)
    assert conv(decode, bad) == capi.KDA_ERR_BAD_SHAPE


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("bad", [dict(num_seqs=0), dict(tokens=-1), dict(channels=0),
                                 dict(state_size=0), dict(state_size=129), dict(groups=0),
                                 dict(groups=5), dict(x_stride=95), dict(dt_stride=95),
                                 dict(z_stride=95), dict(b_stride=31), dict(c_stride=31),
                                 dict(pool_size=0), dict(max_seqlen=-1)])
def test_scan_bad_shapes_refused(decode, bad):
    assert scan(decode, bad) == capi.KDA_ERR_BAD_SHAPE


def test_more_shapes_refused():
    S = capi.KDA_ERR_BAD_SHAPE
    assert conv(True, dict(tokens=0)) == S and scan(True, dict(tokens=0)) == S
    # more rows than 32 bits count
    assert conv(True, dict(num_seqs=1 << 20, tokens=1 << 12, pool_size=1 << 21)) == S
    # equal lengths need rows divisible by the sequences; slot n needs n + 1 slots
    assert conv(shape=dict(tokens=65), cu=None) == S and scan(shape=dict(tokens=65), cu=None) == S
    assert conv(idx=None, shape=dict(pool_size=3)) == S
    assert scan(True, idx=None, shape=dict(pool_size=3)) == S
    for bad in (dict(tokens=-1), dict(heads=0), dict(width=0), dict(width=32769, heads=1,
                x_stride=1 << 20, residual_stride=1 << 20, residual_out_stride=1 << 20,
                gate_stride=1 << 20), dict(x_stride=255), dict(residual_stride=255),
                dict(residual_out_stride=255), dict(gate_stride=255)):
        assert norm(bad) == S, bad
    assert norm(dict(tokens=0), x=None, out=None) == capi.KDA_OK       # nothing to do


def test_unknown_options_refused():
    B = capi.KDA_ERR_BAD_OPTION
    assert conv(flags=1 << 9) == B and scan(flags=1 << 9) == B and norm(flags=2) == B
    assert conv(flags=capi.KDA_LAYER_KEEP_STATE) == B        # decode only
    assert scan(True, flags=capi.KDA_LAYER_CU_SEQLENS_I64) == B
    assert conv(cu=None, flags=capi.KDA_LAYER_CU_SEQLENS_I64) == B
    assert conv(shape=dict(dtype=3)) == B and scan(shape=dict(dtype=-1)) == B
    assert conv(shape=dict(reserved=1)) == B and norm(dict(reserved=1)) == B
    for bad in (dict(dtype=3), dict(out_dtype=2), dict(group=64), dict(group=128),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert norm(bad) == B, bad
    assert norm(scales=BASE + 6 * MB) == B


def test_misaligned_pointers_refused():
    M = capi.KDA_ERR_MISALIGNED
    for f, d in dict(x=1, weight=2, bias=2, state=1, idx=2, cu=2, out=1, status=2).items():
        assert conv(**{f: {"x": BASE, "weight": BASE + MB, "bias": BASE + 2 * MB,
                           "state": BASE + 3 * MB, "idx": BASE + 4 * MB, "cu": BASE + 6 * MB,
                           "out": BASE + 7 * MB, "status": BASE + 9 * MB}[f] + d}) == M, f
    assert conv(cu=BASE + 6 * MB + 4, flags=capi.KDA_LAYER_CU_SEQLENS_I64) == M
    assert scan(state=BASE + 8 * MB + 8) == M and scan(True, steps=BASE + 20 * MB + 4) == M
    assert scan(A=BASE + 2 * MB + 2) == M and scan(B=BASE + 3 * MB + 1) == M
    assert norm(x=BASE + 1) == M and norm(weight=BASE + MB + 2) == M
    assert norm(dict(dtype=2, out_dtype=2), gate=BASE + 3 * MB + 2) == M


def test_aliasing_refused():
    A = capi.KDA_ERR_OUT_ALIAS
    for over in (dict(out=BASE), dict(out=BASE + 3 * MB), dict(state=BASE + 64),
                 dict(status=BASE + 7 * MB), dict(out=BASE + 4 * MB), dict(state=BASE + 5 * MB)):
        assert conv(**over) == A, over
    assert conv(True, steps=BASE + 3 * MB + 96) == A
    for over in (dict(out=BASE), dict(out=BASE + 6 * MB), dict(state=BASE + 2 * MB),
                 dict(status=BASE + 12 * MB), dict(out=BASE + 8 * MB)):
        assert scan(**over) == A, over
    assert scan(True, steps=BASE + 8 * MB + 16) == A
    assert norm(out=BASE + 2) == A and norm(out=BASE + 2 * MB) == A
    assert norm(dict(x_stride=300), out=BASE) == A           # in place needs the same rows
    assert norm(res_out=BASE + 2 * MB, shape=dict(residual_out_stride=512)) == A
    assert norm(out=BASE, res_out=BASE) == A
    assert norm(dict(out_dtype=3), out=BASE, scales=BASE + 6 * MB) == A
    assert norm(dict(out_dtype=3), scales=BASE + 3 * MB) == A


# ---- the Python functions -------------------------------------------------------------
def test_python_checks():
    bf, f32 = torch.bfloat16, torch.float32
    x, w = torch.zeros(8, 16, dtype=bf), torch.zeros(16, 4)
    ok = dict(state=torch.zeros(2, 3, 16, dtype=bf), state_indices=torch.zeros(1, dtype=torch.int32))
    bad = [lambda: K.conv_prefill(x, w),                                    # not on a GPU
           lambda: K.conv_prefill(x.double(), w),
           lambda: K.conv_prefill(x[None], w),
           lambda: K.conv_prefill(x, w.to(bf)),
           lambda: K.conv_prefill(x, w[:8]),
           lambda: K.conv_prefill(x.t().contiguous().t(), w),
           lambda: K.conv_prefill(x[:1].expand(8, 16), w),
           lambda: K.conv_prefill(x, w, parts=3),
           lambda: K.conv_prefill(x, w, num_seqs=3),
           lambda: K.conv_prefill(x, w, cu_seqlens=torch.zeros(3)),
           lambda: K.conv_prefill(x, w, num_seqs=2, cu_seqlens=torch.zeros(2, dtype=torch.int32)),
           lambda: K.conv_prefill(x, w, has_state=torch.ones(1, dtype=torch.bool)),
           lambda: K.conv_prefill(x, w, **dict(ok, state=ok["state"].float())),
           lambda: K.conv_prefill(x, w, **dict(ok, state_indices=torch.zeros(1))),
           lambda: K.conv_prefill(x, w, out=torch.zeros(8, 16)),
           lambda: K.conv_decode(x, w, ok["state"]),
           lambda: K.conv_decode(x.view(2, 4, 16), w, ok["state"][:, :2])]
    B = torch.zeros(8, 2, 4, dtype=bf)
    A = torch.zeros(16, 4)
    bad += [lambda: K.scan_prefill(x, x, A, B, B),                          # not on a GPU
            lambda: K.scan_prefill(x, x.float(), A, B, B),
            lambda: K.scan_prefill(x, x[:4], A, B, B),
            lambda: K.scan_prefill(x, x, A[:8], B, B),
            lambda: K.scan_prefill(x, x, A, B[..., :2], B[..., :2]),
            lambda: K.scan_prefill(x, x, A, B, B[:, :1]),
            lambda: K.scan_prefill(x, x, A, B, B, z=x[:, :8]),
            lambda: K.scan_prefill(x, x, A, B, B, D=torch.zeros(8)),
            lambda: K.scan_prefill(x, x, A, B, B, state=torch.zeros(1, 16, 5)),
            lambda: K.scan_prefill(x, x, A, B.transpose(1, 2), B.transpose(1, 2)),
            lambda: K.scan_decode(x, x, A, B, B, torch.zeros(1, 16, 4))]
    bad += [lambda: K.rms_norm(x),                                          # not on a GPU
            lambda: K.rms_norm(x[0]), lambda: K.rms_norm(x.int()),
            lambda: K.rms_norm(x, torch.zeros(16, dtype=bf)),
            lambda: K.rms_norm(x, residual=x.float()),
            lambda: K.rms_norm(x, residual_out=x),
            lambda: K.rms_norm(x, gate=x, gate_activation="relu"),
            lambda: K.rms_norm(x, out_dtype=f32), lambda: K.rms_norm(x, group=128),
            lambda: K.rms_norm(x, out_dtype=torch.float8_e4m3fn, group=64),
            lambda: K.rms_norm(x, scales=torch.zeros(8, 1))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted:", i)
