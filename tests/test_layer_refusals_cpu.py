"""What the Python functions of the layer operators refuse, on CPU tensors: all that the checks on a
GPU ask (tests/test_layer_checks_gpu.py), each with its message, and last of all that the tensors
are on none."""
import pytest
import torch

import kda_chunked_recurrent_b200 as K
from tests import test_layer_checks_gpu as checks

NO_GPU = "x: a CUDA tensor expected, got one on cpu"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


# (a tensor on the CPU where the others are on a GPU is the one case that has no fault here)
@pytest.mark.parametrize("cases,elsewhere", [("_conv", 1), ("_scan", 0), ("_norm", 0)])
def test_every_refusal_comes_before_the_device(monkeypatch, cases, elsewhere):
    monkeypatch.setattr(checks, "z", z)
    fits = 0
    for message, call in getattr(checks, cases)():
        with pytest.raises(ValueError) as e:
            call()
        if str(e.value).startswith(NO_GPU):
            fits += 1
            continue
        e.match(message)
    assert fits == elsewhere


def test_a_pool_without_slots(monkeypatch):
    monkeypatch.setattr(checks, "z", z)
    checks.test_a_pool_without_slots_is_refused()


@pytest.mark.parametrize("call", [
    lambda x, w, p, i: K.conv_prefill(x, w, state=p, state_indices=i, out=z(8, 16)),
    lambda x, w, p, i: K.conv_decode(x[None], w, p, state_indices=i, return_step_states=True),
    lambda x, w, p, i: K.scan_prefill(x, x, w, z(8, 2, 4), z(8, 2, 4), D=z(16, dtype=F32)),
    lambda x, w, p, i: K.scan_decode(x[None], x[None], w, z(1, 8, 2, 4), z(1, 8, 2, 4),
                                     z(2, 16, 4, dtype=F32), step_states=z(1, 8, 16, 4, dtype=F32)),
    lambda x, w, p, i: K.rms_norm(x, residual=x, gate=x, residual_out=x),
    lambda x, w, p, i: K.rms_norm(x, out_dtype=torch.float8_e4m3fn, scales=z(8, 1, dtype=F32)),
], ids=["conv_prefill", "conv_decode", "scan_prefill", "scan_decode", "rms_norm", "rms_norm 8 bits"])
def test_all_fits_but_the_device(call):
    x, w, pool, slots = z(8, 16), z(16, 4, dtype=F32), z(2, 3, 16), z(1, dtype=I32)
    before = pool.clone()
    with pytest.raises(ValueError, match=NO_GPU):
        call(x, w, pool, slots)
    assert torch.equal(pool, before)


def test_arguments_of_other_kinds_are_type_errors():
    x, w = z(8, 16), z(16, 4, dtype=F32)
    with pytest.raises(TypeError):
        K.conv_prefill(x, w, parts="3")
    with pytest.raises(TypeError):
        K.rms_norm(x, eps="1e-6")
    with pytest.raises(TypeError):
        K.scan_prefill(x, x, w, z(8, 2, 4), z(8, 2, 4), max_seqlen=1.5)
