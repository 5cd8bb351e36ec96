"""What the Python functions of the layer operators refuse, each for its own reason (needs a
GPU: tensors of another device are refused before anything else is looked at)."""
import pytest
import torch

import kda_chunked_recurrent_b200 as K

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def _conv():
    x, w, pool = z(8, 16), z(16, 4, dtype=F32), z(2, 3, 16)
    p, d = K.conv_prefill, K.conv_decode
    return [
        ("x: bfloat16", lambda: p(x.double(), w)), ("x: .T, C.", lambda: p(x[None], w)),
        ("weight: a contiguous", lambda: p(x, w.to(BF))), ("weight: a contiguous", lambda: p(x, w[:8])),
        ("weight: a contiguous", lambda: p(x, w.cpu())), ("weight: .channels", lambda: p(x, w[0])),
        ("weight: a tensor", lambda: p(x, None)), ("x: a tensor", lambda: p(3, w)),
        ("x: the elements", lambda: p(x.t().contiguous().t(), w)),
        ("x: rows must not overlap", lambda: p(x[:1].expand(8, 16), w)),
        ("parts must divide", lambda: p(x, w, parts=3)),
        ("without cu_seqlens", lambda: p(x, w, num_seqs=3)),
        ("cu_seqlens: 3", lambda: p(x, w, cu_seqlens=z(3, dtype=F32))),
        ("cu_seqlens: at least", lambda: p(x, w, cu_seqlens=z(1, dtype=I32))),
        ("num_seqs does not", lambda: p(x, w, num_seqs=2, cu_seqlens=z(2, dtype=I32))),
        ("need a state", lambda: p(x, w, has_state=z(1, dtype=torch.bool))),
        ("state: a contiguous", lambda: p(x, w, state=pool.float())),
        ("state: .slots", lambda: p(x, w, state=pool[0])),
        ("state: a contiguous", lambda: p(x, w, state=z(2, 16, 3))),
        ("state_indices: 1", lambda: p(x, w, state=pool, state_indices=z(2, dtype=I32))),
        ("has_state: 1", lambda: p(x, w, state=pool, has_state=z(1, dtype=I32))),
        ("device_status: 1", lambda: p(x, w, device_status=z(2, dtype=I32))),
        ("out: a contiguous", lambda: p(x, w, out=z(8, 16, dtype=F32))),
        ("out: a contiguous", lambda: p(x, w, parts=2, out=z(8, 16))),
        ("x: .N, T, C.", lambda: d(x, w, pool)),
        ("state: a tensor", lambda: d(x[None], w, None)),
        ("x: rows must lie at one", lambda: d(z(2, 8, 16)[:, ::3][:, :2], w, pool)),
        ("step_states: a contiguous", lambda: d(x[None], w, pool, step_states=z(1, 8, 2, 16))),
        ("state_indices: 1", lambda: d(x[None], w, pool, state_indices=z(1, dtype=torch.int64))),
    ]


def _scan():
    x, A, B = z(8, 16), z(16, 4, dtype=F32), z(8, 2, 4)
    p, d = K.scan_prefill, K.scan_decode
    return [
        ("dt: a", lambda: p(x, x.float(), A, B, B)), ("dt: a", lambda: p(x, x[:4], A, B, B)),
        ("A_log: a contiguous", lambda: p(x, x, A[:8], B, B)), ("A_log: .D, N.", lambda: p(x, x, A[0], B, B)),
        ("B: a", lambda: p(x, x, A, B[..., :2], B)), ("C: a", lambda: p(x, x, A, B, B[:, :1])),
        ("z: a", lambda: p(x, x, A, B, B, z=x[:, :8])),
        ("D: a contiguous", lambda: p(x, x, A, B, B, D=z(8, dtype=F32))),
        ("dt_bias: a contiguous", lambda: p(x, x, A, B, B, dt_bias=z(16))),
        ("state: a contiguous", lambda: p(x, x, A, B, B, state=z(1, 16, 5, dtype=F32))),
        ("B: the elements", lambda: p(x, x, A, z(8, 4, 2).transpose(1, 2), B)),
        ("x: .T, D.", lambda: p(x[0], x, A, B, B)),
        ("state: a tensor", lambda: d(x[None], x[None], A, B[None], B[None], None)),
        ("out: a contiguous", lambda: p(x, x, A, B, B, out=z(16, 8))),
        ("step_states: a contiguous", lambda: d(x[None], x[None], A, B[None], B[None],
                                                z(1, 16, 4, dtype=F32), step_states=z(1, 8, 16, 4))),
    ]


def _norm():
    x, e4 = z(8, 16), torch.float8_e4m3fn
    n = K.rms_norm
    return [
        ("x: .T, W.", lambda: n(x[0])), ("x: bfloat16", lambda: n(x.int())),
        ("weight: a contiguous", lambda: n(x, z(16))), ("residual: a", lambda: n(x, residual=x.float())),
        ("residual_out needs", lambda: n(x, residual_out=x)),
        ("residual_out: a", lambda: n(x, residual=x, residual_out=z(8, 8))),
        ("gate: a", lambda: n(x, gate=z(8, 8))), ("gate_activation", lambda: n(x, gate_activation="relu")),
        ("out_dtype", lambda: n(x, out_dtype=F32)), ("group: 0", lambda: n(x, group=128)),
        ("group: 0", lambda: n(x, out_dtype=e4, group=64)), ("scales belong", lambda: n(x, scales=z(8, 1))),
        ("scales: a contiguous", lambda: n(x, out_dtype=e4, scales=z(8, 2, dtype=F32))),
        ("out: a contiguous", lambda: n(x, out_dtype=e4, out=x)),
    ]


@pytest.mark.parametrize("cases", [_conv, _scan, _norm])
def test_refusals_name_what_is_wrong(cases):
    for message, call in cases():
        with pytest.raises(ValueError, match=message):
            call()
            print("accepted:", message)


def test_the_library_s_refusals_are_kda_errors():
    x, w, pool = z(2, 1, 16), z(16, 4, dtype=F32), z(1, 3, 16)
    with pytest.raises(K.KDAError, match="kda_conv_decode: invalid shape"):
        K.conv_decode(x, w, pool)                      # slot n without indices needs n + 1 slots
    with pytest.raises(K.KDAError, match="kda_conv_prefill: an output overlaps"):
        K.conv_prefill(x[:, 0], w, out=x[:, 0])
    with pytest.raises(K.KDAError, match="kda_conv_prefill: invalid shape"):
        K.conv_prefill(x[:, 0], z(16, 5, dtype=F32))
    with pytest.raises(K.KDAError, match="kda_rms_norm: unknown or unavailable option"):
        K.rms_norm(x[:, 0], eps=-1.0)
    with pytest.raises(K.KDAError, match="kda_scan_prefill: invalid shape"):
        K.scan_prefill(x[:, 0], x[:, 0], z(16, 129, dtype=F32), z(2, 1, 129), z(2, 1, 129))


def test_a_pool_without_slots_is_refused():
    """It would otherwise pass for no pool at all: sequences that leave nothing behind."""
    x, w, A, B = z(8, 16), z(16, 4, dtype=F32), z(16, 4, dtype=F32), z(8, 1, 4)
    with pytest.raises(ValueError, match="with a slot at least"):
        K.conv_prefill(x, w, state=z(0, 3, 16))
    with pytest.raises(ValueError, match="with a slot at least"):
        K.scan_prefill(x, x, A, B, B, state=z(0, 16, 4, dtype=F32))
    with pytest.raises(ValueError, match="with a slot at least"):
        K.conv_decode(x[None], w, z(0, 3, 16))
    with pytest.raises(ValueError, match="with a slot at least"):
        K.scan_decode(x[None], x[None], A, B[None], B[None], z(0, 16, 4, dtype=F32))


def test_empty_batches():
    """No rows: nothing to write, states as the rules have them."""
    x, w, pool = z(0, 16), z(16, 4, dtype=F32), z(2, 3, 16) + 1
    assert K.conv_prefill(x, w).shape == (0, 16)
    cu, cold = z(3, dtype=I32), torch.tensor([True, False], device="cuda")
    K.conv_prefill(x, w, state=pool, has_state=cold, cu_seqlens=cu)
    assert torch.all(pool[0] == 1) and torch.all(pool[1] == 0)
    spool = z(2, 16, 4, dtype=F32) + 1
    B = z(0, 1, 4)
    assert K.scan_prefill(x, x, z(16, 4, dtype=F32), B, B, state=spool, has_state=cold,
                          cu_seqlens=cu).shape == (0, 16)
    assert torch.all(spool[0] == 1) and torch.all(spool[1] == 0)
    assert K.rms_norm(x)[0].shape == (0, 16)
