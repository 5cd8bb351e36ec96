"""The layer operators where offsets pass 32 bits, and foreign values beside what they read
(needs a B200; up to 12 GB)."""
import pytest
import torch

import kda_chunked_recurrent_b200 as K

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _far(rows, C, stride):
    """[rows, C] of a buffer whose last rows lie behind 2^31 elements; the rest is not touched."""
    assert rows * stride > 1 << 31
    x = torch.empty(rows, stride, dtype=BF, device="cuda")[:, 8:8 + C]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x.copy_(torch.randn(rows, C, generator=g, device="cuda"))
    return x


def test_rows_far_apart_give_what_near_rows_give():
    x = _far(9000, 64, 240000)
    near = x.contiguous()
    w = torch.randn(64, 4, device="cuda")
    cu = torch.tensor([0, 3000, 9000], dtype=torch.int32, device="cuda")
    assert torch.equal(K.conv_prefill(x, w, cu_seqlens=cu), K.conv_prefill(near, w, cu_seqlens=cu))
    pool = torch.randn(9000, 3, 64, device="cuda").to(BF)
    other = pool.clone()
    assert torch.equal(K.conv_decode(x[:, None], w, pool)[0], K.conv_decode(near[:, None], w, other)[0])
    assert torch.equal(pool, other)
    for a, b in zip(K.rms_norm(x, residual=x), K.rms_norm(near, residual=near)):
        assert a is b is None or torch.equal(a, b)
    A_log = torch.zeros(64, 16, device="cuda")
    B, C = near[:, None, :16].contiguous(), near[:, None, 16:32].contiguous()
    kw = dict(cu_seqlens=cu, dt_bias=torch.full((64,), -3.0, device="cuda"))
    assert torch.equal(K.scan_prefill(x, x, A_log, B, C, z=x, **kw),
                       K.scan_prefill(near, near, A_log, B, C, z=near, **kw))
    fB, fC = x[:, None, :16], x[:, None, 16:32]
    assert torch.equal(K.scan_prefill(near, near, A_log, fB, fC, **kw),
                       K.scan_prefill(near, near, A_log, B, C, **kw))


def test_more_than_2_31_outputs():
    T, C = 270000, 8000
    x = torch.zeros(T, C, dtype=BF, device="cuda")
    x[-6:] = torch.randn(6, C, device="cuda").to(BF)
    w = torch.randn(C, 4, device="cuda")
    tail = K.conv_prefill(x[-9:].contiguous(), w, silu=False)[-6:]
    assert torch.equal(K.conv_prefill(x, w, silu=False)[-6:], tail)
    assert torch.equal(K.conv_prefill(x, w, silu=False, parts=2)[1, -6:], tail[:, C // 2:])
    want = K.rms_norm(x[-6:].contiguous())[0]
    assert torch.equal(K.rms_norm(x)[0][-6:], want)


def test_a_slot_behind_2_31_elements():
    P, D, S = 2100, 8192, 128
    pool = torch.empty(P, D, S, device="cuda")
    near = torch.randn(1, D, S, device="cuda")
    pool[P - 1] = near[0]
    slot = torch.tensor([P - 1], dtype=torch.int32, device="cuda")
    x = torch.randn(1, 1, D, device="cuda").to(BF)
    B = torch.randn(1, 1, 1, S, device="cuda").to(BF)
    A_log = torch.zeros(D, S, device="cuda")
    a = K.scan_decode(x, x, A_log, B, B, pool, state_indices=slot)[0]
    b = K.scan_decode(x, x, A_log, B, B, near)[0]
    assert torch.equal(a, b) and torch.equal(pool[P - 1], near[0])
    y = torch.randn(40, D, device="cuda").to(BF)
    BC = torch.randn(40, 1, S, device="cuda").to(BF)
    a = K.scan_prefill(y, y, A_log, BC, BC, state=pool, state_indices=slot)
    b = K.scan_prefill(y, y, A_log, BC, BC, state=near)
    assert torch.equal(a, b) and torch.equal(pool[P - 1], near[0])


def test_foreign_nan_are_not_read():
    """NaN in the rows before and behind the sequences, between the slices of a projection, in
    slots that are not named, in rows of padding requests and in a state that is not continued."""
    nan = float("nan")
    buf = torch.full((80, 200), nan, device="cuda")
    buf[10:70, 20:84] = torch.randn(60, 64, device="cuda")
    x = buf.to(BF)[:, 20:84]
    w = torch.randn(64, 4, device="cuda")
    cu = torch.tensor([10, 10, 41, 70], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    cold = torch.tensor([True, False, False], device="cuda")
    cpool = torch.full((6, 3, 64), nan, dtype=BF, device="cuda")
    cpool[0] = 1
    spool = torch.full((6, 64, 16), nan, device="cuda")
    spool[0] = 1
    kw = dict(state_indices=slots, has_state=cold, cu_seqlens=cu)
    A_log = torch.zeros(64, 16, device="cuda")
    B = x[:, None, :16]
    y = K.conv_prefill(x, w, state=cpool, out=torch.zeros(80, 64, dtype=BF, device="cuda"), **kw)
    z = K.scan_prefill(x, x, A_log, B, B, z=x, state=spool, out=torch.zeros_like(y), **kw)
    for t in (y, z):
        assert torch.isfinite(t).all() and torch.all(t[:10] == 0) and torch.all(t[70:] == 0)
    for p in (cpool, spool):
        assert torch.isfinite(p[[0, 2, 4]]).all() and torch.isnan(p[[1, 3, 5]]).all()
    rows = torch.full((3, 1, 64), nan, dtype=BF, device="cuda")
    rows[0] = 1
    dead = torch.tensor([2, -1, 9], dtype=torch.int32, device="cuda")
    a = K.conv_decode(rows, w, cpool, state_indices=dead)[0]
    b = K.scan_decode(rows, rows, A_log, rows[..., None, :16], rows[..., None, :16], spool, z=rows,
                      state_indices=dead)[0]
    for t in (a, b):
        assert torch.isfinite(t[0]).all() and torch.all(t[1:] == 0)


def test_the_same_request_twice_reading_only():
    """Two sequences may name one slot where the pool is only read."""
    pool = torch.randn(2, 64, 16, device="cuda")
    before = pool.clone()
    x = torch.randn(2, 1, 64, device="cuda").to(BF)
    x[1] = x[0]
    B = torch.randn(1, 1, 1, 16, device="cuda").to(BF).expand(2, 1, 1, 16).contiguous()
    slots = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    y = K.scan_decode(x, x, torch.zeros(64, 16, device="cuda"), B, B, pool, state_indices=slots,
                      keep_state=True)[0]
    assert torch.equal(y[0], y[1]) and torch.equal(pool, before)
