"""Padding rows: every negative slot, whatever its value, and every slot behind the pool
(needs a B200)."""
import numpy as np
import pytest
import torch

import kda_chunked_recurrent_b200 as K
from tests.layer_reference import close, conv, f64

pytestmark = pytest.mark.gpu
LEAST, MOST = -2 ** 31, 2 ** 31 - 1


def _slots(N, P, g):
    """Live slots with -2, the least and other negative entries and some behind the pool among
    them, each at even and at odd places, beside live neighbours and beside one another."""
    s = torch.randperm(P, generator=g)[:N].int()
    for i, bad in enumerate([-2, -2, LEAST, P, -2, -1, LEAST, MOST, -7]):
        s[(2 + 5 * i) % N::41] = bad
    s[N - 1] = -2
    return s


# few sequences, and enough of them that a thread takes two
@pytest.mark.parametrize("N", [7, 46, 1301])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("C", [7, 8])
def test_conv_tokens(N, T, C):
    g = torch.Generator().manual_seed(N + T)
    P = N + 5
    x, w = torch.randn(N, T, C, generator=g).cuda(), torch.randn(C, 4, generator=g).cuda()
    pool = torch.randn(P, 3, C, generator=g).cuda()
    before, slots = pool.clone(), _slots(N, P, g)
    out = torch.full_like(x, 7.0)
    steps = torch.full((N, T, 3, C), 8.0, device="cuda") if T > 1 else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.conv_decode(x, w, pool, state_indices=slots.cuda(), out=out, step_states=steps,
                  device_status=status)
    torch.cuda.synchronize()
    out_of_range = any(s >= P for s in slots.tolist())
    assert status.item() == (K.capi.KDA_ERR_BAD_STATE_INDEX if out_of_range else 0)
    live = set()
    for n, s in enumerate(slots.tolist()):
        if not 0 <= s < P:
            assert torch.all(out[n] == 0), f"padding row {n}, slot {s}"
            assert steps is None or torch.all(steps[n] == 8.0)
            continue
        live.add(s)
        y, bound, new = conv(f64(x[n]), f64(w), None, f64(before[s]), True)
        close(out[n], y, bound, torch.float32, f"row {n}, slot {s}")
        assert np.array_equal(f64(pool[s]), new), f"state of row {n}"
    rest = [s for s in range(P) if s not in live]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("N", [7, 46, 1301])
@pytest.mark.parametrize("T", [1, 3])
def test_scan_tokens(N, T):
    """Live rows give what they give beside padding rows of -1."""
    g = torch.Generator().manual_seed(N + T)
    P, D, S = N + 5, 24, 16
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, dt, B, C, A_log = r(N, T, D), r(N, T, D), r(N, T, 1, S), r(N, T, 1, S), r(D, S)
    pool, slots = r(P, D, S), _slots(N, P, g)
    before, other = pool.clone(), pool.clone()
    out = torch.full_like(x, 7.0)
    K.scan_decode(x, dt, A_log, B, C, pool, state_indices=slots.cuda(), out=out)
    dead = (slots < 0) | (slots >= P)
    plain = torch.where(dead, torch.full_like(slots, -1), slots)
    want = K.scan_decode(x, dt, A_log, B, C, other, state_indices=plain.cuda())[0]
    assert torch.equal(out, want) and torch.equal(pool, other)
    assert torch.all(out[dead.cuda()] == 0) and torch.isfinite(out).all()
    rest = sorted(set(range(P)) - set(slots[~dead].tolist()))
    assert torch.equal(pool[rest], before[rest])


def test_prompts():
    """A negative slot of any value starts from zeros and leaves nothing."""
    g = torch.Generator().manual_seed(3)
    lens, D, S = [9, 0, 40, 2, 33], 24, 16
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, dt, B, C, A_log, w = r(84, D), r(84, D), r(84, 1, S), r(84, 1, S), r(D, S), r(D, 4)
    cpool, spool = r(4, 3, D), r(4, D, S)
    cb, sb = cpool.clone(), spool.clone()
    slots = torch.tensor([-2, LEAST, -2, MOST, -9], dtype=torch.int32, device="cuda")
    a = K.conv_prefill(x, w, state=cpool, state_indices=slots, cu_seqlens=cu)
    b = K.scan_prefill(x, dt, A_log, B, C, state=spool, state_indices=slots, cu_seqlens=cu)
    assert torch.equal(a, K.conv_prefill(x, w, cu_seqlens=cu))
    assert torch.equal(b, K.scan_prefill(x, dt, A_log, B, C, cu_seqlens=cu))
    assert torch.equal(cpool, cb) and torch.equal(spool, sb)
