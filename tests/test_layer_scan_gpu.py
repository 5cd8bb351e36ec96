"""The selective scan against its definition in 64 bits (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from tests.layer_reference import TYPES, close, f64, scan

pytestmark = pytest.mark.gpu


def _inputs(rows, D, S, G, dtype, g, *, sliced, gate):
    t = TYPES[dtype]
    pad = 5 if sliced else 0
    r = lambda n: torch.randn(rows, n + pad, generator=g).to(t).cuda()[:, pad:]  # noqa: E731
    bc = r(2 * G * S)
    B, C = bc[:, :G * S].unflatten(1, (G, S)), bc[:, G * S:].unflatten(1, (G, S))
    A_log = (torch.log(torch.arange(1, S + 1).float()) + 0.2 * torch.randn(D, S, generator=g)).cuda()
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(D, generator=g))
    bias = (step + torch.log(-torch.expm1(-step))).cuda()
    return r(D), r(D), A_log, B, C, torch.randn(D, generator=g).cuda(), r(D) if gate else None, bias


def _check_prefill(lens, D, S, G, dtype, *, sliced=False, gate=True, state=True, extra=0, lead=0,
                   softplus=True, skip=True, cu64=False, fixed=False, hint=True, seed=1):
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(seed)
    t, N = TYPES[dtype], len(lens)
    cu = lead + np.concatenate([[0], np.cumsum(lens)])
    rows = int(cu[-1]) + extra
    x, dt, A_log, B, C, Dv, z, bias = _inputs(rows, D, S, G, dtype, g, sliced=sliced, gate=gate)
    if not softplus:
        dt = dt.abs() * 0.05      # steps as they come out of a softplus
        bias = None
    if not skip:
        Dv = None
    P = N + 2
    pool = torch.randn(P, D, S, generator=g).cuda() if state else None
    slots = torch.randperm(P, generator=g)[:N].int().cuda() if state else None
    if state and N > 2:
        slots[1] = -1
    has = (torch.arange(N) % 2 == 0).cuda() if state else None
    before = None if pool is None else pool.clone()
    out = torch.full((rows, D), 7.0, dtype=t, device="cuda")
    K.scan_prefill(x, dt, A_log, B, C, D=Dv, z=z, dt_bias=bias, state=pool, state_indices=slots,
                   has_state=has, softplus=softplus, out=out, max_seqlen=max(lens) if hint else 0,
                   cu_seqlens=None if fixed else torch.tensor(
                       cu, dtype=torch.int64 if cu64 else torch.int32).cuda(),
                   num_seqs=N if fixed else None)
    torch.cuda.synchronize()
    touched = set()
    for n in range(N):
        a, b = cu[n], cu[n + 1]
        slot = int(slots[n]) if state else -1
        h = np.zeros((D, S))
        if slot >= 0 and bool(has[n]):
            h = f64(before[slot])
        cut = lambda v: None if v is None else f64(v[a:b])  # noqa: E731
        y, yb, hs, es = scan(cut(x), cut(dt), f64(A_log), cut(B), cut(C), f64(Dv), cut(z),
                             f64(bias), h, softplus)
        close(out[a:b], y, yb, t, f"rows of sequence {n}")
        if slot >= 0:
            touched.add(slot)
            if b > a:
                close(pool[slot], hs[-1], es[-1], torch.float32, f"state of sequence {n}")
            else:
                assert np.array_equal(f64(pool[slot]), h)
    for s in range(P if state else 0):
        if s not in touched:
            assert torch.equal(pool[s], before[s])
    assert torch.all(out[:cu[0]] == 7.0) and torch.all(out[cu[-1]:] == 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("S", [1, 5, 16, 20, 64, 100, 128])
def test_prompts_every_type_and_state_size(dtype, S):
    _check_prefill([5, 40, 1, 0, 33, 64], 24, S, 2, dtype)


@pytest.mark.parametrize("lens", [[1], [0], [31], [32], [33], [64, 65, 3, 4, 5], [1] * 20, [200]])
def test_prompts_lengths_around_blocks(lens):
    _check_prefill(lens, 40, 16, 1, "bf16")


# channel counts on both sides of every choice of lanes per channel
@pytest.mark.parametrize("D,N", [(1, 1), (7, 1), (600, 2), (1184, 1), (1200, 1), (2400, 1),
                                 (4800, 2), (9472, 1), (9500, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_channel_counts(D, N, dtype):
    _check_prefill([70, 35][:N], D, 16, 1, dtype)


@pytest.mark.parametrize("D,S,G", [(30, 16, 3), (36, 13, 2), (96, 64, 4), (257, 16, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_prompts_slices_groups_odd_sizes(D, S, G, dtype):
    _check_prefill([20, 45], D, S, G, dtype, sliced=True)


def test_prompts_without_gate_skip_state_softplus():
    _check_prefill([40, 3], 32, 16, 1, "bf16", gate=False, skip=False, state=False)
    _check_prefill([40, 3], 32, 16, 1, "f32", softplus=False)
    _check_prefill([50, 50], 32, 16, 1, "bf16", fixed=True, hint=False)


def test_prompts_in_a_padded_batch_and_int64_offsets():
    _check_prefill([21, 0, 40], 32, 16, 1, "bf16", lead=3, extra=50, cu64=True)


def test_prompts_long():
    _check_prefill([3001], 16, 16, 1, "f32", hint=False)
    _check_prefill([2500, 1, 700], 48, 16, 1, "bf16")


def test_prompts_steps_near_zero_and_large():
    """Steps far below and above the usual ones: the series of the softplus and its linear
    end, decays of exactly one and of zero."""
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(8)
    x, dt, A_log, B, C, Dv, z, bias = _inputs(64, 32, 16, 1, "f32", g, sliced=False, gate=True)
    dt = torch.linspace(-110, 110, 64).cuda()[:, None].expand(64, 32).contiguous()
    pool = torch.zeros(1, 32, 16, device="cuda")
    out = K.scan_prefill(x, dt, A_log, B, C, D=Dv, z=z, state=pool)
    y, yb, hs, es = scan(f64(x), f64(dt), f64(A_log), f64(B), f64(C), f64(Dv), f64(z), None,
                         np.zeros((32, 16)), True)
    close(out, y, yb, torch.float32, "rows")
    close(pool[0], hs[-1], es[-1], torch.float32, "state")


def _check_decode(N, T, D, S, G, dtype, *, sliced=False, gate=True, steps=False, keep=False,
                  indices=True, softplus=True, step_bias=True, seed=2):
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(seed)
    t, P = TYPES[dtype], N + 2
    x, dt, A_log, B, C, Dv, z, bias = _inputs(N * T, D, S, G, dtype, g, sliced=sliced, gate=gate)
    if not softplus:
        dt = dt.abs() * 0.05
    if not step_bias:
        bias = None
    f = lambda v: None if v is None else v.unflatten(0, (N, T))  # noqa: E731
    pool = torch.randn(P, D, S, generator=g).cuda()
    before = pool.clone()
    slots = torch.randperm(P, generator=g)[:N].int() if indices else None
    if indices and N > 3:
        slots[1], slots[3] = -1, P
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, st = K.scan_decode(f(x), f(dt), A_log, f(B), f(C), pool, D=Dv, z=f(z), dt_bias=bias,
                            state_indices=None if slots is None else slots.cuda(),
                            softplus=softplus, return_step_states=steps, keep_state=keep,
                            device_status=status)
    torch.cuda.synchronize()
    assert status.item() == (K.capi.KDA_ERR_BAD_STATE_INDEX if indices and N > 3 else 0)
    live = set()
    for n in range(N):
        slot = n if slots is None else int(slots[n])
        if not 0 <= slot < P:
            assert torch.all(out[n] == 0)
            continue
        live.add(slot)
        cut = lambda v: None if v is None else f64(v[n * T:(n + 1) * T])  # noqa: E731
        y, yb, hs, es = scan(cut(x), cut(dt), f64(A_log), cut(B), cut(C), f64(Dv), cut(z),
                             f64(bias), f64(before[slot]), softplus)
        close(out[n], y, yb, t, f"rows of sequence {n}")
        if keep:
            assert torch.equal(pool[slot], before[slot])
        else:
            close(pool[slot], hs[-1], es[-1], torch.float32, f"state of sequence {n}")
        if steps:
            close(st[n], hs, es, torch.float32, f"step states of sequence {n}")
    for s in range(P):
        if s not in live:
            assert torch.equal(pool[s], before[s])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("S", [1, 5, 16, 20, 64, 100, 128])
@pytest.mark.parametrize("T", [1, 4])
def test_tokens_every_type_and_state_size(dtype, S, T):
    _check_decode(6, T, 40, S, 2, dtype, steps=True)


@pytest.mark.parametrize("N,T,D,S,G", [(1, 1, 1, 16, 1), (3, 2, 65, 16, 1), (5, 7, 96, 13, 3),
                                       (2, 1, 1000, 16, 1), (300, 1, 1100, 16, 1)])
def test_tokens_shapes(N, T, D, S, G):
    _check_decode(N, T, D, S, G, "bf16", sliced=True, gate=N != 2)
    if N < 100:
        # negative steps: states that grow; and the steps of a softplus taken before the call
        _check_decode(N, T, D, S, G, "f32", keep=True, indices=False, softplus=False)
        _check_decode(N, T, D, S, G, "f32", indices=False, softplus=False, step_bias=False)


def test_prompt_then_tokens_is_one_prompt():
    """The state handed from the prompt kernel to the token kernel: the rows behind it are
    those of one long prompt (the bound of the definition holds for both)."""
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(6)
    x, dt, A_log, B, C, Dv, z, bias = _inputs(50, 64, 16, 1, "bf16", g, sliced=False, gate=True)
    pool = torch.zeros(1, 64, 16, device="cuda")
    kw = dict(D=Dv, dt_bias=bias)
    cold = torch.zeros(1, dtype=torch.bool, device="cuda")
    outs = [K.scan_prefill(x[:41], dt[:41], A_log, B[:41], C[:41], z=z[:41], state=pool,
                           has_state=cold, **kw)]
    for a, b in [(41, 45)] + [(t, t + 1) for t in range(45, 50)]:
        u = lambda v: v[None, a:b]  # noqa: E731
        outs.append(K.scan_decode(u(x), u(dt), A_log, u(B), u(C), pool, z=u(z), **kw)[0][0])
    y, yb, hs, es = scan(f64(x), f64(dt), f64(A_log), f64(B), f64(C), f64(Dv), f64(z), f64(bias),
                         np.zeros((64, 16)), True)
    close(torch.cat(outs), y, yb, torch.bfloat16, "rows")
    close(pool[0], hs[-1], es[-1], torch.float32, "state")


def test_nan_stays_in_its_sequence_and_channel():
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(7)
    x, dt, A_log, B, C, Dv, z, bias = _inputs(90, 40, 13, 1, "bf16", g, sliced=False, gate=True)
    x[10, 3] = float("nan")
    x[60, 5] = float("inf")
    cu = torch.tensor([0, 45, 90], dtype=torch.int32, device="cuda")
    y = K.scan_prefill(x, dt, A_log, B, C, D=Dv, z=z, dt_bias=bias, cu_seqlens=cu)
    bad = ~torch.isfinite(y)
    assert bad[10:45, 3].all() and bad[60:90, 5].all()
    assert bad.sum() == 35 + 30


# few channels and many rows: the rows of a sequence are shared by several thread blocks
@pytest.mark.parametrize("dtype,D,S,G", [("bf16", 40, 16, 1), ("f32", 250, 13, 2), ("f16", 64, 64, 2),
                                         ("f32", 24, 128, 1), ("bf16", 31, 20, 1)])
@pytest.mark.parametrize("lens", [[512], [513, 0, 31], [1500, 7], [5, 33, 600, 256]])
def test_prompts_few_channels_many_rows(dtype, D, S, G, lens):
    _check_prefill(lens, D, S, G, dtype, extra=5, hint=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,D", [([600], 700), ([1030, 3], 560), ([700], 1184)])
def test_prompts_some_channels_many_rows(dtype, lens, D):
    _check_prefill(lens, D, 16, 1, dtype, hint=False)


def test_prompts_few_channels_small_steps():
    """Steps near 1e-4: what comes before a run of rows still matters at its end."""
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(9)
    x, dt, A_log, B, C, Dv, z, _ = _inputs(2000, 32, 16, 1, "f32", g, sliced=False, gate=True)
    dt = dt.abs() * 1e-4
    pool = torch.randn(1, 32, 16, generator=g).cuda()
    h0 = f64(pool[0])
    out = K.scan_prefill(x, dt, A_log, B, C, D=Dv, z=z, state=pool, softplus=False)
    y, yb, hs, es = scan(f64(x), f64(dt), f64(A_log), f64(B), f64(C), f64(Dv), f64(z), None, h0, False)
    close(out, y, yb, torch.float32, "rows")
    close(pool[0], hs[-1], es[-1], torch.float32, "state")


# many sequences of few rows each
@pytest.mark.parametrize("dtype,D,S,G,N", [("bf16", 1024, 16, 1, 20), ("f32", 1030, 13, 2, 20),
                                           ("f16", 1024, 128, 4, 12), ("bf16", 2051, 20, 1, 7)])
def test_prompts_many_of_few_rows(dtype, D, S, G, N):
    r = np.random.RandomState(4)
    lens = [int(v) for v in r.randint(0, 6, N - 1)] + [16]
    _check_prefill(lens, D, S, G, dtype, sliced=dtype == "f32")
    _check_prefill([1] * N, D, S, G, dtype, state=False, gate=False)
    _check_prefill([3] * N, D, S, G, dtype, fixed=True, hint=False)
