"""The scan at the ends of the range: decay rates of zero and without end, steps that
are not finite, steps below zero (needs a B200)."""
import numpy as np
import pytest
import torch

import kda_chunked_recurrent_b200 as K
from tests.layer_reference import close, f64, scan

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

# (lengths, channels): blocks with rows behind the last; rows shared by several thread blocks;
# many prompts of few rows
FORMS = {"blocks": ([45, 3, 32], 24), "shared": ([700], 24), "few rows": ([16, 5, 1] + [9] * 17, 1024)}


def _inputs(rows, D, S, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, z, B, C = r(rows, D).cuda(), r(rows, D).cuda(), r(rows, 1, S).cuda(), r(rows, 1, S).cuda()
    dt = torch.exp(-5 + 2 * torch.rand(rows, D, generator=g)).cuda()     # steps of 0.007 to 0.05
    return x, dt, z, B, C, r(D).cuda(), g


def _prompts(lens, x, dt, A_log, B, C, pool, **kw):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return K.scan_prefill(x, dt, A_log, B, C, state=pool, cu_seqlens=cu, max_seqlen=max(lens),
                          softplus=False, **kw)


# rates of zero (what log(0) gives), far below and above the usual, and beyond FP32
RATES = [-INF, -3.0e38, -1.0e30, -200.0, -90.0, 0.0, 88.0, 88.5, 88.7, 88.75, 89.0, 89.25, 90.5,
         93.0, 97.0, 101.0, 110.0, 300.0]


def _rates(D, S, g):
    A_log = torch.randn(D, S, generator=g)
    for i, v in enumerate(RATES):
        A_log[i % D, (3 * i) % S] = v
        A_log[D - 1 - i % D, 0] = v
    return A_log.cuda()


@pytest.mark.parametrize("S", [13, 16, 128])
@pytest.mark.parametrize("form", list(FORMS))
def test_rates_of_prompts(form, S):
    lens, D = FORMS[form]
    x, dt, z, B, C, skip, g = _inputs(sum(lens), D, S, S)
    A_log = _rates(D, S, g)
    pool = torch.randn(len(lens), D, S, generator=g).cuda()
    before = f64(pool)
    out = _prompts(lens, x, dt, A_log, B, C, pool, D=skip, z=z)
    torch.cuda.synchronize()
    a = 0
    for n, L in enumerate(lens):
        cut = lambda t: f64(t[a:a + L])  # noqa: E731
        y, yb, hs, es = scan(cut(x), cut(dt), f64(A_log), cut(B), cut(C), f64(skip), cut(z), None,
                             before[n], False)
        close(out[a:a + L], y, yb, torch.float32, f"rows of sequence {n}")
        close(pool[n], hs[-1], es[-1], torch.float32, f"state of sequence {n}")
        a += L


@pytest.mark.parametrize("S", [13, 16, 128])
@pytest.mark.parametrize("T", [1, 4])
def test_rates_of_tokens(T, S):
    N, D = 5, 24
    x, dt, z, B, C, skip, g = _inputs(N * T, D, S, S + T)
    A_log = _rates(D, S, g)
    pool = torch.randn(N, D, S, generator=g).cuda()
    before = f64(pool)
    f = lambda t: t.unflatten(0, (N, T))  # noqa: E731
    out = K.scan_decode(f(x), f(dt), A_log, f(B), f(C), pool, D=skip, z=f(z), softplus=False)[0]
    torch.cuda.synchronize()
    for n in range(N):
        cut = lambda t: f64(t[n * T:(n + 1) * T])  # noqa: E731
        y, yb, hs, es = scan(cut(x), cut(dt), f64(A_log), cut(B), cut(C), f64(skip), cut(z), None,
                             before[n], False)
        close(out[n], y, yb, torch.float32, f"rows of sequence {n}")
        close(pool[n], hs[-1], es[-1], torch.float32, f"state of sequence {n}")


@pytest.mark.parametrize("beyond", [3.0e38, INF])
def test_rates_beyond_the_range_forget_all(beyond):
    """As any rate whose decay is 0; a rate that is NaN stays one."""
    lens, D, S = [45, 3], 24, 16
    x, dt, z, B, C, skip, g = _inputs(48, D, S, 1)
    pool = torch.randn(2, D, S, generator=g).cuda()
    A_log = torch.zeros(D, S, device="cuda")
    got, want = [], []
    for into, v in ((got, beyond), (want, 300.0)):
        A_log[3] = v
        state = pool.clone()
        into += [_prompts(lens, x, dt, A_log, B, C, state), state]
        state = pool.clone()
        into += [K.scan_decode(x[:2, None], dt[:2, None], A_log, B[:2, None], C[:2, None], state,
                               softplus=False)[0], state]
    for a, b in zip(got, want):
        assert torch.equal(a, b) and torch.isfinite(a).all()
    A_log[3] = NAN
    state = pool.clone()
    out = _prompts(lens, x, dt, A_log, B, C, state)
    assert torch.isnan(out[:, 3]).all() and torch.isnan(state[:, 3]).all()
    assert torch.isnan(out).sum() == 48 and torch.isnan(state).sum() == 2 * S


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("at", [2, 3])
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_step_that_is_not_finite_leaves_the_rows_before_it(form, dtype, at, value):
    """A NaN or an infinity in dt, at an even and at an odd row: the rows before it, the other
    channels and the other sequences are what they are without it."""
    lens, D = FORMS[form]
    x, dt, z, B, C, skip, g = _inputs(sum(lens), D, 16, 5)
    x, dt, z, B, C = (t.to(dtype) for t in (x, dt, z, B, C))
    A_log = torch.zeros(D, 16, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    runs = []
    for v in (None, value):
        if v is not None:
            dt = dt.clone()
            dt[at, 5] = v
        pool = torch.zeros(len(lens), D, 16, device="cuda")
        runs.append((K.scan_prefill(x, dt, A_log, B, C, D=skip, z=z, state=pool, cu_seqlens=cu,
                                    max_seqlen=max(lens)), pool))
    (y, p), (yn, pn) = runs
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[at:lens[0], 5] = True
    assert torch.equal(y[~hit], yn[~hit]) and not torch.isfinite(yn[hit]).any()
    assert torch.isfinite(y).all() and not torch.isfinite(pn[0, 5]).any()
    pn[0, 5] = p[0, 5]
    assert torch.equal(p, pn)


def test_a_step_that_is_nan_in_tokens():
    x, dt, z, B, C, skip, g = _inputs(6, 24, 16, 6)
    f = lambda t: t.unflatten(0, (2, 3))  # noqa: E731
    dt[1, 5] = NAN
    pool = torch.zeros(2, 24, 16, device="cuda")
    out = K.scan_decode(f(x), f(dt), torch.zeros(24, 16, device="cuda"), f(B), f(C), pool)[0]
    bad = torch.isnan(out)
    assert bad[0, 1:, 5].all() and bad.sum() == 2
    assert torch.isnan(pool[0, 5]).all() and torch.isnan(pool).sum() == 16


# Rows shared by several thread blocks: a run of rows is one factor there.  With negative steps
# (no softplus) that factor may leave FP32's range where the states do not.
@pytest.mark.parametrize("S,dtype", [(16, torch.float32), (13, torch.bfloat16), (64, torch.float32),
                                     (128, torch.float32)])
def test_shared_rows_growth_of_nothing(S, dtype):
    """700 rows of growth in channels without input before them: the states stay zero."""
    rows, D = 1100, 24
    x, dt, z, B, C, skip, g = _inputs(rows, D, S, 7)
    dt[:700] *= -20            # -0.13 to -1 a row; rates of 1 to S
    x[:700] = 0
    x[:, 3] = 0                # and one channel without any
    x, dt, B, C = (t.to(dtype) for t in (x, dt, B, C))
    A_log = torch.log(torch.arange(1, S + 1).float()).repeat(D, 1).cuda()
    pool = torch.zeros(1, D, S, device="cuda")
    out = K.scan_prefill(x, dt, A_log, B, C, D=skip, state=pool, softplus=False)
    y, yb, hs, es = scan(f64(x[700:]), f64(dt[700:]), f64(A_log), f64(B[700:]), f64(C[700:]),
                         f64(skip), None, None, np.zeros((D, S)), False)
    # A single row's factor is an FP32 number: e^89 is above 2^128, infinite, and infinity times a
    # zero state has no value.  So elements whose factors all lie below e^88 have to be right, and
    # the rows of channels without others (with 128 elements a step of 1 takes the last to e^128).
    fits = f64(-dt).max(0)[:, None] * np.exp(f64(A_log)) < 88
    rows_fit = fits.all(1)
    assert fits.sum() >= D * min(S, 80) and (S == 128 or rows_fit.all())
    ok = torch.tensor(rows_fit).cuda()
    assert torch.all(out[:700, ok] == 0) and (not ok[3] or torch.all(out[:, 3] == 0))
    state = f64(pool[0])
    assert np.all(state[3][fits[3]] == 0)
    close(out[700:, ok], y[:, rows_fit], yb[:, rows_fit], dtype, "rows")
    close(state[fits], hs[-1][fits], es[-1][fits], torch.float32, "state")


def test_shared_rows_growth_of_little():
    """A state of 1e-37 grown by e^112 in one run of rows, and decayed by e^-112 behind it."""
    rows, D, S = 1280, 24, 16       # eight runs of 160 rows
    x, dt, z, B, C, skip, g = _inputs(rows, D, S, 8)
    dt[:] = 0.01
    dt[:160], dt[160:320], dt[320:480] = -0.7, 0.7, -0.35
    x[:480] = 0
    pool = 1e-37 * torch.randn(1, D, S, generator=g).cuda()
    before = f64(pool[0])
    A_log = torch.zeros(D, S, device="cuda")
    out = K.scan_prefill(x, dt, A_log, B, C, D=skip, state=pool, softplus=False)
    y, yb, hs, es = scan(f64(x), f64(dt), f64(A_log), f64(B), f64(C), f64(skip), None, None, before,
                         False)
    close(out, y, yb, torch.float32, "rows")
    close(pool[0], hs[-1], es[-1], torch.float32, "state")


def test_shared_rows_bounded_negative_steps():
    """Steps of both signs whose sums stay small: states of usual size throughout."""
    rows, D, S = 1500, 40, 16
    x, dt, z, B, C, skip, g = _inputs(rows, D, S, 9)
    dt = 0.3 * torch.randn(rows, D, generator=g).cuda()
    dt -= torch.cat([torch.zeros(1, D, device="cuda"), dt[:-1]])      # steps whose sums stay small
    pool = torch.randn(1, D, S, generator=g).cuda()
    before = f64(pool[0])
    A_log = torch.zeros(D, S, device="cuda")
    out = K.scan_prefill(x, dt, A_log, B, C, D=skip, z=z, state=pool, softplus=False)
    y, yb, hs, es = scan(f64(x), f64(dt), f64(A_log), f64(B), f64(C), f64(skip), f64(z), None, before,
                         False)
    assert np.abs(hs).max() < 2.0 ** 40          # far from where nothing is asked
    close(out, y, yb, torch.float32, "rows")
    close(pool[0], hs[-1], es[-1], torch.float32, "state")


def test_shared_rows_keep_an_infinite_state():
    """As row by row: decays above zero leave an infinity what it is."""
    rows, D, S = 2048, 24, 16
    x, dt, z, B, C, skip, g = _inputs(rows, D, S, 10)
    dt[:] = 0.5
    pool = torch.randn(1, D, S, generator=g).cuda()
    pool[0, 4, 7] = INF
    K.scan_prefill(x, dt, torch.zeros(D, S, device="cuda"), B, C, state=pool, softplus=False)
    assert pool[0, 4, 7] == INF and torch.isfinite(pool).sum() == D * S - 1


@pytest.mark.parametrize("N,T,D,S,G", [(5, 7, 96, 13, 3), (3, 4, 65, 16, 1), (2, 6, 40, 128, 2)])
def test_tokens_bounded_negative_steps(N, T, D, S, G):
    """Steps of both signs that leave the states at a usual size, so that every value is asked for."""
    g = torch.Generator().manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, z, B, C = r(N, T, D).cuda(), r(N, T, D).cuda(), r(N, T, G, S).cuda(), r(N, T, G, S).cuda()
    dt, A_log, pool = (0.05 * r(N, T, D)).cuda(), torch.log(1 + torch.rand(D, S, generator=g) * 9).cuda(), \
        r(N, D, S).cuda()
    before = f64(pool)
    out, steps = K.scan_decode(x, dt, A_log, B, C, pool, z=z, softplus=False, return_step_states=True)
    for n in range(N):
        y, yb, hs, es = scan(f64(x[n]), f64(dt[n]), f64(A_log), f64(B[n]), f64(C[n]), None, f64(z[n]),
                             None, before[n], False)
        assert np.abs(hs).max() < 2.0 ** 40
        close(out[n], y, yb, torch.float32, f"rows of sequence {n}")
        close(steps[n], hs, es, torch.float32, f"step states of sequence {n}")
        close(pool[n], hs[-1], es[-1], torch.float32, f"state of sequence {n}")
