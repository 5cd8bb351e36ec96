"""The short convolution against its definition in 64 bits (needs a B200)."""
import numpy as np
import pytest
import torch

from tests.layer_reference import TYPES, close, conv, f64

pytestmark = pytest.mark.gpu


def _rows(rows, C, dtype, g, stride):
    """[rows, C] of N(0, 1) whose rows lie `stride` elements apart, in a longer buffer."""
    buf = torch.randn(rows * stride + 8, generator=g).to(dtype).cuda()
    return buf[3 if stride % 8 else 0:][:rows * stride].view(rows, stride)[:, :C]


def _check_prefill(lens, C, W, dtype, *, parts=1, silu=True, bias=True, state=True, extra=0,
                   lead=0, stride=None, cu64=False, fixed=False, seed=1, indices=True):
    """Sequences of these lengths behind `lead` foreign rows and before `extra` ones."""
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(seed)
    t, N = TYPES[dtype], len(lens)
    cu = lead + np.concatenate([[0], np.cumsum(lens)])
    rows = int(cu[-1]) + extra
    x = _rows(rows, C, t, g, stride or C)
    w = torch.randn(C, W, generator=g).cuda()
    b = torch.randn(C, generator=g).cuda() if bias else None
    P = N + 3
    pool = torch.randn(P, W - 1, C, generator=g).to(t).cuda() if state else None
    slots = torch.randperm(P, generator=g)[:N].int().cuda() if indices else None
    if state and indices and N > 2:
        slots[1] = -1
    has = (torch.arange(N) % 2 == 0).cuda() if state else None
    before = None if pool is None else pool.clone()
    shape = (rows, C) if parts == 1 else (parts, rows, C // parts)
    out = torch.full(shape, 7.0, dtype=t, device="cuda")
    got = K.conv_prefill(x, w, bias=b, state=pool, state_indices=slots if state else None,
                         has_state=has, parts=parts, silu=silu, out=out,
                         cu_seqlens=None if fixed else torch.tensor(
                             cu, dtype=torch.int64 if cu64 else torch.int32).cuda(),
                         num_seqs=N if fixed else None)
    torch.cuda.synchronize()
    assert got is out
    flat = out if parts == 1 else out.movedim(0, 1).reshape(rows, C)
    X = f64(x)
    touched = set()
    for n in range(N):
        slot = -1 if not state else (n if slots is None else int(slots[n]))
        past = np.zeros((W - 1, C))
        if slot >= 0 and bool(has[n]):
            past = f64(before[slot])
        y, bound, new = conv(X[cu[n]:cu[n + 1]], f64(w), f64(b), past, silu)
        close(flat[cu[n]:cu[n + 1]], y, bound, t, f"sequence {n}")
        if slot >= 0:
            assert np.array_equal(f64(pool[slot]), new), f"state of sequence {n}"
            touched.add(slot)
    for s in range(P if state else 0):
        if s not in touched:
            assert torch.equal(pool[s], before[s])
    # rows outside the sequences are left as they were
    assert torch.all(flat[:cu[0]] == 7.0) and torch.all(flat[cu[-1]:] == 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_prompts_every_type_and_width(dtype, W):
    _check_prefill([5, 40, 1, 0, 17, 3, 2, 100], 96, W, dtype)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 3], [2, 1, 1, 2, 0, 1], [15, 16, 17, 31, 32, 33],
                                  [1] * 70, [300, 1, 299]])
def test_prompts_lengths_around_strips(lens):
    _check_prefill(lens, 72, 4, "bf16")


@pytest.mark.parametrize("C,parts,stride", [(1, 1, None), (7, 1, None), (1003, 1, 1005), (96, 3, 100),
                                            (27, 3, 40), (264, 1, 272), (2056, 1, None), (512, 4, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_channels_parts_and_strides(C, parts, stride, dtype):
    _check_prefill([9, 30, 2], C, 4, dtype, parts=parts, stride=stride)


def test_prompts_without_state_bias_activation():
    _check_prefill([33, 2, 20], 64, 4, "bf16", state=False, bias=False, silu=False)
    _check_prefill([20, 20, 20], 64, 3, "bf16", fixed=True, indices=False)


def test_prompts_in_a_padded_batch_and_int64_offsets():
    _check_prefill([21, 0, 30], 64, 4, "bf16", lead=5, extra=40, cu64=True)
    _check_prefill([21, 14], 64, 4, "f16", extra=1)


def test_prompts_many_sequences_and_many_rows():
    r = np.random.RandomState(3)
    _check_prefill([int(v) for v in r.randint(0, 9, 1100)], 40, 4, "bf16")
    # enough rows that a thread block walks two strips
    _check_prefill([3000, 17, 4100], 2048, 4, "bf16", seed=9)


def _check_decode(N, T, C, W, dtype, *, parts=1, silu=True, steps=False, keep=False, P=None,
                  indices=True, stride=None, seed=2):
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(seed)
    t, P = TYPES[dtype], P or N + 2
    x = _rows(N * T, C, t, g, stride or C).unflatten(0, (N, T))
    w, b = torch.randn(C, W, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    pool = torch.randn(P, W - 1, C, generator=g).to(t).cuda()
    before = pool.clone()
    slots = torch.randperm(P, generator=g)[:N].int() if indices else None
    if indices and N > 3:
        slots[1], slots[3] = -1, P
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, st = K.conv_decode(x, w, pool, bias=b, state_indices=None if slots is None else slots.cuda(),
                            parts=parts, silu=silu, return_step_states=steps, keep_state=keep,
                            device_status=status)
    torch.cuda.synchronize()
    assert status.item() == (K.capi.KDA_ERR_BAD_STATE_INDEX if indices and N > 3 else 0)
    flat = out if parts == 1 else out.movedim(0, 2).reshape(N, T, C)
    live = set()
    for n in range(N):
        slot = n if slots is None else int(slots[n])
        if not 0 <= slot < P:
            assert torch.all(flat[n] == 0)
            continue
        live.add(slot)
        past, X = f64(before[slot]), f64(x[n])
        y, bound, new = conv(X, f64(w), f64(b), past, silu)
        close(flat[n], y, bound, t, f"sequence {n}")
        assert np.array_equal(f64(pool[slot]), f64(before[slot]) if keep else new)
        if steps:
            u = np.concatenate([past, X])
            assert np.array_equal(f64(st[n]), np.stack([u[i + 1:i + W] for i in range(T)]))
    for s in range(P):
        if s not in live:
            assert torch.equal(pool[s], before[s])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 4])
def test_tokens_every_type_and_width(dtype, W, T):
    _check_decode(6, T, 96, W, dtype, steps=True)


@pytest.mark.parametrize("N,T,C,parts,stride", [(1, 1, 1, 1, None), (5, 3, 27, 3, 31),
                                                (4, 1, 512, 4, 1024), (3, 9, 1001, 1, None),
                                                (2, 1, 4608, 3, None), (900, 1, 5000, 1, None)])
def test_tokens_shapes(N, T, C, parts, stride):
    _check_decode(N, T, C, 4, "bf16", parts=parts, stride=stride, silu=False)
    if N < 100:
        _check_decode(N, T, C, 4, "f32", parts=parts, stride=stride, keep=True, indices=False, P=N)


def test_prompt_then_tokens_is_one_prompt_bitwise():
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 50, 96, generator=g).bfloat16().cuda()
    w, pool = torch.randn(96, 4, generator=g).cuda(), torch.zeros(1, 3, 96, dtype=torch.bfloat16).cuda()
    whole = K.conv_prefill(x[0], w)
    first = K.conv_prefill(x[0, :41], w, state=pool, has_state=torch.zeros(1, dtype=torch.bool).cuda())
    rest = [K.conv_decode(x[:, 41:45].contiguous(), w, pool)[0][0]]
    rest += [K.conv_decode(x[:, t:t + 1].contiguous(), w, pool)[0][0] for t in range(45, 50)]
    assert torch.equal(whole, torch.cat([first] + rest))


def test_infinities_and_nan_stay_in_their_windows():
    import kda_chunked_recurrent_b200 as K
    x = torch.ones(40, 16, dtype=torch.bfloat16, device="cuda")
    x[20, 3], x[30, 5] = float("nan"), float("inf")
    w = torch.ones(16, 4, device="cuda")
    cu = torch.tensor([0, 21, 40], dtype=torch.int32, device="cuda")
    y = K.conv_prefill(x, w, cu_seqlens=cu, silu=False)
    nan = torch.isnan(y)
    assert nan.sum() == 1 and nan[20, 3]          # the next sequence does not see it
    inf = torch.isinf(y)
    assert inf.sum() == 4 and inf[30:34, 5].all()
