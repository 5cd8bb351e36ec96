"""The root-mean-square norm against its definition in 64 bits (needs a B200)."""
import numpy as np
import pytest
import torch

from tests.layer_reference import TYPES, close, f64, half_step, norm

pytestmark = pytest.mark.gpu

# relative error of y before its rounding: the sum of squares (no cancellation; a chain of at
# most 64 FP32 additions and the tree above it), its root and the products: 128 steps of 2^-24
REL = 128 * 2.0 ** -24


def _check(T, H, W, dtype, *, residual=False, gate=None, bits8=False, group=0, weight=True, pad=0,
           in_place="", eps=1e-6, seed=1, edit=None):
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    make = lambda: torch.randn(T, H * W + pad, generator=g).to(t).cuda()[:, pad:].unflatten(  # noqa: E731
        1, (H, W))
    x, res, z = make(), make() if residual else None, make() if gate else None
    if edit:
        edit(x)
    w = (1 + 0.3 * torch.randn(W, generator=g)).cuda() if weight else None
    X, R, Z = f64(x), f64(res), f64(z)
    kw = {}
    if in_place == "x":
        kw = dict(out=x)
    elif in_place == "residual":
        kw = dict(residual_out=res)
    elif in_place == "x for the sum":
        kw = dict(residual_out=x)
    out, ro, sc = K.rms_norm(x, w, eps=eps, residual=res, gate=z, gate_activation=gate or "silu",
                             out_dtype=torch.float8_e4m3fn if bits8 else None, group=group, **kw)
    torch.cuda.synchronize()
    r, y = norm(X, f64(w), R, Z, eps, gate == "sigmoid")
    if residual:
        close(ro, r, 2.0 ** -24 * np.abs(r), t, "sum")
    else:
        assert ro is None
    # an exponential's argument is rounded: the gate's factor is off by up to |z| more steps
    rel = REL * (1 + (np.abs(Z) / 64 if gate else 0))
    if not bits8:
        assert sc is None and out.dtype == t
        close(out, y, rel * np.abs(y), t, "out")
        return
    n = group or W
    assert sc.shape == (T, H, -(-W // n)) and out.dtype == torch.float8_e4m3fn
    S = f64(sc)
    for i in range(S.shape[-1]):
        part = np.abs(y[..., i * n:(i + 1) * n])
        want = np.maximum(part.max(-1), 2.0 ** -40) / 448
        worst = REL * (1 + (np.abs(Z).max() / 64 if gate else 0))
        assert np.all(np.abs(S[..., i] - want) <= want * worst)
    of = np.repeat(S, n, -1)[..., :W]
    got = f64(out.float()) * of
    # one E4M3 rounding of a value that carries the error above (a value next to a tie may
    # go to either side, each within half a step)
    tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * of) * (1 + 2.0 ** -10) + 2 * worst * np.abs(y)
    assert np.all(np.abs(got - y) <= tol)
    assert f64(out.float()).max() <= 448


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("W", [1, 7, 8, 64, 100, 128, 200, 256, 500, 512, 1000, 1024, 2000, 4096,
                               5000, 8192, 16384, 20000, 32768])
def test_every_width_and_type(dtype, W):
    _check(5, 1, W, dtype, residual=True)
    _check(3, 1, W, dtype, gate="silu", bits8=True, group=128)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("gate", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("bits8,group", [(False, 0), (True, 0), (True, 128)])
def test_every_combination(dtype, residual, gate, bits8, group):
    _check(9, 3, 128, dtype, residual=residual, gate=gate, bits8=bits8, group=group)
    _check(4, 1, 1100, dtype, residual=residual, gate=gate, bits8=bits8, group=group, pad=3)


@pytest.mark.parametrize("T,H,W", [(1, 1, 128), (1, 12, 128), (1, 5, 40), (17, 1, 250), (2000, 12, 128),
                                   (3, 2, 3000), (700, 1, 2560)])
def test_row_counts(T, H, W):
    _check(T, H, W, "bf16", residual=True, gate="sigmoid", bits8=True, pad=8)
    _check(T, H, W, "bf16", weight=False)


@pytest.mark.parametrize("in_place", ["x", "residual", "x for the sum"])
@pytest.mark.parametrize("W", [128, 1000, 4096])
def test_in_place(in_place, W):
    _check(30, 1, W, "bf16", residual=in_place != "x", in_place=in_place)


def test_rows_of_zeros_and_tiny_values():
    """A zero row gives zeros; without eps it is 0 / 0, as the formula has it.  A row of tiny
    values is below the smallest scale: its codes are the values over that scale."""
    import kda_chunked_recurrent_b200 as K
    x = torch.zeros(3, 256, device="cuda")
    x[1] = 1e-30
    out, _, sc = K.rms_norm(x, out_dtype=torch.float8_e4m3fn, group=128)
    assert torch.all(out.float() == 0)
    assert torch.all(sc == torch.tensor(2.0 ** -40 / 448).cuda())
    assert torch.all(K.rms_norm(x)[0][0] == 0)
    assert torch.all(torch.isnan(K.rms_norm(x, eps=0.0)[0][0]))


def test_nan_and_infinity_stay_in_their_rows():
    import kda_chunked_recurrent_b200 as K
    x = torch.ones(4, 256, device="cuda")
    x[1, 7], x[2, 200] = float("nan"), float("inf")
    y = K.rms_norm(x)[0]
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 200]) and torch.all(y[2, :200] == 0)
    q, _, sc = K.rms_norm(x, out_dtype=torch.float8_e4m3fn, group=128)
    assert torch.isnan(sc[1]).all() and torch.isnan(q[1].float()).all()
    assert torch.isfinite(sc[0]).all() and torch.isfinite(q[3].float()).all()
    # a gate's NaN marks the scale of its group and no other
    gate = torch.ones(4, 256, device="cuda")
    gate[0, 3] = float("nan")
    q, _, sc = K.rms_norm(torch.ones_like(x), gate=gate, out_dtype=torch.float8_e4m3fn, group=128)
    assert torch.isnan(sc[0, 0]) and torch.isfinite(sc[0, 1]) and torch.isfinite(sc[1:]).all()


def test_large_values_keep_their_norm():
    """Squares of large FP16 and BF16 values are summed in FP32."""
    _check(3, 1, 4096, "f16", edit=lambda x: x.mul_(10000))
    _check(3, 1, 4096, "bf16", edit=lambda x: x.mul_(1e15))
