"""Rows of 65 to 128 elements, the heads of a token, in every type and mode (needs a B200)."""
import pytest

from tests.test_layer_norm_gpu import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("W", [65, 68, 72, 100, 120, 127, 128])
@pytest.mark.parametrize("residual", [False, True])
def test_short_rows(dtype, W, residual):
    for T, H in ((1, 1), (7, 3), (37, 12)):
        _check(T, H, W, dtype, residual=residual)
        _check(T, H, W, dtype, residual=residual, gate="silu", pad=4)
        _check(T, H, W, dtype, residual=residual, gate="sigmoid", bits8=True, group=128)
        _check(T, H, W, dtype, residual=residual, bits8=True)


@pytest.mark.parametrize("W", [72, 128])
def test_short_rows_in_place(W):
    _check(29, 5, W, "f32", in_place="x")
    _check(29, 5, W, "f32", residual=True, in_place="residual")
    _check(29, 5, W, "f32", residual=True, in_place="x for the sum")
