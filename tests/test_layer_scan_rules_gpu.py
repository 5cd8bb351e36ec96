"""The scan of prompts on both sides of the choices that depend on the state's size: rows shared by
8, 4 or 1 thread blocks, and prompts of few rows (needs a B200)."""
import numpy as np
import pytest

from tests.test_layer_scan_gpu import _check_prefill

pytestmark = pytest.mark.gpu


# tiles of 16 channels up to 64 elements, of 8 above: 9 to 10 tiles and 32 to 33 are the borders
@pytest.mark.parametrize("S,D", [(20, 144), (20, 160), (32, 512), (32, 528), (64, 144), (64, 150),
                                 (64, 512), (64, 520), (100, 72), (100, 80), (128, 256), (128, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_rows_of_wide_states(S, D, dtype):
    _check_prefill([530], D, S, 1, dtype, extra=3, hint=False)


@pytest.mark.parametrize("S,D,G", [(64, 40, 2), (128, 24, 3), (33, 90, 1)])
def test_shared_rows_of_several_sequences(S, D, G):
    _check_prefill([520, 0, 31, 64], D, S, G, "f16", extra=3, hint=False)


@pytest.mark.parametrize("S", [64, 65, 100, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("most", [16, 17, 28, 29])
def test_few_rows_of_wide_states(S, dtype, most):
    r = np.random.RandomState(S + most)
    _check_prefill([int(v) for v in r.randint(0, most + 1, 10)] + [most], 1024, S, 2, dtype)
