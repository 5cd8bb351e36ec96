"""Counts next to 2^31: the kernels reckon with sequence and head numbers in 32 bits, so what would
pass them is refused.  On the host, with addresses that are never read."""
import numpy as np
import pytest
import torch

from kda_chunked_recurrent_b200 import capi

BASE, GB = 0x100000000000, 1 << 30
TOP = 2 ** 31 - 1
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on addresses that are none")


def _conv(num):
    sh = capi.kda_conv_shape_t(num_seqs=num, tokens=64, channels=8, width=4, parts=1, pool_size=0,
                               dtype=0, reserved=0, x_stride=8)
    return capi.kda_conv_prefill(BASE, BASE + GB, None, None, None, None, BASE + 20 * GB, sh,
                                 BASE + 2 * GB, None, 0, None)


def _scan(num):
    sh = capi.kda_scan_shape_t(num_seqs=num, tokens=64, channels=8, state_size=4, groups=1,
                               pool_size=0, dtype=0, max_seqlen=0, x_stride=8, dt_stride=8,
                               z_stride=8, b_stride=4, c_stride=4)
    return capi.kda_scan_prefill(BASE, BASE + GB, BASE + 2 * GB, BASE + 3 * GB, BASE + 4 * GB, None,
                                 None, None, None, None, None, BASE + 20 * GB, sh, BASE + 5 * GB,
                                 None, 0, None)


def _norm(heads, width):
    n = heads * width
    sh = capi.kda_norm_shape_t(tokens=2, heads=heads, width=width, group=0, dtype=0, out_dtype=0,
                               x_stride=n, residual_stride=n, residual_out_stride=n, gate_stride=n,
                               eps=1e-6, reserved=0)
    return capi.kda_rms_norm(BASE, None, None, None, sh, BASE + 20 * GB, None, None, 0, None)


@pytest.mark.parametrize("num", [TOP, TOP - 1, TOP - 31, TOP - 4095])
def test_sequence_counts_that_pass_32_bits_are_refused(num):
    assert _conv(num) == capi.KDA_ERR_BAD_SHAPE and _scan(num) == capi.KDA_ERR_BAD_SHAPE


@pytest.mark.parametrize("heads,width", [(TOP, 1), (TOP - 60, 1), (TOP // 2, 2), (TOP - 4095, 1)])
def test_head_counts_that_pass_32_bits_are_refused(heads, width):
    assert _norm(heads, width) == capi.KDA_ERR_BAD_SHAPE


@no_gpu
def test_the_largest_counts_reach_the_device_check():
    dev = capi.KDA_ERR_UNSUPPORTED_DEVICE
    assert _conv(TOP - 4096) == dev and _scan(TOP - 4096) == dev
    assert _norm(TOP - 4096, 1) == dev and _norm((TOP - 4096) // 64, 64) == dev


def _wraps(v):
    return np.int64(v) != np.int64(np.int32(np.uint32(int(v) & 0xffffffff)))


@pytest.mark.parametrize("num,wraps", [(TOP - 1, True), (TOP - 4096, False)])
def test_why_the_search_of_a_sequence_needs_the_limit(num, wraps):
    """find_seq: lane l of 32 probes lo + (l + 1) ceil((hi - lo) / 32), in 32 bits; hi - lo + 31
    is taken before.  A probe that wraps is negative, passes for one inside the range, and its
    offset would be read from in front of the array."""
    step = (num + 31) // 32
    assert (_wraps(num + 31) or _wraps(32 * step)) == wraps


@pytest.mark.parametrize("heads,wraps", [(TOP - 60, True), (TOP - 4096, False)])
def test_why_the_norm_s_heads_need_the_limit(heads, wraps):
    """A thread's head is the block's first head plus its row in the block, at most 63 on, and only
    then brought back below the number of heads; an element's place in its token is at most the last
    head's first element plus 8 * 511 + 7 before it is looked whether it is there."""
    assert _wraps(heads - 1 + 63) == wraps
    assert _wraps(heads - 1 + 8 * 511 + 7) == wraps
