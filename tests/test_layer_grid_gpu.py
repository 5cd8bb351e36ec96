"""Work that no launch can hold is refused as a shape (needs a B200; up to 1 GB)."""
import pytest
import torch

import kda_chunked_recurrent_b200 as K

pytestmark = pytest.mark.gpu


def test_more_thread_blocks_than_a_launch_may_have():
    ch, n = 1 << 24, 140000
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    x, cu = z(0, ch), z(n + 1, t=torch.int32)
    with pytest.raises(K.KDAError, match="kda_conv_prefill: invalid shape"):
        K.conv_prefill(x, z(ch, 2), cu_seqlens=cu)
    with pytest.raises(K.KDAError, match="kda_scan_prefill: invalid shape"):
        K.scan_prefill(x, x, z(ch, 1), z(0, 1, 1), z(0, 1, 1), cu_seqlens=cu)
    torch.cuda.synchronize()
    assert K.rms_norm(z(4, 8))[0].shape == (4, 8)        # and the next call is as any
