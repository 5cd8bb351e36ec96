"""The norm's 8-bit codes and scales where the norm itself is exact (needs a B200).

Rows of ones without eps have a root mean square of one, so y is the weight to the last bit:
scale = max |w| / 448 and code = e4m3(w / scale) can be asked for exactly, from quotients that are
rounded once (half a step of FP32, 2^-24)."""
import numpy as np
import pytest
import torch

import kda_chunked_recurrent_b200 as K

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


def _near_borders(W, group, seed):
    """Weights whose quotients lie at the borders between E4M3 numbers, and one step to a side."""
    r = np.random.RandomState(seed)
    codes = torch.arange(0, 127, dtype=torch.uint8).view(E4).double().numpy()
    borders = (codes[1:] + codes[:-1]) / 2
    w = np.empty(W, np.float32)
    for lo in range(0, W, group):
        n = min(group, W - lo)
        amax = np.float32(np.exp(r.uniform(-3, 3)))
        scale = np.float32(np.float64(amax) / 448)
        v = (r.choice(borders, n) * np.float64(scale)).astype(np.float32)
        v = np.nextafter(v, np.float32(1e9) * r.choice([-1, 1], n).astype(np.float32),
                         dtype=np.float32) * r.choice([-1, 1], n).astype(np.float32)
        v = np.where(r.rand(n) < 0.5, v, (r.choice(borders, n) * np.float64(scale)).astype(np.float32))
        v[r.randint(n)] = amax
        w[lo:lo + n] = np.clip(v, -amax, amax)
    return torch.tensor(w)


def _codes(q):
    return torch.tensor(q, dtype=torch.float32).clamp(-448, 448).to(E4).float().numpy()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("W", [60, 100, 128, 131, 250, 512, 1024, 2000, 4096, 9000, 20000])
def test_codes_are_the_rounded_quotients(W, group):
    for seed in range(3):
        w = _near_borders(W, group or W, seed)
        x = torch.ones(3, W, device="cuda")
        out, _, scales = K.rms_norm(x, w.cuda(), eps=0.0, out_dtype=E4, group=group)
        got, sc = out.float().cpu().numpy(), scales.cpu().numpy()
        w64 = w.double().numpy()
        for lo in range(0, W, group or W):
            part = w64[lo:lo + (group or W)]
            want = np.float32(np.abs(part).max() / 448)
            assert np.all(sc[:, lo // (group or W)] == want)
            q = part / np.float64(want)
            # a quotient rounded once to FP32 lies within 2^-24 of it (a hundredth for the
            # correction's own roundings)
            one, other = (_codes(q * (1 + s * 1.01 * 2.0 ** -24)) for s in (-1, 1))
            codes = got[:, lo:lo + (group or W)]
            assert np.all((codes == one) | (codes == other))


def test_an_infinite_scale():
    """Numbers over an infinite scale are zero, the infinity itself is a NaN; the other groups and
    rows are what they are without it."""
    x = torch.ones(3, 256, device="cuda")
    gate = torch.ones(3, 256, device="cuda")
    plain, _, sp = K.rms_norm(x, gate=gate, out_dtype=E4, group=128)
    gate[1, 5] = float("inf")
    out, _, sc = K.rms_norm(x, gate=gate, out_dtype=E4, group=128)
    assert torch.isinf(sc[1, 0]) and torch.isnan(out.float()[1, 5])
    rest = torch.ones(3, 256, dtype=torch.bool, device="cuda")
    rest[1, :128] = False
    assert torch.equal(out.float()[rest], plain.float()[rest]) and torch.equal(sc[[0, 2]], sp[[0, 2]])
    zero = out.float()[1, :128]
    assert torch.all(zero[:5] == 0) and torch.all(zero[6:] == 0)


def test_large_and_small_scales():
    """Maxima of 2^127 and below the smallest scale."""
    for amax in (1.5 * 2.0 ** 127, 1.7 * 2.0 ** 126, 2.0 ** -39, 2.0 ** -45, 1e-30):
        w = torch.linspace(-1, 1, 256).double() * amax
        w = w.float()
        out, _, sc = K.rms_norm(torch.ones(1, 256, device="cuda"), w.cuda(), eps=0.0, out_dtype=E4)
        want = np.float32(max(float(w.abs().max()), 2.0 ** -40) / 448)
        assert sc.item() == want
        q = w.double().numpy() / np.float64(want)
        one, other = (_codes(q * (1 + s * 1.01 * 2.0 ** -24)) for s in (-1, 1))
        got = out.float().cpu().numpy()[0]
        assert np.all((got == one) | (got == other))
