"""The layer operators in 64 bits, element by element from their definitions, each with a
bound of what FP32 arithmetic and one rounding may add.

Unit: u = 2^-24, half a step of FP32.  The kernels' special functions (ex2, lg2, rcp
approximations) are off by at most 2^-22 relative, and an exponential's argument is rounded
before it is taken, which adds |argument| u log2(e) relative.  One FP32 operation with such
operands stays within kOp = 2^-20 of its absolute terms, which is the unit of the bounds.
"""
import numpy as np
import torch

kOp = 2.0 ** -20
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def half_step(dtype, y):
    """Half a rounding step of ``dtype`` at y: eps / 2 relative; below the smallest normal
    number half of the subnormals' distance."""
    fi = torch.finfo(dtype)
    return np.maximum(np.abs(y) * fi.eps / 2, fi.smallest_normal * fi.eps / 2)


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def conv(x, w, bias, past, silu):
    """One sequence: x [L, C], past [W - 1, C] -> y, bound (before rounding), new state."""
    W, L = w.shape[1], x.shape[0]
    u = np.concatenate([past, x], 0)
    acc = np.zeros_like(x)
    mag = np.zeros_like(x)
    for j in range(W):
        acc += u[j:j + L] * w[:, j]
        mag += np.abs(u[j:j + L] * w[:, j])
    if bias is not None:
        acc += bias
        mag += np.abs(bias)
    # |silu'| <= 1.1, and the sigmoid's own error is one kOp of |acc| <= mag
    return (acc * sigmoid(acc) if silu else acc), (2.2 if silu else 1.0) * kOp * mag, u[L:]


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def scan(x, dt, A_log, B, C, D, z, dt_bias, h, plus):
    """One sequence: x, dt, z [L, D]; B, C [L, G, N]; h [D, N] -> y, bound, the states
    after every row [L, D, N] and their bound.

    H carries the sums of absolute terms and E the error: a row multiplies the error by the
    decay and adds one unit of everything it touches (the decay's error grows with its
    argument)."""
    L, Dn = x.shape
    G = B.shape[1]
    of = np.arange(Dn) // (Dn // G)
    A = -np.exp(A_log)
    h = h.copy()
    H, E = np.abs(h), np.zeros_like(h)
    y, yb = np.zeros((L, Dn)), np.zeros((L, Dn))
    hs, es = np.zeros((L,) + h.shape), np.zeros((L,) + h.shape)
    for t in range(L):
        v = dt[t] + (0 if dt_bias is None else dt_bias)
        # the sum's rounding is relative to its terms; softplus has slope <= 1
        dv = kOp * (np.abs(dt[t]) + (0 if dt_bias is None else np.abs(dt_bias)))
        d = softplus(v) if plus else v
        rel = (kOp * np.abs(d) + dv * (sigmoid(v) if plus else 1.0)) / np.maximum(np.abs(d), 1e-300)
        a = np.exp(d[:, None] * A)
        b = (d * x[t])[:, None] * B[t][of]
        arg = np.abs(d[:, None] * A)
        E = a * E + a * H * (kOp * (1 + arg) + arg * rel[:, None]) + np.abs(b) * (kOp + rel[:, None])
        h = a * h + b
        H = a * H + np.abs(b)
        E += kOp * H
        hs[t], es[t] = h, E
        y[t] = (h * C[t][of]).sum(-1)
        yb[t] = (E * np.abs(C[t][of])).sum(-1) + kOp * (H * np.abs(C[t][of])).sum(-1)
        if D is not None:
            y[t] += D * x[t]
            yb[t] += kOp * np.abs(D * x[t])
    if z is not None:
        g = z * sigmoid(z)
        yb = yb * np.abs(g) + 2 * kOp * np.abs(y * z)
        y = y * g
    return y, yb, hs, es


def norm(x, w, residual, gate, eps, sigmoid_gate):
    """Rows [..., W] -> r, y and the relative bound of y (sums of squares have no
    cancellation: their relative error is at most log2 of the row's length steps)."""
    r = x if residual is None else x + residual
    y = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * w
    if gate is not None:
        y = y * sigmoid(gate) * (1.0 if sigmoid_gate else gate)
    return r, y


def close(got, want, bound, dtype, what):
    """Within the bound and one rounding.  bound / kOp is at least the sum of the absolute
    terms behind a value: above 2^100 of them FP32, which ends at 2^128, may have left its
    range on the way (negative steps let a state grow without end), and nothing is asked."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    tol = bound + half_step(dtype, np.abs(want) + bound)
    bad = ~(np.abs(got - want) <= tol) & ~(bound / kOp > 2.0 ** 100)
    assert not bad.any(), (
        f"{what}: {bad.sum()} of {bad.size} values off, the worst by "
        f"{np.nanmax(np.where(bad, np.abs(got - want) / tol, 0)):.3g} times its tolerance, first at "
        f"{np.argwhere(bad)[0]}, nan {np.isnan(got).sum()}")
