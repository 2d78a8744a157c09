"""Plain 64-bit forms of the 8-bit operators, for the tests (numpy, no library code)."""
import numpy as np

NAN = float("nan")


def quantize(x):
    """x fp64 values of bf16/fp16/fp32 numbers, [rows, cols] -> (codes int8, scales fp32)."""
    x = np.asarray(x, np.float64)
    a = np.abs(x).max(1)
    with np.errstate(all="ignore"):
        s = (a.astype(np.float32) / np.float32(127)).astype(np.float32)      # correctly rounded
        q = np.rint(x / s.astype(np.float64)[:, None])                       # ties to even
    q = np.clip(np.where(s[:, None] > 0, q, 0), -127, 127)
    bad = ~np.isfinite(a)
    s[bad] = NAN
    q[bad] = 0
    return q.astype(np.int8), s


def values(codes, scales):
    return codes.astype(np.float64) * scales.astype(np.float64)[:, None]


def matmul32(cx, sx, cw, sw, bias=None):
    """int8_matmul before its last rounding: the exact integer sum and the stated fp32 steps."""
    acc = cx.astype(np.int64) @ cw.astype(np.int64).T
    v = (acc.astype(np.float32) * sx[:, None]).astype(np.float64) * sw.astype(np.float64)[None]
    if bias is not None:
        v = v + bias.astype(np.float64)[None]     # fp64: far more than the fma's 24 bits
    return v.astype(np.float32)


def layer(u, Wt, A, B, alpha, g):
    """y of the layer for inputs x (fp64); the adapter reads pool(x)."""
    x = np.asarray(u, np.float64)
    p = x.reshape(x.shape[0], -1, g).mean(2)
    return x @ Wt.T + alpha / A.shape[1] * (p @ A) @ B


def layer_backward(x, dy, Wt, A, B, alpha, g, T=None):
    p = x.reshape(x.shape[0], -1, g).mean(2)
    s = alpha / A.shape[1]
    G = dy @ B.T
    T = p @ A if T is None else T
    dx = dy @ Wt + s / g * np.repeat(G @ A.T, g, axis=1)
    return dx, s * p.T @ G, s * T.T @ dy
