"""Plain 64-bit forms of the training operators (numpy), for their tests.

Written from the definitions in include/mep.h: checkpoint rows, layer norm and
its gradients, the gated activation and its gradients, grouped weight
gradients.
"""

import numpy as np

BLOCK = 128
U = 2.0 ** -24  # unit roundoff of fp32


def row_bytes(C):
    return -(-(-(-C // 16) * 16 + -(-C // BLOCK)) // 32) * 32


def quantise(x):
    """(q int64 [N, C], s int64 [N, nb]) of x float64 [N, C]."""
    N, C = x.shape
    nb = -(-C // BLOCK)
    q = np.zeros((N, C), np.int64)
    s = np.zeros((N, nb), np.int64)
    for b in range(nb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        for i in range(N):
            top = np.max(np.abs(v[i]))
            if not np.isfinite(top):
                s[i, b] = 255
                continue
            k = -126
            if top > 0:
                k = max(int(np.frexp(top)[1]) - 1 - 6, -126)
            s[i, b] = k + 127
            q[i, b * BLOCK:b * BLOCK + v.shape[1]] = np.clip(np.rint(np.ldexp(v[i], -k)), -127, 127)
    return q, s


def values(q, s):
    step = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return q * np.repeat(step, BLOCK, axis=1)[:, :q.shape[1]]


def pack(q, s):
    """Checkpoint rows, uint8 [N, row_bytes(C)]. Blocks with s = 255 get q = 0."""
    N, C = q.shape
    rows = np.zeros((N, row_bytes(C)), np.uint8)
    rows[:, :C] = q.astype(np.int8).view(np.uint8)
    at = -(-C // 16) * 16
    rows[:, at:at + s.shape[1]] = s
    return rows


def kept(x):
    """x float64 [N, C] after 8 bits."""
    return values(*quantise(x))


def norm(x, w, b, eps):
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    return c * rstd[:, None] * w + b, mean, rstd


def norm_backward(dy, x, w, mean, rstd):
    xhat = (x - mean[:, None]) * rstd[:, None]
    t = dy * w
    dx = rstd[:, None] * (t - t.mean(1)[:, None] - xhat * (t * xhat).mean(1)[:, None])
    return dx, (dy * xhat).sum(0), dy.sum(0)


def sigmoid(g):
    return 0.5 * (1.0 + np.tanh(0.5 * g)) if np.ndim(g) == 0 else np.where(
        g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_backward(da, g, u):
    s = sigmoid(g)
    return da * u * s * (1.0 + g * (1.0 - s)), da * g * s


def wgrad(x, dy, cu, E):
    """home [E, H, H'] and slot [R, B, H, H'] (float64), and the same of |x|^T |dy|."""
    R, G = cu.shape
    SK = x.shape[0] // R
    H, Hp = x.shape[1], dy.shape[1]
    out = []
    for a, d in ((x, dy), (np.abs(x), np.abs(dy))):
        home = np.zeros((E, H, Hp))
        slot = np.zeros((R, G - E, H, Hp))
        for r in range(R):
            lo = 0
            for j in range(G):
                hi = int(cu[r, j])
                if hi > lo:
                    part = a[r * SK + lo:r * SK + hi].T @ d[r * SK + lo:r * SK + hi]
                    if j < E:
                        home[j] += part
                    else:
                        slot[r, j - E] += part
                lo = hi
        out += [home, slot]
    return out
