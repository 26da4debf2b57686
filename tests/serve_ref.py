"""Plain 64-bit forms of the serving operators and the router, for their tests.

Written from the definitions in include/mep.h: matrices in 4 bits, their
product with a few rows, the layer for a few tokens, the router's choice and
its gradient. numpy for the formats and the router, torch in 64 bits for sums.

Bounds. Tensor-core sums are taken to add with relative error 2^-23 each (they
do not round to nearest), so that n products are off by n * 2^-23 * sum |x w|;
an output in bf16 is off by 2^-8, in fp32 by 2^-24 of its value once more.
"""

import numpy as np
import torch

TC = 2.0 ** -23


def bf16(x):
    """The nearest bf16 (ties to even) of float64 values, as float64; by way of fp32, which the tests' values are."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


# ------------------------------------------------------------------------------------------ matrices in 4 bits


def w4_quantise(w, group):
    """(q int [K, N], s float64 [ceil(K / group), N]) of w float64 [K, N]."""
    K, N = w.shape
    n = -(-K // group)
    q, s = np.zeros((K, N), np.int64), np.zeros((n, N))
    for i in range(n):
        v = w[i * group:(i + 1) * group]
        top = np.abs(v).max(0)
        fine = np.isfinite(top)
        s[i] = np.where(fine, bf16(np.where(fine, top, 0).astype(np.float32) * (np.float32(1) / np.float32(7))), np.nan)
        ok = s[i] > 0
        d = np.where(ok, s[i], 1)
        r = np.rint(np.where(ok, np.where(np.isfinite(v), v, 0) / d, 0))
        q[i * group:(i + 1) * group] = np.clip(r, -7, 7)
    return q, s


def w4_values(q, s, group):
    return q * np.repeat(s, group, 0)[:q.shape[0]]


def w4_bytes(K, N, group):
    return -(-N // 64) * -(-K // 128) * (4096 + 128 // group * 128)


def w4_pack(q, s, group):
    """The bytes of one matrix, element by element."""
    K, N = q.shape
    kb, block = -(-K // 128), 4096 + 128 // group * 128
    out = np.zeros((-(-N // 64), kb, block), np.uint8)
    out[:, :, :4096] = 0x88
    bits = torch.from_numpy(s.astype(np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    for n in range(N):
        c, l, g = n % 64 // 16, n // 8 % 2, n % 8
        for k in range(K):
            r = k % 128
            h, j, i, t, e = r // 64, r // 16 % 4, r // 8 % 2, r // 2 % 4, r % 2
            at = ((((4 * h + c) * 8 + g) * 4 + t) * 4 + j) * 4 + 2 * e + i
            b = out[n // 64, k // 128]
            b[at] = (b[at] & (0xF0 if l == 0 else 0x0F)) | ((q[k, n] + 8) << (4 * l))
        for gi in range(s.shape[0]):
            row = gi * group
            at = 4096 + 2 * (row % 128 // group * 64 + 16 * c + 2 * g + l)
            out[n // 64, row // 128, at:at + 2] = np.array([bits[gi, n]], np.uint16).view(np.uint8)
    return out.reshape(-1)


# ------------------------------------------------------------------------------------------ products


def product(x, w):
    """(x @ w, |x| @ |w|) in 64 bits."""
    x, w = x.double(), w.double()
    return x @ w, x.abs() @ w.abs()


def product_bound(exact, absolute, K, half):
    """Of a sum of K products and its groups' (32 rows at least) scaled sums, rounded by `half` of its value."""
    n = K + 2 * (K // 32 + 2)
    return half * exact.abs() + (1 + half) * n * TC * absolute


def layer(x, idx, w, w1, w2):
    """(out, bound) of the layer in 64 bits. x [T, H], idx [T, K] (-1: none), w [T, K], w1(e) -> [H, 2F], w2(e) -> [F, H]."""
    T, H = x.shape
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    for e in sorted(set(idx.flatten().tolist()) - {-1}):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        a1, a2 = w1(e).double(), w2(e).double()
        F = a2.shape[0]
        gu, mag = product(x[t], a1)
        off = (H + 2 * (H // 32 + 2)) * TC * mag
        g, u, dg, du = gu[:, :F], gu[:, F:], off[:, :F], off[:, F:]
        silu = g * torch.sigmoid(g)
        a = silu * u
        # |silu'| <= 1.1; 2^-20 for fp32 exp, division and products; half a step of bf16
        da = 1.1 * dg * (u.abs() + du) + silu.abs() * du
        da = da + (a.abs() + da) * (2.0 ** -8 + 2.0 ** -20)
        y, _ = product(a, a2)
        wt = w[t, k].double()[:, None]
        out.index_add_(0, t, wt * y)
        dy = da @ a2.abs() + (F + 2 * (F // 32 + 2)) * TC * ((a.abs() + da) @ a2.abs())
        bound.index_add_(0, t, wt.abs() * (dy + (idx.shape[1] + 1) * 2.0 ** -23 * (y.abs() + dy)))
    return out, bound + 2.0 ** -8 * (out.abs() + bound)


# ------------------------------------------------------------------------------------------ the router


def route(logits, bias, K, skip):
    """(idx, w) of float32 logits [N, E]: by a stable sort on (NaN first, then descending), softmax in 64 bits."""
    key = logits + (np.float32(0) if bias is None else bias.astype(np.float32))
    N, E = logits.shape
    idx = np.empty((N, K), np.int64)
    w = np.empty((N, K))
    for t in range(N):
        order = sorted(range(E), key=lambda e: (0, 0.0, e) if np.isnan(key[t, e]) else (1, -float(key[t, e]), e))
        idx[t] = order[:K]
        top = logits[t, idx[t]].astype(np.float64)
        if np.isnan(top).any() or (top == np.inf).any():
            w[t] = np.nan
            if not np.isnan(top).any():  # infinity: exp(-inf) stays 0 over a NaN sum
                w[t] = np.nan
        elif (top == -np.inf).all():
            w[t] = 0
        else:
            ex = np.where(top == -np.inf, 0, np.exp(top - top.max()))
            w[t] = ex / ex.sum()
        if skip:
            idx[t] = np.where(top == -np.inf, -1, idx[t])
    return idx, w


def route_backward(dw, w, idx, E):
    """(dlogits, bound factor) in 64 bits; an expert that stands twice gets both."""
    N, K = dw.shape
    d = np.zeros((N, E))
    mag = np.zeros((N, E))
    s = (w * dw).sum(1, keepdims=True)
    sm = np.abs(w * dw).sum(1, keepdims=True)
    for t in range(N):
        for k in range(K):
            if idx[t, k] >= 0:
                d[t, idx[t, k]] += w[t, k] * (dw[t, k] - s[t, 0])
                mag[t, idx[t, k]] += abs(w[t, k]) * (abs(dw[t, k]) + sm[t, 0])
    return d, mag
