"""mep_layer_norm, mep_ckpt_save / load and mep_swiglu, with their backward passes, against plain 64-bit forms.

Checkpoint rows hold nothing but exact power-of-two scaling and one rounding:
they are compared byte for byte. The bounds of the others, with u = 2^-24:

* Sums over a row. No chain of additions is longer than L = 128 (a thread
  adds at most 64 terms in turn, a warp's lanes are joined in 5 steps, at most
  32 warps in turn), so a sum is off by at most L u times the sum of
  magnitudes; a factor inside a term adds its own roundings.
* rstd: a relative error e in the variance is e / 2 in rstd; the variance is
  off by (L + 4) u relatively and by the square of the mean's error, plus 3 u
  for the addition of eps, the root and the division.
* xhat = (x - mean) * rstd in two or three roundings, each of a value of at
  most (|x| + |mean|) rstd: 3 u (|x| + |mean|) rstd, called ex.
* Sums over rows (dweight, dbias) are bounded for any order: (N + 3) u times
  the sum of magnitudes.
* sigmoid: __expf is off by 2 + 1.173 |g| ulp (CUDA's documented bound), one
  ulp at most 2 u relatively; 1 / (1 + e) adds at most 6 u. sigmoid's relative
  error is at most es = u (4 + 2.4 |g| + 6). Below g = -87 the reciprocal may
  be flushed to zero: 2^-125 absolutely.
* One rounding of the result: 2^-8 relatively for bf16 (8 significant bits;
  2^-134 for the smallest), u for fp32.
"""

import ctypes

import numpy as np
import pytest
import torch

import load_balancing_topk_gb300 as mep
import train_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = ref.U
L = 128
BF16, F32 = torch.bfloat16, torch.float32


def _np(t):
    return t.detach().double().cpu().numpy()


def _round(dt, v):
    return np.abs(v) * (2.0 ** -8 if dt == BF16 else U) + (2.0 ** -134 if dt == BF16 else 2.0 ** -150)


def _within(got, want, tol, what):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / tol):.2f} of the bound"


def _x(N, H, dt, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, H, generator=g) * torch.exp(torch.randn(H, generator=g)) * scale + shift
    return x.to(dt)


def _rows_view(shape, dtype, off):
    """An uninitialised tensor that starts off bytes into its (256-byte aligned) storage."""
    size = torch.empty(0, dtype=dtype).element_size()
    n = int(np.prod(shape))
    flat = torch.empty(n + off // size, dtype=dtype, device=DEV)
    return flat[off // size:].view(shape)


# one column, less than a vector, odd, one block, blocks cut, several vectors a lane, the widest
WIDTHS = [1, 7, 8, 120, 128, 136, 257, 1001, 1408, 2048, 4104, 7168, 16384]


# ------------------------------------------------------------------------------------------------ checkpoints


def _assert_rows(got, x, what):
    """Checkpoint rows of x, byte for byte (q of a block without finite values is free)."""
    q, s = ref.quantise(x)
    want, got = ref.pack(q, s), got.cpu().numpy()
    C = x.shape[1]
    free = np.zeros(want.shape, bool)
    free[:, :C] = np.repeat(s == 255, 128, axis=1)[:, :C]
    bad = (got != want) & ~free
    assert not bad.any(), f"{what}: {bad.sum()} bytes differ, first at {np.argwhere(bad)[:3].tolist()}"


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", WIDTHS + [20001])
def test_ckpt_rows_and_values(C, dt):
    N = 37 if C < 2000 else 5
    x = _x(N, C, dt, C)
    ck = mep.mep_ckpt_save(x.to(DEV))
    assert ck.shape == (N, mep.ckpt_row_bytes(C)) and mep.ckpt_row_bytes(C) == ref.row_bytes(C)
    _assert_rows(ck, _np(x), "rows")
    want = ref.kept(_np(x))
    for out in (BF16, F32):
        np.testing.assert_array_equal(_np(mep.mep_ckpt_load(ck, C, dtype=out)), want)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [256, 300, 333])
def test_ckpt_special_values(C, dt):
    big = torch.finfo(dt).max
    x = torch.zeros(9, C, dtype=dt)
    x[0] = -0.0
    x[1, 5] = float("nan")
    x[2, 130] = float("inf")
    x[3, C - 1] = -float("inf")
    x[4] = torch.linspace(-1, 1, C).to(dt) * torch.tensor(big, dtype=dt)
    x[5, ::3] = 2.0 ** -133                       # subnormal in bf16 and fp32
    x[6] = torch.linspace(-1, 1, C).to(dt) * 2.0 ** -120
    x[7, :] = big
    x[8, 0], x[8, 1:] = big, 1.0                  # everything beside it is below a step
    ck = mep.mep_ckpt_save(x.to(DEV))
    _assert_rows(ck, _np(x), "rows")
    got = _np(mep.mep_ckpt_load(ck, C, dtype=BF16))
    np.testing.assert_array_equal(got, ref.kept(_np(x)))
    assert np.isnan(got[1, :128]).all() and not np.isnan(got[1, 128:]).any()
    assert np.isnan(got[2, 128:256]).all() and np.isnan(got[3, C - 1])


@pytest.mark.parametrize("off", [16, 32])
def test_ckpt_rows_16_bytes_into_their_storage(off):
    x = _rows_view((11, 264), BF16, off)
    x.copy_(_x(11, 264, BF16, 3))
    rb = mep.ckpt_row_bytes(264)
    ck = _rows_view((11, rb), torch.uint8, off)
    out = _rows_view((11, 264), BF16, off)
    mep.mep_ckpt_save(x, ck)
    _assert_rows(ck, _np(x), "rows")
    mep.mep_ckpt_load(ck, 264, out)
    np.testing.assert_array_equal(_np(out), ref.kept(_np(x)))


def test_ckpt_rows_through_dispatch():
    """Rows kept before mep_dispatch and permuted as bytes are the rows of the permuted activation."""
    R, S, K, E, B, H = 4, 33, 3, 8, 4, 200
    g = torch.Generator().manual_seed(5)
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(R * S)]).to(torch.int32).to(DEV)
    p = mep.mep_plan(idx, R, S, K, E, B)
    x = _x(R * S, H, BF16, 6).to(DEV)
    buf = mep.mep_dispatch(x, p.dst_pos, p.status, R, S, K)
    rows = mep.mep_dispatch(mep.mep_ckpt_save(x).view(BF16), p.dst_pos, p.status, R, S, K)
    assert int(p.status.item()) == 0
    assert torch.equal(rows.view(torch.uint8), mep.mep_ckpt_save(buf))


# ------------------------------------------------------------------------------------------------- layer norm


def _norm_tol(x, w, b, eps, dt):
    y, mean, rstd = ref.norm(x, w, b, eps)
    em = ((L + 1) * U * np.abs(x).mean(1))[:, None]
    var = ((x - mean[:, None]) ** 2).mean(1)[:, None]
    ax = np.abs(x) + np.abs(mean)[:, None]
    # the centred terms are themselves off by em + u (|x| + |mean|)
    ec = em + 2 * U * ax
    ev = (L + 4) * U * var + 2 * np.sqrt(var) * 2 * U * np.sqrt((ax ** 2).mean(1))[:, None] + (em + 2 * U * np.sqrt((ax ** 2).mean(1))[:, None]) ** 2
    er = 0.5 * ev / (var + eps) * (1 + 1e-3) + 3 * U  # relative error of rstd
    rs = rstd[:, None]
    xhat = np.abs((x - mean[:, None]) * rs)
    ey = np.abs(w) * (rs * ec + xhat * (er + 3 * U)) + 2 * U * (np.abs(w) * xhat + np.abs(b))
    return y, mean, rstd, ey + _round(dt, np.abs(y) + ey), em[:, 0] + U * np.abs(mean), (er * rs)[:, 0]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", WIDTHS)
def test_norm_forward(H, dt):
    N = 37 if H < 4000 else 6
    x = _x(N, H, dt, H, shift=0.5)
    g = torch.Generator().manual_seed(H)
    w, b = 1 + 0.3 * torch.randn(H, generator=g), torch.randn(H, generator=g)
    rb = mep.ckpt_row_bytes(H)
    xc, yc = (torch.full((N, rb), 77, dtype=torch.uint8, device=DEV) for _ in range(2))
    y, mean, rstd = mep.mep_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), 1e-5, x_ckpt=xc, y_ckpt=yc)
    want, m, r, ty, tm, tr = _norm_tol(_np(x), _np(w), _np(b), 1e-5, dt)
    _within(mean, m, tm, "mean")
    _within(rstd, r, tr, "rstd")
    _within(y, want, ty, "y")
    _assert_rows(xc, _np(x), "x_ckpt")
    _assert_rows(yc, _np(y), "y_ckpt")  # of y as it came out


@pytest.mark.parametrize("N", [1, 2, 3, 5, 63, 1000, 4099])
@pytest.mark.parametrize("H", [8, 96, 512, 1536])
def test_norm_row_counts(N, H):
    x = _x(N, H, BF16, N + H)
    dy = _x(N, H, BF16, N + H + 1)
    w = 1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(H))
    xd = x.to(DEV)
    y, mean, rstd = mep.mep_layer_norm(xd, w.to(DEV), None, 1e-5)
    want, m, r, ty, tm, tr = _norm_tol(_np(x), _np(w), np.zeros(H), 1e-5, BF16)
    _within(y, want, ty, "y")
    _check_backward(dy, x, w, mean, rstd, BF16)


@pytest.mark.parametrize("p_dt", [BF16, F32], ids=["params_bf16", "params_f32"])
@pytest.mark.parametrize("which", ["both", "weight", "bias", "none"])
def test_norm_parameter_types(which, p_dt):
    N, H = 19, 264
    x, dy = _x(N, H, BF16, 1), _x(N, H, BF16, 2)
    g = torch.Generator().manual_seed(3)
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(p_dt) if which in ("both", "weight") else None
    b = torch.randn(H, generator=g).to(p_dt) if which in ("both", "bias") else None
    wn = np.ones(H) if w is None else _np(w)
    bn = np.zeros(H) if b is None else _np(b)
    y, mean, rstd = mep.mep_layer_norm(x.to(DEV), None if w is None else w.to(DEV), None if b is None else b.to(DEV))
    want, _, _, ty, _, _ = _norm_tol(_np(x), wn, bn, 1e-5, BF16)
    _within(y, want, ty, "y")
    _check_backward(dy, x, w, mean, rstd, BF16)


def _backward_tol(dy, x, w, mean, rstd, dt):
    N, H = x.shape
    dx, dw, db = ref.norm_backward(dy, x, w, mean, rstd)
    rs = np.abs(rstd)[:, None]
    xhat = np.abs((x - mean[:, None]) * rstd[:, None])
    ex = 3 * U * (np.abs(x) + np.abs(mean)[:, None]) * rs
    t = np.abs(dy * w)
    s1, s2 = t.mean(1)[:, None], (t * xhat).mean(1)[:, None]
    e1 = (L + 3) * U * s1
    e2 = (L + 5) * U * s2 + (t * ex).mean(1)[:, None]
    # the sums' own sizes are bounded by those of their terms; the rest: four roundings of each of the three parts
    tol = rs * (e1 + xhat * e2 + ex * s2 + 5 * U * (t + s1 + xhat * s2))
    tw = (N + 4) * U * np.abs(dy * xhat).sum(0) + (np.abs(dy) * ex).sum(0)
    tb = (N + 1) * U * np.abs(dy).sum(0)
    return dx, dw, db, tol + _round(dt, np.abs(dx) + tol), tw + 2.0 ** -140, tb + 2.0 ** -140


def _check_backward(dy, x, w, mean, rstd, dt, ckpt=False):
    """x, dy, w on the host (w None or any type); mean, rstd on the device."""
    H = x.shape[1]
    xd = x.to(DEV)
    xn = _np(x)
    if ckpt:
        xd = mep.mep_ckpt_save(xd)
        xn = ref.kept(xn)
    wd = None if w is None else w.to(DEV)
    wn = np.ones(H) if w is None else _np(w)
    dx, dw, db = mep.mep_layer_norm_backward(dy.to(DEV), xd, wd, mean, rstd)
    want = _backward_tol(_np(dy), xn, wn, _np(mean), _np(rstd), dt)
    for got, v, tol, what in zip((dx, dw, db), want[:3], want[3:], ("dx", "dweight", "dbias")):
        _within(got, v, tol, what)
    alone = mep.mep_layer_norm_backward(dy.to(DEV), xd, wd, mean, rstd, params=False)
    assert alone[1] is None and alone[2] is None and torch.equal(alone[0], dx)


@pytest.mark.parametrize("ckpt", [False, True], ids=["as_it_was", "kept"])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", WIDTHS)
def test_norm_backward(H, dt, ckpt):
    N = 37 if H < 4000 else 6
    x, dy = _x(N, H, dt, H, shift=0.5), _x(N, H, dt, H + 1)
    w = 1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(H))
    _, mean, rstd = mep.mep_layer_norm(x.to(DEV), w.to(DEV), None)
    _check_backward(dy, x, w, mean, rstd, dt, ckpt)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [2050, 4099, 4104, 5120, 5128, 8200])
def test_norm_wide_rows_over_many_turns(H, dt):
    N = 1501
    x, dy = _x(N, H, dt, H, shift=0.5), _x(N, H, dt, H + 1)
    w = 1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(H))
    yc = torch.full((N, mep.ckpt_row_bytes(H)), 77, dtype=torch.uint8, device=DEV)
    y, mean, rstd = mep.mep_layer_norm(x.to(DEV), w.to(DEV), None, y_ckpt=yc)
    want, m, r, ty, tm, tr = _norm_tol(_np(x), _np(w), np.zeros(H), 1e-5, dt)
    _within(mean, m, tm, "mean")
    _within(rstd, r, tr, "rstd")
    _within(y, want, ty, "y")
    assert torch.equal(yc, mep.mep_ckpt_save(y))  # (rows against the plain form: test_ckpt_rows_and_values)
    for ckpt in (False, True):
        _check_backward(dy, x, w, mean, rstd, dt, ckpt)


def test_norm_rows_16_bytes_into_their_storage():
    N, H = 70, 272
    x, y, dy, dx = (_rows_view((N, H), BF16, 16) for _ in range(4))
    x.copy_(_x(N, H, BF16, 1))
    dy.copy_(_x(N, H, BF16, 2))
    w = _rows_view((H,), F32, 16)
    w.copy_(1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(3)))
    xc = _rows_view((N, mep.ckpt_row_bytes(H)), torch.uint8, 16)
    _, mean, rstd = mep.mep_layer_norm(x, w, w, 1e-5, y=y, x_ckpt=xc)
    want, _, _, ty, _, _ = _norm_tol(_np(x), _np(w), _np(w), 1e-5, BF16)
    _within(y, want, ty, "y")
    _assert_rows(xc, _np(x), "x_ckpt")
    for src, xn in ((x, _np(x)), (xc, ref.kept(_np(x)))):
        got = mep.mep_layer_norm_backward(dy, src, w, mean, rstd, dx=dx)
        want = _backward_tol(_np(dy), xn, _np(w), _np(mean), _np(rstd), BF16)
        for v, e, t, what in zip(got, want[:3], want[3:], ("dx", "dweight", "dbias")):
            _within(v, e, t, what)


def test_norm_far_offset_and_constant_rows():
    """Rows whose mean is far above their spread, and rows without spread."""
    x = torch.randn(4, 512, generator=torch.Generator().manual_seed(0)) + torch.tensor([[1e4], [-3e3], [0.0], [0.0]])
    x[2:] = torch.tensor([[7.25], [0.0]])
    y, mean, rstd = mep.mep_layer_norm(x.to(DEV))
    want, m, r, ty, tm, tr = _norm_tol(_np(x), np.ones(512), np.zeros(512), 1e-5, F32)
    _within(mean, m, tm, "mean")
    _within(rstd[:2], r[:2], tr[:2], "rstd")
    _within(y[:2], want[:2], ty[:2], "y")
    # 7.25 * 512 is exact in any order: nothing is left of these rows but rstd = eps^-1/2
    assert not y[2:].any() and torch.equal(mean[2:].cpu(), torch.tensor([7.25, 0.0]))
    np.testing.assert_allclose(_np(rstd[2:]), np.float32(1e-5) ** -0.5, rtol=4 * U)


def test_norm_nan_stays_in_its_row():
    N, H = 40, 384
    x, dy = _x(N, H, BF16, 1).to(DEV), _x(N, H, BF16, 2).to(DEV)
    clean = mep.mep_layer_norm(x)
    x[7, 3], x[11, 380] = float("nan"), float("inf")
    xc = torch.empty((N, mep.ckpt_row_bytes(H)), dtype=torch.uint8, device=DEV)
    y, mean, rstd = mep.mep_layer_norm(x, x_ckpt=xc)
    rows = torch.ones(N, dtype=torch.bool, device=DEV)
    rows[[7, 11]] = False
    assert torch.equal(y[rows], clean[0][rows]) and y[~rows].isnan().all()
    for src in (x, xc):
        dx, dw, db = mep.mep_layer_norm_backward(dy, src, None, mean, rstd)
        assert not dx[rows].isnan().any() and dx[~rows].isnan().all()
        assert dw.isnan().all() and not db.isnan().any()


def test_norm_gradients_add_to_what_is_there_and_repeat_their_bits():
    N, H = 700, 320
    x, dy = _x(N, H, BF16, 1).to(DEV), _x(N, H, BF16, 2).to(DEV)
    _, mean, rstd = mep.mep_layer_norm(x)
    _, dw, db = mep.mep_layer_norm_backward(dy, x, None, mean, rstd)
    again = mep.mep_layer_norm_backward(dy, x, None, mean, rstd)
    assert torch.equal(dw, again[1]) and torch.equal(db, again[2])
    w2, b2 = torch.full((H,), 3.0, device=DEV), torch.full((H,), -5.0, device=DEV)
    mep.mep_layer_norm_backward(dy, x, None, mean, rstd, dweight=w2, dbias=b2, accumulate=True)
    assert torch.equal(w2, 3.0 + dw) and torch.equal(b2, -5.0 + db)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [128, 2048, 4099])
def test_norm_one_workspace_for_batches_of_any_length(H, dt):
    long = 20000
    ws = torch.empty(mep.layer_norm_backward_workspace_bytes(long, H), dtype=torch.uint8, device=DEV)
    x, dy = (torch.randn(long, H, device=DEV, generator=torch.Generator(DEV).manual_seed(i)).to(dt) for i in (1, 2))
    _, mean, rstd = mep.mep_layer_norm(x)
    for n in (long, 4863, 1300, 607, 455, 3):
        ws.fill_(255)  # NaN, were any of it read before it is written
        got = mep.mep_layer_norm_backward(dy[:n], x[:n], None, mean[:n], rstd[:n], workspace=ws)
        want = mep.mep_layer_norm_backward(dy[:n], x[:n], None, mean[:n], rstd[:n])
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and not got[1].isnan().any()


def test_norm_without_rows():
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    y, mean, rstd = mep.mep_layer_norm(x)
    dx, dw, db = mep.mep_layer_norm_backward(x, x, None, mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    mep.mep_layer_norm_backward(x, x, None, mean, rstd, dweight=dw.fill_(2), dbias=db.fill_(3), accumulate=True)
    assert (dw == 2).all() and (db == 3).all()
    assert mep.mep_ckpt_load(mep.mep_ckpt_save(x), 64).shape == (0, 64)


def _directional(f, args, dirs, h):
    return (f(*[a + h * d for a, d in zip(args, dirs)]) - f(*[a - h * d for a, d in zip(args, dirs)])) / (2 * h)


def test_norm_gradients_against_differences():
    """<gradient, direction> against the central difference of the plain forward pass in 64 bits.

    The difference is off by h^2 / 6 times a third derivative (below 1e-7 of
    the sum of magnitudes at h = 1e-4 here) and 1e-16 / h; the kernel's
    gradients are within the bounds above, below 1e-4 of that sum."""
    N, H = 9, 200
    x, dy = _x(N, H, F32, 1), _x(N, H, F32, 2)
    g = torch.Generator().manual_seed(3)
    w, b = 1 + 0.3 * torch.randn(H, generator=g), torch.randn(H, generator=g)
    _, mean, rstd = mep.mep_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV))
    grads = [_np(t) for t in mep.mep_layer_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), mean, rstd)]
    args = [_np(t) for t in (x, w, b)]
    dirs = [np.random.default_rng(4 + i).normal(size=a.shape) for i, a in enumerate(args)]
    for k in range(3):
        only = [d if i == k else 0 * d for i, d in enumerate(dirs)]
        num = _directional(lambda *a: (ref.norm(*a, np.float32(1e-5))[0] * _np(dy)).sum(), args, only, 1e-4)
        ana = (grads[k] * dirs[k]).sum()
        assert abs(num - ana) <= 1e-4 * np.abs(grads[k] * dirs[k]).sum(), k


# ------------------------------------------------------------------------------------------------ gated activation


def _es(g):
    return U * (10 + 2.4 * np.abs(g))


def _swiglu_tol(g, u):
    a = ref.swiglu(g, u)
    e = np.abs(a) * (_es(g) + 3 * U) + np.abs(g * u) * 2.0 ** -125
    return a, e + _round(BF16, np.abs(a) + e)


def _swiglu_backward_tol(da, g, u):
    dg, du = ref.swiglu_backward(da, g, u)
    s, es, tiny = ref.sigmoid(g), _es(g), 2.0 ** -125
    # 1 - s is off by s es + u; g (1 - s) and the sum by two more roundings
    eg = np.abs(da * u) * ((s * (es + 3 * U) + tiny) * (1 + np.abs(g) * (1 - s)) + s * (np.abs(g) * (s * es + 3 * U) + 2 * U))
    eu = np.abs(da * g) * (s * (es + 3 * U) + tiny)
    return dg, du, eg + _round(BF16, np.abs(dg) + eg), eu + _round(BF16, np.abs(du) + eu)


def _check_swiglu(gu, da, off=0):
    rows, F = da.shape
    gd = _rows_view((rows, 2 * F), BF16, off)
    gd.copy_(gu)
    dd = _rows_view((rows, F), BF16, off)
    dd.copy_(da)
    a, again = _rows_view((rows, F), BF16, off), _rows_view((rows, F), BF16, off)
    dgu = _rows_view((rows, 2 * F), BF16, off)
    ck = _rows_view((rows, 2, mep.ckpt_row_bytes(F)), torch.uint8, off)
    ck.fill_(77)
    mep.mep_swiglu(gd, a=a, ckpt=ck)
    x = _np(gu).reshape(2 * rows, F)
    _assert_rows(ck.view(2 * rows, -1), x, "ckpt")
    g, u = x[0::2], x[1::2]
    want, tol = _swiglu_tol(g, u)
    _within(a, want, tol, "a")
    assert torch.equal(mep.mep_swiglu(gd), a)
    for src, kept in ((gd, x), (ck, ref.kept(x))):
        g, u = kept[0::2], kept[1::2]
        mep.mep_swiglu_backward(dd, src, dgu=dgu, a=again)
        dg, du, tg, tu = _swiglu_backward_tol(_np(da), g, u)
        _within(dgu[:, :F], dg, tg, "dg")
        _within(dgu[:, F:], du, tu, "du")
        want, tol = _swiglu_tol(g, u)
        _within(again, want, tol, "a again")
        alone, none = mep.mep_swiglu_backward(dd, src, again=False)
        assert none is None and torch.equal(alone, dgu)


@pytest.mark.parametrize("F", [1, 7, 8, 64, 128, 136, 200, 333, 704, 1408, 2050, 4096])
@pytest.mark.parametrize("rows", [1, 67])
def test_swiglu(rows, F):
    _check_swiglu(_x(rows, 2 * F, BF16, F, scale=2.0), _x(rows, F, BF16, F + 1))


@pytest.mark.parametrize("off", [16, 32])
@pytest.mark.parametrize("F", [64, 272])
def test_swiglu_rows_16_bytes_into_their_storage(F, off):
    _check_swiglu(_x(9, 2 * F, BF16, F, scale=2.0), _x(9, F, BF16, F + 1), off)


def test_swiglu_far_values():
    """Gates at which the exponential over- or underflows, and zeros."""
    g = torch.tensor([0.0, -0.0, 20.0, -20.0, 87.0, -87.0, 89.0, -89.0, 500.0, -500.0, 3e4, -3e4, 1e-30, -1e-30])
    u = torch.tensor([1.0, -2.0, 1e-20, 1e10])
    G, Uu = torch.meshgrid(g, u, indexing="ij")
    F = G.numel()
    gu = torch.cat([G.reshape(-1), Uu.reshape(-1)]).view(1, 2 * F).bfloat16()
    a = mep.mep_swiglu(gu.to(DEV))
    want, tol = _swiglu_tol(_np(gu)[:, :F], _np(gu)[:, F:])
    _within(a, want, tol, "a")
    da = torch.ones(1, F, dtype=BF16)
    dgu, _ = mep.mep_swiglu_backward(da.to(DEV), gu.to(DEV))
    dg, du, tg, tu = _swiglu_backward_tol(_np(da), _np(gu)[:, :F], _np(gu)[:, F:])
    _within(dgu[:, :F], dg, tg, "dg")
    _within(dgu[:, F:], du, tu, "du")


def test_swiglu_gates_whose_sigmoid_is_tiny():
    """Gates down to -104, where sigmoid leaves fp32's range, beside values that make their products large again.

    sigmoid(g) = k / (k + 2^(-g log2 e - 24)): the exponent is off by its rounding, 2^-24 (24 + 1.45 |g|), and that of
    log2 e, 2^-24 * 1.45 |g|, both times ln 2 in the result; ex2 adds 2^-22.5, the sum 2^-24, the reciprocal 2^-23: at most
    U (23 + 2 |g|). Subnormal results are off by 2^-149 at most instead, and so are products of them."""
    g = torch.linspace(-104, -80, 97)
    u = torch.tensor([1.0, -1e30, 1e38])
    G, Uu = torch.meshgrid(g, u, indexing="ij")
    F = G.numel()
    gu = torch.cat([G.reshape(-1), Uu.reshape(-1)]).view(1, 2 * F).bfloat16()
    gn, un = _np(gu)[:, :F], _np(gu)[:, F:]
    es, sub = U * (23 + 2 * np.abs(gn)), (1 + np.abs(gn)) * 2.0 ** -149
    want = ref.swiglu(gn, un)
    e = np.abs(want) * (es + 3 * U) + 2 * np.abs(un) * sub
    for a in (mep.mep_swiglu(gu.to(DEV)), mep.mep_swiglu_backward(torch.ones(1, F, dtype=BF16, device=DEV), gu.to(DEV))[1]):
        _within(a, want, e + _round(BF16, np.abs(want) + e), "a")
    dgu, _ = mep.mep_swiglu_backward(torch.ones(1, F, dtype=BF16, device=DEV), gu.to(DEV))
    dg, du = ref.swiglu_backward(np.ones_like(gn), gn, un)
    eg = np.abs(un) * ref.sigmoid(gn) * (1 + np.abs(gn)) * (es + 6 * U) + 2 * (1 + np.abs(un)) * sub
    eu = np.abs(du) * (es + 3 * U) + 2 * sub
    _within(dgu[:, :F], dg, eg + _round(BF16, np.abs(dg) + eg), "dg")
    _within(dgu[:, F:], du, eu + _round(BF16, np.abs(du) + eu), "du")
    assert (_np(dgu)[:, F:][gn > -90] != 0).all()


def test_swiglu_overflow_stays_visible():
    gu = torch.randn(4, 512, generator=torch.Generator().manual_seed(0)).bfloat16().to(DEV)
    gu[1, 5], gu[2, 256 + 200] = float("inf"), float("nan")
    ck = torch.empty((4, 2, mep.ckpt_row_bytes(256)), dtype=torch.uint8, device=DEV)
    mep.mep_swiglu(gu, ckpt=ck)
    dgu, a = mep.mep_swiglu_backward(torch.ones(4, 256, dtype=BF16, device=DEV), ck)
    assert a[1, :128].isnan().all() and not a[1, 128:].isnan().any()
    assert a[2, 128:].isnan().all() and not a[[0, 3]].isnan().any()
    assert dgu[2, 128:256].isnan().all()       # dg needs u


def test_swiglu_gradients_against_differences():
    """As for the norm: central differences of the plain form in 64 bits; the kernel's bf16 results are within 2^-8."""
    rows, F = 5, 72
    gu, da = _x(rows, 2 * F, BF16, 1), _x(rows, F, BF16, 2)
    dgu, _ = mep.mep_swiglu_backward(da.to(DEV), gu.to(DEV))
    d = np.random.default_rng(3).normal(size=(rows, 2 * F))
    num = _directional(lambda v: (ref.swiglu(v[:, :F], v[:, F:]) * _np(da)).sum(), [_np(gu)], [d], 1e-4)
    assert abs(num - (_np(dgu) * d).sum()) <= 2.0 ** -8 * np.abs(_np(dgu) * d).sum()


# ------------------------------------------------------------------------------------------------ many rows, large tensors


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,H", [(30001, 128), (30001, 256), (20001, 512), (9001, 1408), (8001, 2048)])
def test_norm_over_many_turns(N, H, dt):
    """So many rows that every CTA goes round its slots of rows copied ahead more than once."""
    x, dy = _x(N, H, dt, H, shift=0.5), _x(N, H, dt, H + 1)
    g = torch.Generator().manual_seed(H)
    w, b = 1 + 0.3 * torch.randn(H, generator=g), torch.randn(H, generator=g)
    rb = mep.ckpt_row_bytes(H)
    xc, yc = (torch.full((N, rb), 77, dtype=torch.uint8, device=DEV) for _ in range(2))
    y, mean, rstd = mep.mep_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV))
    want, m, r, ty, tm, tr = _norm_tol(_np(x), _np(w), _np(b), 1e-5, dt)
    _within(mean, m, tm, "mean")
    _within(rstd, r, tr, "rstd")
    _within(y, want, ty, "y")
    again = mep.mep_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), x_ckpt=xc, y_ckpt=yc)
    assert all(torch.equal(p, q) for p, q in zip(again, (y, mean, rstd)))
    assert torch.equal(xc, mep.mep_ckpt_save(x.to(DEV))) and torch.equal(yc, mep.mep_ckpt_save(y))
    dx, dw, db = mep.mep_layer_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), mean, rstd)
    want = _backward_tol(_np(dy), _np(x), _np(w), _np(mean), _np(rstd), dt)
    for got, v, tol, what in zip((dx, dw, db), want[:3], want[3:], ("dx", "dweight", "dbias")):
        _within(got, v, tol, what)


@pytest.mark.parametrize("H", [128, 264, 2048, 8200])
def test_fp32_rows_16_bytes_into_their_storage(H):
    """16 bytes off a 32-byte boundary: eight values go out in two pieces."""
    N = 45
    x, y, dy, dx, back = (_rows_view((N, H), F32, 16) for _ in range(5))
    assert x.data_ptr() % 32 == 16
    x.copy_(_x(N, H, F32, 1))
    dy.copy_(_x(N, H, F32, 2))
    w = _rows_view((H,), F32, 16)
    w.copy_(1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(3)))
    dw, db = _rows_view((H,), F32, 16), _rows_view((H,), F32, 16)
    xc = _rows_view((N, mep.ckpt_row_bytes(H)), torch.uint8, 16)
    _, mean, rstd = mep.mep_layer_norm(x, w, w, 1e-5, y=y, x_ckpt=xc)
    want, m, r, ty, tm, tr = _norm_tol(_np(x), _np(w), _np(w), 1e-5, F32)
    _within(y, want, ty, "y")
    _assert_rows(xc, _np(x), "x_ckpt")
    mep.mep_ckpt_load(xc, H, back)
    np.testing.assert_array_equal(_np(back), ref.kept(_np(x)))
    for src, xn in ((x, _np(x)), (xc, ref.kept(_np(x)))):
        got = mep.mep_layer_norm_backward(dy, src, w, mean, rstd, dx=dx, dweight=dw, dbias=db)
        want = _backward_tol(_np(dy), xn, _np(w), _np(mean), _np(rstd), F32)
        for v, e, t, what in zip(got, want[:3], want[3:], ("dx", "dweight", "dbias")):
            _within(v, e, t, what)


def _room(nbytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 1.2 * nbytes:
        pytest.skip("not enough memory")


def _runs(N, columns):
    """First, middle and last rows, and those around the 2^31st element."""
    at = 2 ** 31 // columns
    assert 4 < at < N - 5
    return [slice(0, 9), slice(N // 2, N // 2 + 9), slice(at - 4, at + 5), slice(N - 300, N)]


@pytest.mark.parametrize("N,H", [(300001, 7168), (1048201, 2049)])
def test_norm_of_more_than_2_31_elements(N, H):
    """Rows beyond 2^31 elements come out as they do on their own (tested above), bit for bit."""
    _room(22 << 30)
    assert N * H > 2 ** 31
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.randn(N, H, generator=g, device=DEV, dtype=BF16)
    w, b = torch.randn(H, generator=g, device=DEV), torch.randn(H, generator=g, device=DEV)
    xc, yc = (torch.empty((N, mep.ckpt_row_bytes(H)), dtype=torch.uint8, device=DEV) for _ in range(2))
    y, mean, rstd = mep.mep_layer_norm(x, w, b, x_ckpt=xc, y_ckpt=yc)
    dy = torch.randint(-1, 2, (N, H), generator=g, device=DEV, dtype=torch.int8).to(BF16)
    for run in _runs(N, H):
        want = mep.mep_layer_norm(x[run].clone(), w, b)
        assert all(torch.equal(p[run], q) for p, q in zip((y, mean, rstd), want))
        assert torch.equal(xc[run], mep.mep_ckpt_save(x[run].clone()))
        assert torch.equal(yc[run], mep.mep_ckpt_save(y[run].clone()))
    for src in (x, xc):
        dx, _, db = mep.mep_layer_norm_backward(dy, src, w, mean, rstd, dx=y)
        for run in _runs(N, H):
            want = mep.mep_layer_norm_backward(dy[run].clone(), src[run].clone(), w, mean[run].clone(), rstd[run].clone())
            assert torch.equal(dx[run], want[0])
        # -1, 0 and 1 add up to integers below 2^24: exact in any order
        assert torch.equal(db, dy.sum(0, dtype=torch.float32))


@pytest.mark.parametrize("rows,F", [(800001, 1408), (800001, 1407)])
def test_swiglu_of_more_than_2_31_elements(rows, F):
    _room(20 << 30)
    g = torch.Generator(DEV).manual_seed(1)
    gu = torch.randn(rows, 2 * F, generator=g, device=DEV, dtype=BF16)
    da = torch.randn(rows, F, generator=g, device=DEV, dtype=BF16)
    assert gu.numel() > 2 ** 31
    ck = torch.empty((rows, 2, mep.ckpt_row_bytes(F)), dtype=torch.uint8, device=DEV)
    a = mep.mep_swiglu(gu, ckpt=ck)
    for src in (gu, ck):
        dgu, again = mep.mep_swiglu_backward(da, src)
        for run in _runs(rows, 2 * F):
            want = mep.mep_swiglu_backward(da[run].clone(), src[run].clone())
            assert torch.equal(dgu[run], want[0]) and torch.equal(again[run], want[1])
        del dgu, again
    for run in _runs(rows, 2 * F):
        kept = torch.empty((ck[run].shape), dtype=torch.uint8, device=DEV)
        assert torch.equal(a[run], mep.mep_swiglu(gu[run].clone(), ckpt=kept)) and torch.equal(ck[run], kept)


@pytest.mark.parametrize("C", [8, 1])
def test_ckpt_of_more_blocks_than_a_launch_takes(C):
    """2^30 + 12345 rows of one block each: two launches."""
    N = 2 ** 30 + 12345
    _room(N * (32 + 4 * C))
    x = torch.zeros((N, C), dtype=BF16, device=DEV)
    runs = [slice(0, 100), slice(2 ** 30 - 50, 2 ** 30 + 50), slice(N - 100, N)]
    for run in runs:
        x[run] = torch.randn(100, C, device=DEV)
    ck = mep.mep_ckpt_save(x)
    for run in runs:
        assert torch.equal(ck[run], mep.mep_ckpt_save(x[run].clone()))
    back = mep.mep_ckpt_load(ck, C)
    assert back.numel() == x.numel()
    for run in runs:
        assert torch.equal(back[run], mep.mep_ckpt_load(ck[run].clone(), C))
        back[run] = 0
    assert not back.any()


# ------------------------------------------------------------------------------------------------ runs of rows


@pytest.mark.parametrize("first", range(1, 8))
@pytest.mark.parametrize("C", [9, 333, 2050])
def test_a_run_of_rows_of_a_larger_tensor(C, first):
    """Rows [first, first + n) of odd-width tensors, in place: results of the same rows on their own, nothing else touched."""
    n, total = 21, 40
    run = slice(first, first + n)

    def own(t):
        return t[run].clone()

    def untouched(t, v):
        return (t[:first] == v).all() and (t[first + n:] == v).all()

    for dt in (BF16, F32):
        x, dy = _x(total, C, dt, C + first).to(DEV), _x(total, C, dt, C + first + 1).to(DEV)
        params = torch.randn(2 * C, generator=torch.Generator().manual_seed(C)).to(DEV)
        w, b = params[:C], params[C:]  # one behind the other in one buffer
        y, dx = torch.full_like(x, 3.0), torch.full_like(x, 3.0)
        mean, rstd = torch.full((2, total), 3.0, device=DEV)
        xc = torch.empty((n, mep.ckpt_row_bytes(C)), dtype=torch.uint8, device=DEV)
        mep.mep_layer_norm(x[run], w, b, y=y[run], mean=mean[run], rstd=rstd[run], x_ckpt=xc)
        want = mep.mep_layer_norm(own(x), w.clone(), b.clone())
        assert all(torch.equal(a[run], v) and untouched(a, 3.0) for a, v in zip((y, mean, rstd), want))
        assert torch.equal(xc, mep.mep_ckpt_save(x[run])) and torch.equal(xc, mep.mep_ckpt_save(own(x)))
        back = torch.full_like(x, 3.0)
        mep.mep_ckpt_load(xc, C, back[run])
        assert torch.equal(back[run], mep.mep_ckpt_load(xc, C, dtype=dt)) and untouched(back, 3.0)
        for src in (x[run], xc):
            grads = torch.full((2 * C + 1,), 3.0, device=DEV)
            mep.mep_layer_norm_backward(dy[run], src, w, mean[run], rstd[run], dx=dx[run], dweight=grads[:C],
                                        dbias=grads[C:2 * C])
            want = mep.mep_layer_norm_backward(own(dy), src.clone(), w.clone(), own(mean), own(rstd))
            assert torch.equal(dx[run], want[0]) and untouched(dx, 3.0)
            assert torch.equal(grads[:C], want[1]) and torch.equal(grads[C:2 * C], want[2]) and grads[2 * C] == 3
    gu, da = _x(total, 2 * C, BF16, C + first + 2).to(DEV), _x(total, C, BF16, C + first + 3).to(DEV)
    a, again, dgu = torch.full_like(da, 3.0), torch.full_like(da, 3.0), torch.full_like(gu, 3.0)
    gc = torch.empty((n, 2, mep.ckpt_row_bytes(C)), dtype=torch.uint8, device=DEV)
    mep.mep_swiglu(gu[run], a=a[run], ckpt=gc)
    assert torch.equal(a[run], mep.mep_swiglu(own(gu))) and untouched(a, 3.0)
    for src in (gu[run], gc):
        mep.mep_swiglu_backward(da[run], src, dgu=dgu[run], a=again[run])
        want = mep.mep_swiglu_backward(own(da), src.clone())
        assert torch.equal(dgu[run], want[0]) and torch.equal(again[run], want[1])
        assert untouched(dgu, 3.0) and untouched(again, 3.0)


# ------------------------------------------------------------------------------------------------ streams, graphs, refusals


def test_on_another_stream_and_in_a_graph():
    N, H = 300, 512
    x, dy = _x(N, H, BF16, 1).to(DEV), _x(N, H, BF16, 2).to(DEV)
    gu, da = _x(N, 2 * H, BF16, 3).to(DEV), _x(N, H, BF16, 4).to(DEV)

    def step():
        xc = torch.empty((N, mep.ckpt_row_bytes(H)), dtype=torch.uint8, device=DEV)
        gc = torch.empty((N, 2, mep.ckpt_row_bytes(H)), dtype=torch.uint8, device=DEV)
        y, mean, rstd = mep.mep_layer_norm(x, x_ckpt=xc)
        out = [y, *mep.mep_layer_norm_backward(dy, xc, None, mean, rstd), mep.mep_swiglu(gu, ckpt=gc)]
        return out + [*mep.mep_swiglu_backward(da, gc), mep.mep_ckpt_load(mep.mep_ckpt_save(x), H)]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.add_(1)
    gu.mul_(0.5)
    graph.replay()
    replayed = [t.clone() for t in got]
    assert all(torch.equal(a, b) for a, b in zip(replayed, step()))


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF16, device=DEV)
    m = torch.zeros(4, device=DEV)
    with pytest.raises(TypeError):
        mep.mep_layer_norm(x.half())
    with pytest.raises(ValueError):
        mep.mep_layer_norm(x.t())                              # strides
    with pytest.raises(ValueError):
        mep.mep_layer_norm(x.cpu())
    with pytest.raises(ValueError):
        mep.mep_layer_norm(x, torch.ones(63, device=DEV))
    with pytest.raises(TypeError):
        mep.mep_layer_norm(x, torch.ones(64, device=DEV), torch.ones(64, dtype=BF16, device=DEV))
    with pytest.raises(mep.MepError):
        mep.mep_layer_norm(x, eps=-1.0)
    with pytest.raises(mep.MepError):
        mep.mep_layer_norm(x, eps=float("nan"))
    with pytest.raises(mep.MepError):
        mep.mep_layer_norm(torch.zeros(1, 16392, dtype=BF16, device=DEV))
    with pytest.raises(mep.MepError):                          # 8 bytes into its storage
        mep.mep_layer_norm(torch.zeros(4 * 64 + 4, dtype=BF16, device=DEV)[4:].view(4, 64))
    with pytest.raises(TypeError):                             # x in another type than dy
        mep.mep_layer_norm_backward(x, x.float(), None, m, m)
    with pytest.raises(ValueError):                            # rows of another width
        mep.mep_layer_norm_backward(x, torch.zeros(4, 64, dtype=torch.uint8, device=DEV), None, m, m)
    with pytest.raises(ValueError):
        mep.mep_layer_norm_backward(x, x, None, m, m, accumulate=True)
    with pytest.raises(ValueError):
        mep.mep_layer_norm_backward(x, x, None, m, m, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        mep.mep_ckpt_save(x.half())
    with pytest.raises(ValueError):
        mep.mep_ckpt_load(torch.zeros(4, 64, dtype=torch.uint8, device=DEV), 64)
    with pytest.raises(TypeError):
        mep.mep_ckpt_load(torch.zeros(4, 96, dtype=torch.uint8, device=DEV), 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        mep.mep_swiglu(torch.zeros(4, 63, dtype=BF16, device=DEV))
    with pytest.raises(TypeError):
        mep.mep_swiglu(x.float())
    with pytest.raises(ValueError):
        mep.mep_swiglu_backward(x, x)
    with pytest.raises(ValueError):
        mep.mep_swiglu_backward(x, torch.zeros(4, 2, 64, dtype=torch.uint8, device=DEV))
