"""The router's choice and its gradient against 64-bit forms.

Weights: fp32 exp (2 ulp), a sum of K terms and a division: relative error at
most (K + 8) * 2^-24 plus 2^-24 * (largest difference of logits) for the
rounded argument. Gradients: the sum of K products, a difference and a product,
(K + 4) * 2^-24 of the magnitudes; bf16 adds 2^-8 of the value."""

import numpy as np
import pytest
import torch

import load_balancing_topk_gb300 as mep
import serve_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(N, E, seed, dtype, kind="normal"):
    rng = np.random.default_rng([seed, N, E])
    x = rng.normal(size=(N, E)).astype(np.float32)
    if kind == "ties":
        x = np.round(x * 2) / 2
    elif kind == "masked":
        x[rng.random((N, E)) < 0.5] = -np.inf
        x[:: max(1, N // 5)] = -np.inf
    elif kind == "wide":
        x = x * np.float32(30)
    elif kind == "zeros":
        x = np.where(rng.random((N, E)) < 0.5, np.float32(0.0), np.float32(-0.0))
    elif kind == "lowest":
        x[rng.random((N, E)) < 0.5] = np.finfo(np.float32).min
        x[0] = np.finfo(np.float32).min
    elif kind == "nan":
        x[rng.random((N, E)) < 0.1] = np.nan
        x[rng.random((N, E)) < 0.05] = np.inf
        x[rng.random((N, E)) < 0.2] = -np.inf
    t = torch.from_numpy(x).to(dtype)
    return t.cuda(), t.float().numpy()


def check(t, x, K, bias, skip):
    b = None if bias is None else torch.from_numpy(bias).cuda()
    idx, w = mep.mep_route(t, K, b, skip_masked=skip)
    want_idx, want_w = ref.route(x, bias, K, skip)
    assert (idx.cpu().numpy() == want_idx).all()
    got = w.cpu().numpy().astype(np.float64)
    assert (np.isnan(got) == np.isnan(want_w)).all()
    top = np.take_along_axis(x.astype(np.float64), np.maximum(want_idx, 0), 1)
    fin = np.where(np.isfinite(top), top, 0)
    span = (fin.max(1) - fin.min(1))[:, None]
    fine = ~np.isnan(want_w)
    tol = ((K + 8) + span) * U * want_w + 2.0 ** -149
    assert (np.abs(got - want_w) <= tol)[fine].all()
    return idx, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,K", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (777, 43, 5), (129, 64, 6), (64, 256, 8), (33, 257, 9),
                                   (17, 384, 8), (9, 64, 64), (5, 4096, 64), (40, 1000, 1), (1000, 31, 31), (7, 33, 32),
                                   (3, 100, 33), (6, 511, 10), (4, 513, 8), (65, 128, 4), (9, 2049, 16), (200, 8, 2)])
def test_shapes(N, E, K, dtype):
    t, x = make(N, E, 1, dtype)
    check(t, x, K, None, False)


@pytest.mark.parametrize("kind", ["ties", "masked", "wide", "zeros", "lowest", "nan"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("N,E,K", [(60, 43, 5), (30, 256, 8), (11, 640, 12), (20, 16, 16)])
def test_values(kind, dtype, skip, N, E, K):
    t, x = make(N, E, 2, dtype, kind)
    check(t, x, K, None, skip)


@pytest.mark.parametrize("E", [20, 300, 700])
def test_every_nan_is_the_same_and_on_top(E):
    """Negative ones and ones with payloads too."""
    x = torch.zeros(4, E)
    bits = x.view(torch.int32)
    bits[0, 5], bits[0, 3], bits[0, 7] = 0x7FC00000, -(1 << 22), 0x7F800001
    x[1, 4], x[1, 2] = float("inf"), float("-inf")
    bits[1, 6] = -1
    bits[2, 0], bits[2, 1] = -(1 << 31), 0
    bits[3, 9] = -(1 << 23) + 1
    idx, w = mep.mep_route(x.cuda(), 3)
    assert idx.tolist() == [[3, 5, 7], [6, 4, 0], [0, 1, 2], [9, 0, 1]]
    assert torch.isnan(w[[0, 1, 3]]).all() and (w[2] - 1 / 3).abs().max() < 1e-6


@pytest.mark.parametrize("E,K", [(256, 8), (64, 6), (128, 32), (100, 3), (200, 33)])
@pytest.mark.parametrize("values", [1, 2, 3, 5, 9, 17, 33, 100])
def test_few_different_values(E, K, values):
    """From all equal (every value reaches any bound) to nearly all different; every choice by place."""
    g = torch.Generator(device="cuda").manual_seed(E + values)
    t = torch.randint(0, values, (400, E), generator=g, device="cuda").float()
    idx, _ = mep.mep_route(t, K)
    assert (idx.long() == torch.sort(t, dim=1, descending=True, stable=True)[1][:, :K]).all()


@pytest.mark.parametrize("kind", ["normal", "masked", "ties"])
def test_bias_chooses_but_does_not_weigh(kind):
    t, x = make(100, 64, 3, torch.float32, kind)
    bias = np.random.default_rng(4).normal(size=64).astype(np.float32) * 2
    idx, _ = check(t, x, 6, bias, True)
    plain, _ = mep.mep_route(t, 6, skip_masked=True)
    assert (idx != plain).any()


def test_rows_at_odd_addresses_and_given_outputs():
    base, x = make(50, 37, 5, torch.bfloat16)
    idx = torch.full((51, 3), -7, dtype=torch.int32, device="cuda")
    w = torch.full((51, 3), -7.0, device="cuda")
    got = mep.mep_route(base[7:20], 3, topk_idx=idx[1:14], topk_w=w[1:14])
    want = ref.route(x[7:20], None, 3, False)
    assert got[0].data_ptr() == idx[1:14].data_ptr()
    assert (idx[1:14].cpu().numpy() == want[0]).all()
    assert (idx[0] == -7).all() and (idx[14:] == -7).all() and (w[0] == -7).all() and (w[14:] == -7).all()


def test_agrees_with_the_synthetic_routing():
    from load_balancing_topk_gb300 import synth

    rng = np.random.default_rng(9)
    x = rng.normal(size=(500, 64)).astype(np.float32)
    idx, w = mep.mep_route(torch.from_numpy(x).cuda(), 6)
    want = synth._topk_desc(synth._order_key(x), 6)
    assert (idx.cpu().numpy() == want).all()
    assert np.abs(w.cpu().numpy() - synth._softmax_f32(np.take_along_axis(x, want, 1))).max() <= 20 * U


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,K", [(1, 1, 1), (5, 7, 3), (777, 43, 5), (129, 64, 6), (64, 256, 8), (33, 257, 9), (9, 64, 64),
                                   (5, 4096, 64), (1000, 31, 31), (3, 100, 33), (17, 384, 8), (4, 513, 8)])
def test_backward(N, E, K, dtype):
    t, x = make(N, E, 6, torch.float32, "masked")
    idx, w = mep.mep_route(t, K, skip_masked=True)
    dw = torch.randn(N, K, device="cuda")
    got = mep.mep_route_backward(dw, w, idx, E, dtype=dtype)
    want, mag = ref.route_backward(dw.double().cpu().numpy(), w.double().cpu().numpy(), idx.cpu().numpy(), E)
    tol = (K + 4) * U * mag + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    assert got.dtype == dtype
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


def test_backward_is_the_derivative():
    x = torch.randn(20, 24, dtype=torch.float64)
    dw = torch.randn(20, 5, dtype=torch.float64)
    idx, w = mep.mep_route(x.float().cuda(), 5)
    got = mep.mep_route_backward(dw.float().cuda(), w, idx, 24).double().cpu()
    at, h = idx.cpu().long(), 1e-6

    def loss(z):
        return (torch.softmax(torch.gather(z, 1, at), 1) * dw).sum(1)

    for e in range(24):
        up, down = x.clone(), x.clone()
        up[:, e] += h
        down[:, e] -= h
        diff = (loss(up) - loss(down)) / (2 * h)
        assert (diff - got[:, e]).abs().max() < 2e-6


def test_backward_repeated_and_bad_indices():
    idx = torch.tensor([[3, 3, 1], [0, -1, 2], [5, 1, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 0.25], [0.5, 0.0, 0.5], [0.2, 0.3, 0.5]], device="cuda")
    dw = torch.tensor([[1.0, -2.0, 0.5], [1.0, 7.0, 3.0], [1.0, 2.0, 3.0]], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, mag = ref.route_backward(dw[:2].double().cpu().numpy(), w[:2].double().cpu().numpy(), idx[:2].cpu().numpy(), 5)
    got = mep.mep_route_backward(dw[:2], w[:2], idx[:2], 5, status=status).double().cpu().numpy()
    assert (np.abs(got - want) <= 7 * U * mag).all() and int(status) == 0
    got = mep.mep_route_backward(dw, w, idx, 5, status=status).double().cpu().numpy()
    assert int(status) == mep.STATUS_CODE["MEP_ERR_BAD_ROUTING"]
    assert (np.abs(got[:2] - want) <= 7 * U * mag).all()
    keep = torch.full((3, 5), 9.0, device="cuda")
    mep.mep_route_backward(dw, w, idx, 5, dlogits=keep, status=status)
    assert (keep == 9).all()


@pytest.mark.parametrize("E,K", [(8, 4), (40, 35)])
def test_backward_leaves_out_what_was_not_chosen(E, K):
    """A place of -1 may hold anything: NaN in its gradient or its weight reaches no logit."""
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(9, E, generator=g, device="cuda")
    logits[2, 3:] = -float("inf")
    logits[5] = -float("inf")
    idx, w = mep.mep_route(logits, K, skip_masked=True)
    dw = torch.randn(9, K, generator=g, device="cuda")
    want = mep.mep_route_backward(dw, w, idx, E)
    dw[idx < 0] = float("nan")
    assert bool((idx < 0).any()) and torch.equal(mep.mep_route_backward(dw, w, idx, E), want)
    assert torch.equal(mep.mep_route_backward(dw, w.masked_fill(idx < 0, float("nan")), idx, E), want)


def test_many_rows_and_another_stream():
    N, E, K = 200003, 16, 2
    side = torch.cuda.Stream()
    t = torch.randn(N, E, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        idx, w = mep.mep_route(t, K)
        d = mep.mep_route_backward(w, w, idx, E)
    torch.cuda.current_stream().wait_stream(side)
    top, at = torch.sort(t, dim=1, descending=True, stable=True)  # (topk leaves the order of equal values open)
    top, at = top[:, :K], at[:, :K]
    assert (idx.long() == at).all()
    p = torch.softmax(top.double(), 1)
    want = torch.zeros(N, E, dtype=torch.float64, device="cuda").scatter_(1, at, p * (p - (p * p).sum(1, keepdim=True)))
    assert (d.double() - want).abs().max() < 1e-6


def test_more_than_2_31_logits():
    N, E, K = (1 << 31) // 4096 + 3, 4096, 3
    t = torch.zeros(N, E, dtype=torch.bfloat16, device="cuda")
    t[-1, 4000], t[-1, 17], t[-1, 4095] = 3.0, 2.0, 1.0
    idx, w = mep.mep_route(t, K)
    assert idx[-1].tolist() == [4000, 17, 4095] and idx[-2].tolist() == [0, 1, 2]
    del t
    d = mep.mep_route_backward(torch.ones_like(w) * torch.tensor([1.0, 2.0, 3.0], device="cuda"), w, idx, E, dtype=torch.bfloat16)
    assert int((d[-1] != 0).sum()) == 3 and int((d[-2] != 0).sum()) <= 3


def test_empty():
    t = torch.empty(0, 8, device="cuda")
    idx, w = mep.mep_route(t, 2)
    assert idx.shape == (0, 2) and mep.mep_route_backward(w, w, idx, 8).shape == (0, 8)


def test_graph():
    t = torch.randn(300, 40, device="cuda")
    dw = torch.randn(300, 4, device="cuda")
    mep.mep_route(t, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx, w = mep.mep_route(t, 4)
        d = mep.mep_route_backward(dw, w, idx, 40)
    for _ in range(3):
        t.copy_(torch.randn(300, 40, device="cuda"))
        g.replay()
        i2, w2 = mep.mep_route(t, 4)
        assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(d, mep.mep_route_backward(dw, w2, i2, 40))


def test_the_binding_refuses():
    t = torch.randn(4, 8, device="cuda")
    idx, w = mep.mep_route(t, 2)
    for f in (lambda: mep.mep_route(t, 0), lambda: mep.mep_route(t, 9), lambda: mep.mep_route(t.half(), 2),
              lambda: mep.mep_route(t.t(), 2), lambda: mep.mep_route(t, 2, torch.zeros(7, device="cuda")),
              lambda: mep.mep_route(t, 2, topk_idx=idx.long()), lambda: mep.mep_route_backward(w, w, idx.long(), 8),
              lambda: mep.mep_route_backward(w, w, idx, 1), lambda: mep.mep_route_backward(w, w, idx, 8, dtype=torch.float16),
              lambda: mep.mep_route(torch.randn(2, 200, device="cuda"), 65)):
        with pytest.raises((TypeError, ValueError, mep.MepError)):
            f()
