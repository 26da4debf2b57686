"""Host checks of the serving operators' and the router's C ABI, before anything reaches the GPU, and the plain
64-bit forms that their tests go by."""

import ctypes

import numpy as np
import pytest
import torch

import load_balancing_topk_gb300 as mep
import serve_ref as ref
from load_balancing_topk_gb300 import _build

BF16, F32, CKPT8, W4 = 0, 1, 2, 3
BAD = mep.STATUS_CODE["MEP_ERR_INVALID_ARG"]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mep.load_library()


def test_w4_bytes(lib):
    assert mep.w4_bytes(1, 1, 128) == 4224 and mep.w4_bytes(128, 64, 32) == 4608 and mep.w4_bytes(129, 65, 64) == 4 * 4352
    assert mep.w4_bytes(7168, 2816, 128) == 44 * 56 * 4224
    for K, N, group in ((0, 1, 128), (1, 0, 128), ((1 << 20) + 1, 1, 128), (1, (1 << 20) + 1, 128), (1, 1, 16), (1, 1, 0), (1, 1, -32)):
        with pytest.raises(mep.MepError):
            mep.w4_bytes(K, N, group)
    assert lib.mep_w4_bytes(1, 1, 128, None) == BAD


def test_w4_rejects_bad_args(lib):
    save = lambda w=16, t=BF16, M=2, K=8, N=16, parts=2, group=64, o=32: lib.mep_w4_save(w, t, M, K, N, parts, group, o, None)  # noqa: E731
    load = lambda w=16, t=BF16, M=2, K=8, N=16, parts=2, group=64, o=32: lib.mep_w4_load(o, M, K, N, parts, group, t, w, None)  # noqa: E731
    for f in (save, load):
        for kw in (dict(w=None), dict(o=None), dict(t=CKPT8), dict(t=W4), dict(t=-1), dict(M=-1), dict(M=1 << 31), dict(K=0),
                   dict(K=(1 << 20) + 1), dict(N=0), dict(N=17), dict(N=(1 << 21) + 2), dict(parts=0), dict(parts=-1), dict(group=16),
                   dict(group=96), dict(w=17), dict(w=18, t=F32), dict(o=40), dict(M=1 << 30, parts=2),
                   dict(M=1 << 20, K=1 << 20, N=1 << 20, parts=1)):
            assert f(**kw) == BAD, kw
        assert f(M=0, w=None, o=None) == 0


def test_w4_product_rejects_bad_args(lib):
    need = mep.w4_product_workspace_bytes(4, 64, 64, 128)

    def f(x=16, w=32, T=4, K=64, N=64, group=128, ws=256, wb=need, yt=BF16, y=16):
        return lib.mep_w4_product(x, w, None, T, K, N, group, ws, wb, yt, y, None)

    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(ws=None), dict(wb=need - 1), dict(T=-1), dict(T=65), dict(K=0), dict(N=0),
               dict(K=(1 << 20) + 1), dict(N=(1 << 20) + 1), dict(group=31), dict(yt=2), dict(yt=-1), dict(x=24), dict(w=40),
               dict(ws=260), dict(y=17), dict(y=18, yt=F32), dict(x=17, K=63)):
        assert f(**kw) == BAD, kw
    assert f(T=0, x=None, w=None, y=None, ws=None, wb=0) == 0
    out = ctypes.c_size_t(0)
    for args in ((65, 8, 8, 128), (-1, 8, 8, 128), (1, 0, 8, 128), (1, 8, 0, 128), (1, 8, 8, 100)):
        assert lib.mep_w4_product_workspace_bytes(*args, ctypes.byref(out)) == BAD
    assert lib.mep_w4_product_workspace_bytes(1, 8, 8, 128, None) == BAD


def test_expert_layer_rejects_bad_args(lib):
    need = mep.expert_layer_workspace_bytes(4, 2, 8, 64, 64)

    def f(x=16, i=16, w=16, w1=16, w2=16, t=BF16, group=0, T=4, K=2, E=8, H=64, F=64, ws=256, wb=need, o=16):
        return lib.mep_expert_layer(x, i, w, w1, w2, t, group, None, T, K, E, H, F, ws, wb, o, None)

    for kw in (dict(x=None), dict(i=None), dict(w=None), dict(w1=None), dict(w2=None), dict(ws=None), dict(o=None), dict(wb=need - 1),
               dict(t=F32), dict(t=CKPT8), dict(t=4), dict(t=W4, group=0), dict(t=W4, group=48), dict(T=-1), dict(T=65), dict(K=0),
               dict(K=65), dict(E=0), dict(E=4097), dict(H=4), dict(H=60), dict(F=0), dict(F=12), dict(H=65544),
               dict(F=32776), dict(x=24), dict(i=18), dict(w=18), dict(w1=24), dict(w2=24), dict(ws=260), dict(o=24)):
        assert f(**kw) == BAD, kw
    assert f(T=0, x=None, i=None, w=None, w1=None, w2=None, ws=None, wb=0, o=None) == 0
    out = ctypes.c_size_t(0)
    assert lib.mep_expert_layer_workspace_bytes(4, 2, 8, 64, 64, BF16, 0, None) == BAD
    assert lib.mep_expert_layer_workspace_bytes(65, 2, 8, 64, 64, BF16, 0, ctypes.byref(out)) == BAD


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("K,E,H,F", [(1, 1, 8, 8), (2, 8, 128, 64), (6, 64, 2048, 1408), (8, 256, 7168, 1408), (64, 4096, 64, 32)])
def test_a_layer_workspace_for_many_tokens_serves_fewer(lib, K, E, H, F, w4):
    sizes = [mep.expert_layer_workspace_bytes(T, K, E, H, F, w4) for T in range(65)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("K,N", [(1, 1), (7168, 7168), (2048, 65536), (1001, 1407)])
def test_a_product_workspace_for_many_rows_serves_fewer(lib, K, N):
    sizes = [mep.w4_product_workspace_bytes(T, K, N) for T in range(65)]
    assert sizes == sorted(sizes)


def test_route_rejects_bad_args(lib):
    fwd = lambda x=16, t=F32, b=16, N=4, E=8, K=2, i=16, w=16: lib.mep_route(x, t, b, N, E, K, 0, i, w, None)  # noqa: E731
    bwd = lambda x=16, t=F32, b=16, N=4, E=8, K=2, i=16, w=16: lib.mep_route_backward(b, w, i, None, N, E, K, t, x, None)  # noqa: E731
    for f in (fwd, bwd):
        for kw in (dict(x=None), dict(i=None), dict(w=None), dict(t=CKPT8), dict(t=-1), dict(N=-1), dict(N=1 << 31), dict(E=0),
                   dict(E=4097), dict(K=0), dict(K=9), dict(E=100, K=65), dict(x=17, t=BF16), dict(x=18), dict(i=18), dict(w=18), dict(b=18)):
            assert f(**kw) == BAD, kw
        assert f(N=0, x=None, i=None, w=None) == 0
    assert bwd(b=None) == BAD


# ------------------------------------------------------------------------------------------ the plain forms


def test_reference_quantises_as_defined():
    w = np.array([[7.0, 0.0, 1.0, np.inf], [-3.4, 0.0, -0.5, 1.0], [0.49, 0.0, 0.25, 2.0]])
    q, s = ref.w4_quantise(w, 32)
    assert q[:, 0].tolist() == [7, -3, 0] and s[0, 0] == 1.0
    assert (q[:, 1] == 0).all() and s[0, 1] == 0 and np.isnan(s[0, 3])
    assert abs(s[0, 2] - 1 / 7) <= 2.0 ** -8 / 7 and q[:, 2].tolist()[0] == 7
    v = ref.w4_values(q, s, 32)
    assert np.isnan(v[:, 3]).all() and (v[:, 1] == 0).all()


def test_reference_pack_places_every_weight_once():
    K, N = 130, 70
    q = np.random.default_rng(0).integers(-7, 8, (K, N))
    s = np.ones((-(-K // 64), N))
    b = ref.w4_pack(q, s, 64).reshape(2, 2, -1)
    halves = np.stack([b[:, :, :4096] & 15, b[:, :, :4096] >> 4])
    counts = np.bincount(halves.reshape(-1), minlength=16)
    want = np.bincount((q + 8).reshape(-1), minlength=16)
    want[8] += halves.size - q.size
    assert (counts == want).all()


def test_reference_route_against_torch():
    x = np.random.default_rng(1).normal(size=(50, 20)).astype(np.float32)
    idx, w = ref.route(x, None, 4, False)
    top, at = torch.topk(torch.from_numpy(x), 4, dim=1)
    assert (at.numpy() == idx).all() and np.abs(torch.softmax(top.double(), 1).numpy() - w).max() < 1e-15
    z = torch.from_numpy(x).double().requires_grad_(True)
    dw = torch.randn(50, 4, dtype=torch.float64)
    (torch.softmax(torch.gather(z, 1, at), 1) * dw).sum().backward()
    d, _ = ref.route_backward(dw.numpy(), w, idx, 20)
    assert np.abs(d - z.grad.numpy()).max() < 1e-12


def test_reference_layer_against_plain_products():
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(5, 16, generator=g), torch.rand(5, 2, generator=g)
    idx = torch.tensor([[0, 2], [1, -1], [-1, -1], [2, 1], [0, 1]], dtype=torch.int32)
    w1, w2 = torch.randn(3, 16, 16, generator=g), torch.randn(3, 8, 16, generator=g)
    out, bound = ref.layer(x, idx, w, lambda e: w1[e], lambda e: w2[e])
    most = torch.zeros(5, 16, dtype=torch.float64)
    for t in range(5):
        want = torch.zeros(16, dtype=torch.float64)
        for k in range(2):
            if idx[t, k] >= 0:
                gu = x[t].double() @ w1[idx[t, k]].double()
                a = torch.nn.functional.silu(gu[:8]) * gu[8:]
                want += w[t, k].double() * (a @ w2[idx[t, k]].double())
                most[t] += w[t, k].double() * (a.abs() @ w2[idx[t, k]].double().abs())
        assert (out[t] - want).abs().max() < 1e-12
    # two roundings to bf16, of the activation and of the result
    assert (out[2] == 0).all() and (bound >= 2.0 ** -8 * out.abs()).all() and (bound <= 3 * 2.0 ** -8 * most).all()
