"""Host checks of the training operators' C ABI: sizes, types, null and misaligned pointers are
refused before anything reaches the GPU."""

import ctypes

import pytest

import load_balancing_topk_gb300 as mep
from load_balancing_topk_gb300 import _build

BF16, F32, CKPT8 = 0, 1, 2
BAD = mep.STATUS_CODE["MEP_ERR_INVALID_ARG"]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mep.load_library()


def test_row_bytes(lib):
    assert [mep.ckpt_row_bytes(c) for c in (1, 16, 128, 2048, 2049, 7168)] == [32, 32, 160, 2080, 2112, 7232]
    for c in (0, -1, (1 << 24) + 1):
        with pytest.raises(mep.MepError):
            mep.ckpt_row_bytes(c)
    assert lib.mep_ckpt_row_bytes(8, None) == BAD


def test_ckpt_rejects_bad_args(lib):
    for fn in (lambda *a: lib.mep_ckpt_save(*a, None), lambda x, t, N, C, k: lib.mep_ckpt_load(k, N, C, t, x, None)):
        assert fn(16, 3, 4, 64, 32) == BAD             # type
        assert fn(16, CKPT8, 4, 64, 32) == BAD         # type
        assert fn(16, BF16, -1, 64, 32) == BAD
        assert fn(16, BF16, 1 << 31, 64, 32) == BAD
        assert fn(16, BF16, 4, 0, 32) == BAD
        assert fn(16, BF16, 4, (1 << 24) + 1, 32) == BAD
        assert fn(None, BF16, 4, 64, 32) == BAD
        assert fn(16, BF16, 4, 64, None) == BAD
        assert fn(24, BF16, 4, 64, 32) == BAD          # misaligned
        assert fn(16, BF16, 4, 64, 40) == BAD
        assert fn(None, BF16, 0, 64, None) == 0        # no rows


def test_layer_norm_rejects_bad_args(lib):
    def fwd(x=16, t=BF16, w=16, b=16, pt=F32, eps=1e-5, N=4, H=64, y=16, m=16, r=16, xc=None, yc=None):
        return lib.mep_layer_norm(x, t, w, b, pt, eps, N, H, y, m, r, xc, yc, None)

    for kw in (dict(t=2), dict(t=-1), dict(pt=2), dict(eps=-1.0), dict(eps=float("nan")), dict(N=-1), dict(N=1 << 31),
               dict(H=0), dict(H=16385), dict(x=None), dict(y=None), dict(m=None), dict(r=None), dict(x=24), dict(w=24),
               dict(b=20), dict(y=24), dict(m=20), dict(r=20), dict(xc=24), dict(yc=24)):
        assert fwd(**kw) == BAD, kw
    assert fwd(x=None, y=None, m=None, r=None, N=0) == 0

    def bwd(dy=16, t=BF16, x=16, xt=BF16, w=16, pt=F32, m=16, r=16, N=4, H=64, ws=256, wb=1 << 20, dx=16, dw=16, db=16):
        return lib.mep_layer_norm_backward(dy, t, x, xt, w, pt, m, r, N, H, ws, wb, dx, dw, db, 0, None)

    need = mep.layer_norm_backward_workspace_bytes(4, 64)
    for kw in (dict(t=2), dict(xt=F32), dict(xt=3), dict(pt=2), dict(N=-1), dict(H=0), dict(H=16385), dict(dy=None),
               dict(x=None), dict(m=None), dict(r=None), dict(dx=None), dict(ws=None), dict(wb=need - 1), dict(dy=24),
               dict(x=24), dict(w=24), dict(m=20), dict(r=20), dict(ws=24), dict(dx=24), dict(dw=20), dict(db=20)):
        assert bwd(**kw) == BAD, kw
    for args in ((-1, 64), (4, 0), (4, 16385)):
        with pytest.raises(mep.MepError):
            mep.layer_norm_backward_workspace_bytes(*args)
    assert lib.mep_layer_norm_backward_workspace_bytes(4, 64, None) == BAD
    assert bwd(N=0, dw=None, db=None) == 0


# around every length at which the backward pass goes over to larger CTAs (152 * rows a turn * row groups), and beyond
LENGTHS = sorted({0, 1, 2, 1 << 20, (1 << 31) - 1, *(max(0, 152 * k + d) for k in range(1, 33) for d in (-1, 0, 1)), *range(5, 40000, 997)})


@pytest.mark.parametrize("H", [1, 128, 257, 640, 1001, 1408, 2048, 4099, 4104, 5120, 6144, 7168, 12288, 16384])
def test_a_norm_workspace_for_many_rows_serves_fewer(lib, H):
    sizes = [mep.layer_norm_backward_workspace_bytes(n, H) for n in LENGTHS]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("H,Hp", [(8, 8), (128, 64), (520, 1160), (2048, 1408)])
def test_a_wgrad_workspace_for_many_rows_serves_fewer(lib, H, Hp):
    sizes = [mep.grouped_wgrad_workspace_bytes(4, S, 2, 8, 4, H, Hp) for S in (0, 1, 2, 63, 64, 65, 500, 4096, 1 << 20)]
    assert sizes == sorted(sizes)


def test_swiglu_rejects_bad_args(lib):
    for args in ((None, 4, 64, 16, None), (16, 4, 64, None, None), (24, 4, 64, 16, None), (16, 4, 64, 24, None),
                 (16, 4, 64, 16, 24), (16, -1, 64, 16, None), (16, 1 << 30, 64, 16, None), (16, 4, 0, 16, None),
                 (16, 4, (1 << 24) + 1, 16, None)):
        assert lib.mep_swiglu(*args, None) == BAD, args
    assert lib.mep_swiglu(None, 0, 64, None, None, None) == 0
    for args in ((None, 16, BF16, 4, 64, 16, 16), (16, None, BF16, 4, 64, 16, 16), (16, 16, F32, 4, 64, 16, 16),
                 (16, 16, BF16, 4, 64, None, 16), (24, 16, BF16, 4, 64, 16, 16), (16, 24, BF16, 4, 64, 16, 16),
                 (16, 16, CKPT8, 4, 64, 24, 16), (16, 16, CKPT8, 4, 64, 16, 24), (16, 16, BF16, -1, 64, 16, 16),
                 (16, 16, BF16, 4, 0, 16, 16)):
        assert lib.mep_swiglu_backward(*args, None) == BAD, args
    assert lib.mep_swiglu_backward(None, None, BF16, 0, 64, None, None, None) == 0


def test_grouped_wgrad_rejects_bad_args(lib):
    need = mep.grouped_wgrad_workspace_bytes(2, 4, 2, 8, 4, 64, 64)

    def f(x=16, xt=BF16, dy=16, cu=16, R=2, S=4, K=2, E=8, B=4, H=64, Hp=64, ws=256, wb=None, home=16, slot=16):
        return lib.mep_grouped_wgrad(x, xt, dy, cu, None, R, S, K, E, B, H, Hp, 0, ws, need if wb is None else wb, home, slot,
                                     None)

    for kw in (dict(xt=F32), dict(xt=3), dict(R=0), dict(R=1025), dict(S=-1), dict(K=0), dict(K=65), dict(E=0), dict(E=4097),
               dict(B=-1), dict(B=32768), dict(H=4), dict(H=12), dict(Hp=0), dict(Hp=12), dict(S=1 << 30), dict(x=None),
               dict(dy=None), dict(cu=None), dict(home=None), dict(slot=None), dict(ws=None), dict(wb=need - 1), dict(x=24),
               dict(dy=24), dict(home=20), dict(slot=20), dict(ws=260)):
        assert f(**kw) == BAD, kw
    out = ctypes.c_size_t(0)
    assert lib.mep_grouped_wgrad_workspace_bytes(2, 4, 2, 8, 4, 64, 64, None) == BAD
    assert lib.mep_grouped_wgrad_workspace_bytes(0, 4, 2, 8, 4, 64, 64, ctypes.byref(out)) == BAD


def test_where_tensors_may_start(lib):
    """Whole vectors (a multiple of 8 columns): 16 bytes; other widths: the element; checkpoint rows and workspaces 16.
    (Only refusals: what is allowed is launched in the GPU tests.)"""
    for C in (63, 65, 1):
        assert lib.mep_ckpt_save(17, BF16, 4, C, 32, None) == BAD
        assert lib.mep_ckpt_save(18, F32, 4, C, 32, None) == BAD
        assert lib.mep_ckpt_save(16, BF16, 4, C, 34, None) == BAD
        assert lib.mep_ckpt_load(40, 4, C, BF16, 16, None) == BAD
        assert lib.mep_swiglu(17, 4, C, 16, None, None) == BAD
        assert lib.mep_swiglu(16, 4, C, 17, None, None) == BAD
        assert lib.mep_swiglu(16, 4, C, 16, 24, None) == BAD
        assert lib.mep_swiglu_backward(16, 24, CKPT8, 4, C, 16, 16, None) == BAD
        assert lib.mep_swiglu_backward(16, 17, BF16, 4, C, 16, 16, None) == BAD
        for at in range(4):  # x, y, mean, rstd
            p = [16] * 4
            p[at] = 18
            assert lib.mep_layer_norm(p[0], F32, 16, 16, F32, 1e-5, 4, C, p[1], p[2], p[3], None, None, None) == BAD
        for w, b, xc, yc in ((18, 16, None, None), (16, 18, None, None), (16, 16, 36, None), (16, 16, None, 36)):
            assert lib.mep_layer_norm(16, BF16, w, b, F32, 1e-5, 4, C, 16, 16, 16, xc, yc, None) == BAD
        assert lib.mep_layer_norm_backward(16, BF16, 24, CKPT8, 16, F32, 16, 16, 4, C, 256, 1 << 20, 16, 16, 16, 0, None) == BAD
        assert lib.mep_layer_norm_backward(16, BF16, 16, BF16, 16, F32, 16, 16, 4, C, 260, 1 << 20, 16, 16, 16, 0, None) == BAD
        assert lib.mep_layer_norm_backward(16, BF16, 16, BF16, 16, F32, 16, 16, 4, C, 256, 1 << 20, 16, 18, 16, 0, None) == BAD
