"""The plain 64-bit forms of the training operators against things known otherwise."""

import numpy as np
import pytest
import torch

import train_ref as ref


def test_checkpoint_of_known_values():
    x = np.zeros((3, 130))
    x[0, :4] = [1.0, -0.5, 1.0 / 64, 3.0 / 128]   # largest 1: step 2^-6; 1.5 steps go to the even 2
    x[1, 5] = 127.5                                # step 1: kept at 127
    x[2, 129] = 2.0 ** -133                        # smallest bf16: step 2^-126, gone
    q, s = ref.quantise(x)
    assert q[0, :4].tolist() == [64, -32, 1, 2] and s[0].tolist() == [121, 1]
    assert q[1, 5] == 127 and s[1, 0] == 127
    assert not q[2].any() and s[2].tolist() == [1, 1]
    v = ref.values(q, s)
    assert v[0, :4].tolist() == [1.0, -0.5, 1.0 / 64, 2.0 / 64]
    rows = ref.pack(q, s)
    assert rows.shape == (3, 160) and rows[0, 144] == 121 and rows[0, 145] == 1 and not rows[:, 146:].any()


@pytest.mark.parametrize("C,want", [(1, 32), (16, 32), (128, 160), (2048, 2080), (2049, 2112), (7168, 7232)])
def test_row_bytes(C, want):
    assert ref.row_bytes(C) == want


def test_checkpoint_error_is_half_a_step_for_bf16():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(64, 257, generator=g) * torch.exp(4 * torch.randn(64, 1, generator=g))).bfloat16().double().numpy()
    q, s = ref.quantise(x)
    half = np.repeat(np.ldexp(1.0, s - 128), 128, axis=1)[:, :257]
    assert (np.abs(ref.values(q, s) - x) <= half).all()
    top = np.abs(np.pad(x, ((0, 0), (0, 127))).reshape(64, 3, 128)).max(2)
    assert (np.ldexp(1.0, s - 128) <= top / 128).all()
    v = ref.values(q, s)
    assert (torch.from_numpy(v).bfloat16().double().numpy() == v).all()  # exact in bf16


def test_gradients_are_the_automatic_ones():
    rng = np.random.default_rng(1)
    x, w, b, dy = rng.normal(size=(5, 37)), rng.normal(size=37), rng.normal(size=37), rng.normal(size=(5, 37))
    xt, wt, bt = (torch.from_numpy(v).requires_grad_() for v in (x, w, b))
    y, mean, rstd = ref.norm(x, w, b, 1e-5)
    out = torch.nn.functional.layer_norm(xt, (37,), wt, bt, 1e-5)
    np.testing.assert_allclose(out.detach().numpy(), y, rtol=1e-12, atol=1e-12)
    out.backward(torch.from_numpy(dy))
    for got, t in zip(ref.norm_backward(dy, x, w, mean, rstd), (xt, wt, bt)):
        np.testing.assert_allclose(got, t.grad.numpy(), rtol=1e-11, atol=1e-12)
    g, u, da = (torch.from_numpy(rng.normal(size=(4, 9)) * 3).requires_grad_() for _ in range(3))
    a = torch.nn.functional.silu(g) * u
    np.testing.assert_allclose(a.detach().numpy(), ref.swiglu(g.detach().numpy(), u.detach().numpy()), rtol=1e-12)
    a.backward(da.detach())
    dg, du = ref.swiglu_backward(da.detach().numpy(), g.detach().numpy(), u.detach().numpy())
    np.testing.assert_allclose(dg, g.grad.numpy(), rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(du, u.grad.numpy(), rtol=1e-11, atol=1e-13)


def test_wgrad_is_the_gradient_of_the_grouped_product():
    rng = np.random.default_rng(2)
    cu = np.array([[3, 3, 7, 9], [0, 6, 6, 9]])  # E = 3, B = 1, two ranks of 9 rows
    x, dy = rng.normal(size=(18, 4)), rng.normal(size=(18, 5))
    home, slot, _, _ = ref.wgrad(x, dy, cu, 3)
    wh = torch.zeros(3, 4, 5, dtype=torch.float64, requires_grad=True)
    ws = torch.zeros(2, 1, 4, 5, dtype=torch.float64, requires_grad=True)
    loss = 0.0
    for r in range(2):
        for row in range(9):
            j = int(np.searchsorted(cu[r], row, side="right"))
            w = wh[j] if j < 3 else ws[r, j - 3]
            loss = loss + (torch.from_numpy(x[9 * r + row]) @ w * torch.from_numpy(dy[9 * r + row])).sum()
    loss.backward()
    np.testing.assert_allclose(home, wh.grad.numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(slot, ws.grad.numpy(), rtol=1e-12, atol=1e-14)
