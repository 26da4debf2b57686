"""The layer's results where floating point ends: infinite weights and activations, gates whose silu is tiny, activations
between bf16's largest number and fp32's.

Inputs are whole numbers or powers of two where that makes the formula's value exact; elsewhere the bound is what the
header promises: an activation off by 2^-16 of itself (2^-20 more for exp, division and products), a result by 2^-8."""

import pytest
import torch

import load_balancing_topk_gb300 as mep

pytestmark = pytest.mark.gpu
INF = float("inf")


def layer(w1, w2, x, idx, w, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mep.mep_expert_layer(x, idx, w, w1, w2, status, **kw)
    assert int(status) == 0
    return out


def whole(H, F, T, seed, E=2):
    """x, w1 and gates and ups in 64 bits: x[t, 0] = 1 and one more column of x is t's own, so that a gate is 20 + t % 8
    (fp32's silu of it is itself) and an up runs through -120 .. 120 without 0; activations are whole, up to 3240."""
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(T, H)
    x[:, 0] = 1
    x[:, 1] = torch.arange(T) % 8
    x[:, H - 1] = 1
    w1 = torch.zeros(E, H, 2 * F)
    w1[:, 0, :F] = 20
    w1[:, 1, :F] = 1
    up = torch.randint(1, 121, (E, F), generator=g) * (1 - 2 * torch.randint(0, 2, (E, F), generator=g))
    w1[:, H - 1, F:] = up.float()
    a = (20 + torch.arange(T) % 8)[None, :, None].double() * up[:, None, :].double()  # [E, T, F]
    return x.bfloat16().cuda(), w1.bfloat16().cuda(), a.cuda()


def same(got, want):
    """bf16 values equal to 64-bit ones that fp32 holds; any NaN is a NaN."""
    want = want.float().bfloat16()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan]), int((got[~nan] != want[~nan]).sum())


@pytest.mark.parametrize("H,F,T", [(64, 32, 5), (256, 200, 40), (2048, 1408, 8), (7168, 1408, 3)])
def test_an_infinite_weight_of_the_second_product(H, F, T):
    """A single infinity in a column makes the result infinite, of the activation's sign times its own; two of opposite
    signs make it NaN; the other columns are as they would be."""
    x, w1, a = whole(H, F, T, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    w2 = torch.randint(-1, 2, (2, F, H), generator=g, device="cuda").bfloat16()
    for h, rows in ((0, [0]), (1, [F - 1]), (H // 2, [F // 2]), (H - 1, [7]), (9, [0, F - 1]), (17, [3, 4])):
        for n, f in enumerate(rows):
            w2[0, f, h] = INF if (h + n) % 2 else -INF
    w2[0, :, 25] = INF  # NaN where activations of both signs meet it
    w2[1, 2, 30] = -INF
    idx = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(T, 1)
    idx[-1, 0] = -1
    w = torch.tensor([[1.0, 2.0]], device="cuda").repeat(T, 1)
    got = layer(w1, w2, x, idx, w)
    want = 2 * (a[1] @ w2[1].double())
    want[:-1] += (a[0] @ w2[0].double())[:-1]
    assert torch.isinf(want[0, [0, 1, H // 2, H - 1, 30]]).all() and torch.isnan(want[0, 25]) and torch.isfinite(want[-1, :30]).all()
    same(got, want)


@pytest.mark.parametrize("side", [1, -1])
def test_an_infinite_activation(side):
    """A gate times an up beyond fp32: the columns that it meets are infinite, nothing is NaN but where the weight is 0."""
    H, F, T = 136, 72, 9
    x, w1, a = whole(H, F, T, 3)
    w1[0, 1, F + 5] = side * 3e38
    g = torch.Generator(device="cuda").manual_seed(4)
    w2 = torch.randint(0, 2, (2, F, H), generator=g, device="cuda").mul(2).sub(1).bfloat16()
    w2[0, 5, 11] = 0
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    got = layer(w1, w2, x, idx, torch.ones(T, 1, device="cuda"))
    act = a[0].clone()
    act[1:, 5] = side * INF  # x[t, 1] is 0 for tokens 0 and 8
    act[8, 5] = a[0, 8, 5]
    want = act @ w2[0].double()
    assert torch.isinf(want[3]).sum() == H - 1 and torch.isnan(want[3, 11]) and torch.isfinite(want[[0, 8]]).all()
    same(got, want)


@pytest.mark.parametrize("group", [0, 32, 128])
def test_gates_whose_sigmoid_is_tiny(group):
    """From -87 down to -104 silu is 1e-37 to 1e-43 of 1, which an up of 1e38 makes an ordinary activation."""
    H, F, T = 64, 128, 4
    gates = -torch.linspace(86.5, 104, F).bfloat16().float()
    x = torch.zeros(T, H).bfloat16().cuda()
    x[:, 0], x[:, 40] = 1, torch.tensor([1, -1, 0.5, 2]).cuda()
    w1 = torch.zeros(1, H, 2 * F)
    w1[0, 0, :F], w1[0, 40, F:] = gates, 1e38
    w2 = torch.zeros(1, F, H)
    w2[0, torch.arange(F), torch.arange(F) % H] = torch.where(torch.arange(F) < H, 1.0, 0.0)
    w2b = w2.roll(H, 1)  # the second half of the gates
    w1 = w1.bfloat16().cuda()
    kind, q1, v1 = {}, w1, w1
    if group:
        q1, kind = mep.mep_w4_save(w1, group, parts=2), dict(F=F, group=group)
        v1 = mep.mep_w4_load(q1, H, 2 * F, group, dtype=torch.float32)
    gu = x.double() @ v1[0].double()
    g, u = gu[:, :F], gu[:, F:]
    a = g / (1 + torch.exp(-g)) * u
    idx, w = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    for m in (w2, w2b):
        q2 = v2 = m.bfloat16().cuda()
        if group:
            q2 = mep.mep_w4_save(q2, group)
            v2 = mep.mep_w4_load(q2, F, H, group, dtype=torch.float32)
        got = layer(q1, q2, x, idx, w, **kind)
        want = a @ v2[0].double()
        assert float(want.abs().min()) > 1e-6
        assert ((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -16 + 2.0 ** -19) * want.abs()).all()


def test_gates_further_out_are_zeros():
    """Below that the activation leaves fp32: zeros, whatever the sign, never NaN."""
    H, F, T = 64, 128, 2
    x, w1 = torch.zeros(T, H, device="cuda").bfloat16(), torch.zeros(1, H, 2 * F, device="cuda").bfloat16()
    x[:, 0] = torch.tensor([1, 2]).cuda()
    w1[0, 0, :F] = -torch.logspace(2.7, 37.9, F, device="cuda")
    w1[0, 0, F:] = 1e30
    w2 = torch.ones(1, F, H, device="cuda").bfloat16()
    got = layer(w1, w2, x, torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda"))
    assert (got == 0).all()


def test_activations_between_the_largest_bf16_and_the_largest_fp32():
    """3.3965e38 rounds to infinity in bf16 and is a number in fp32; times 2^-30 it is an ordinary result."""
    H, F, T = 64, 8, 2
    top_bf16, top = float(torch.finfo(torch.bfloat16).max), float(torch.finfo(torch.float32).max)
    gates = torch.arange(17, 250).double()
    ups = (torch.arange(128, 256).double() * 2.0 ** 113)[:, None] * 2.0 ** -torch.arange(0, 9).double()[None, :]
    a = gates[:, None, None] * ups
    at = torch.nonzero((a > (top_bf16 + 2.0 ** 128) / 2) & (a < top * (1 - 2.0 ** -10)))
    at = at[torch.linspace(0, len(at) - 1, F).long()]
    gate, up = gates[at[:, 0]], ups[at[:, 1], at[:, 2]]
    x, w1, w2 = torch.zeros(T, H), torch.zeros(1, H, 2 * F), torch.zeros(1, F, H)
    x[:, 0], x[0, 33], x[1, 33] = 1, 1, -1
    w1[0, 0, :F], w1[0, 33, F:] = gate.float(), up.float()
    w2[0, torch.arange(F), torch.arange(F)] = 2.0 ** -30
    got = layer(w1.bfloat16().cuda(), w2.bfloat16().cuda(), x.bfloat16().cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"),
                torch.ones(T, 1, device="cuda"))
    want = (gate * up * 2.0 ** -30).cuda()
    for t, sign in ((0, 1), (1, -1)):
        assert ((got[t, :F].double() - sign * want).abs() <= (2.0 ** -8 + 2.0 ** -16 + 2.0 ** -20) * want).all(), got[t, :F]
    assert (got[:, F:] == 0).all()
