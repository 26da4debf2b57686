"""The serving operators at the limits of the header: the widest layers, the longest and widest matrices in 4 bits, as many
assignments as a layer takes. Normal inputs, in the norm: one rounding of the result (2^-8 in bf16, 2^-24 in fp32) and
2^-23 of the running sum, which is of the size of the result, for each of a sum's additions."""

import pytest
import torch

import load_balancing_topk_gb300 as mep

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(*shape, g, scale=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=g)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def product(x, w, step=1 << 14):
    """x @ w in 64 bits, a few rows of w at a time."""
    return sum(x[:, k:k + step].double() @ w[k:k + step].double() for k in range(0, x.shape[1], step))


def layer(x, idx, w, w1, w2):
    out, F = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), w2.shape[1]
    for e in sorted(set(idx.flatten().tolist()) - {-1}):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        gu = product(x[t], w1[e])
        a = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        out.index_add_(0, t, w[t, k].double()[:, None] * product(a, w2[e]))
    return out


def check_layer(x, idx, w, w1, w2, group):
    E, H, F = w1.shape[0], w1.shape[1], w2.shape[1]
    kind, q1, q2 = {}, w1, w2
    if group:
        kind, q1, q2 = dict(F=F, group=group), mep.mep_w4_save(w1, group, parts=2), mep.mep_w4_save(w2, group)
        w1 = mep.mep_w4_load(q1, H, 2 * F, group, dtype=torch.float32)
        w2 = mep.mep_w4_load(q2, F, H, group, dtype=torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = mep.expert_layer_workspace_bytes(x.shape[0], idx.shape[1], E, H, F, bool(group), group or 128)
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = mep.mep_expert_layer(x, idx, w, q1, q2, status, workspace=ws[:need], **kind)
    assert int(status) == 0 and bool((ws[need:] == 0xA5).all())
    assert off(got, layer(x, idx, w, w1, w2)) <= 2.0 ** -8 + (2 * H + F) * 2.0 ** -23


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T,E,H,F", [(2, 1, 65536, 32768), (64, 2, 65536, 72), (33, 2, 136, 32768)])
def test_the_widest_layers(T, E, H, F, group):
    g = gen(1)
    w1, w2 = normal(E, H, 2 * F, g=g, scale=H ** -0.5), normal(E, F, H, g=g, scale=F ** -0.5)
    idx = torch.arange(T, device="cuda", dtype=torch.int32).remainder(E)[:, None]
    check_layer(normal(T, H, g=g), idx, torch.ones(T, 1, device="cuda"), w1, w2, group)


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("E,H,F", [(4096, 64, 32), (64, 136, 72), (100, 520, 264)])
def test_as_many_assignments_as_there_can_be(E, H, F, group):
    """64 tokens of 64 experts each: every expert in use, or every token on every expert."""
    g = gen(2)
    w1, w2 = normal(E, H, 2 * F, g=g, scale=H ** -0.5), normal(E, F, H, g=g, scale=F ** -0.5)
    if E == 4096:
        idx = torch.randperm(E, generator=g, device="cuda").reshape(64, 64)
    else:
        idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:64] for _ in range(64)])
    check_layer(normal(64, H, g=g), idx.to(torch.int32), torch.rand(64, 64, generator=g, device="cuda"), w1, w2, group)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T,K,N", [(3, 1 << 20, 65), (64, (1 << 20) - 3, 8), (3, 40, 1 << 20), (64, 129, (1 << 20) - 1)])
def test_the_longest_and_the_widest_matrices(T, K, N, group):
    g = gen(3)
    x, w = normal(T, K, g=g), normal(K, N, g=g)
    w4 = mep.mep_w4_save(w, group)
    w = mep.mep_w4_load(w4, K, N, group, dtype=torch.float32)
    need = mep.w4_product_workspace_bytes(T, K, N, group)
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = mep.mep_w4_product(x, w4, N, group, dtype=torch.float32, workspace=ws[:need])
    assert bool((ws[need:] == 0xA5).all())
    assert off(got, product(x, w)) <= 2.0 ** -24 + K * 2.0 ** -23
