"""The layer bit for bit at the sizes of real use, on whole numbers.

Gates are whole and 17 at least, where fp32's silu(g) is g itself (1 + e^-17 rounds to 1); ups are whole, so that
activations are whole numbers of up to 17 bits: exact in two bf16, and in one only up to 8 bits. The sums of the second
product, whichever order they are taken in, stay whole and below 2^23, and the weights of the experts are small whole
numbers: everything up to the one rounding of the result is exact, and the result is the 64-bit one, rounded. Every
column's groups of 32, 64 or 128 rows hold a magnitude of 7 and no larger one, or nothing, so that their scale is 1 and 4
bits hold the weights as they are.

Beside them normal inputs, whose error in the 2-norm is that of the one rounding, 2^-8 at most, and of fp32 sums: leaving
out a single row of a sum shows in either."""

import pytest
import torch

import load_balancing_topk_gb300 as mep
import serve_ref as ref

pytestmark = pytest.mark.gpu
# T, K, E, H, F: the smallest, the medium layer, the large one, sums that end inside a step, a panel and a block
SIZES = [(1, 1, 1, 64, 64), (5, 2, 4, 200, 136), (1, 6, 64, 2048, 1408), (8, 6, 64, 2048, 1408), (64, 8, 16, 2048, 1408), (64, 1, 1, 2048, 1408),
         (1, 8, 8, 7168, 1408), (3, 2, 4, 7168, 1408), (16, 8, 32, 7168, 1408), (64, 2, 3, 7168, 1408), (40, 4, 8, 1000, 1000),
         (33, 3, 5, 4104, 72), (17, 3, 7, 136, 2504), (64, 8, 8, 2056, 520)]


def sparse(shape, g):
    """-1, 0, 0, 0, 0, 0, 0, 1."""
    r = torch.randint(0, 8, shape, generator=g, device="cuda", dtype=torch.int8)
    return (r == 7).to(torch.bfloat16) - (r == 0).to(torch.bfloat16)


def weights(H, F, g):
    """One expert's: rows 0 mod 32 of the first product are +-7, where x is 0 but for row 0 (row 16 instead for the ups),
    and the ups of columns 0 mod 32 are 0, whose activations are then 0 and whose rows of the second product hold +-7."""
    gate, up, down = sparse((H, F), g), sparse((H, F), g), sparse((F, H), g)
    for m in (gate, up, down):
        m[::32] = 7 * torch.randint(0, 2, m[::32].shape, generator=g, device="cuda").mul(2).sub(1).to(torch.bfloat16)
    gate[0] = 7
    up[16], up[0] = up[0].clone(), 0
    up[:, ::32] = 0
    return torch.cat([gate, up], 1), down


class Whole:
    def __init__(self, E, H, F, used, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.H, self.F = E, H, F
        self.w1 = torch.empty(E, H, 2 * F, dtype=torch.bfloat16, device="cuda")
        self.w2 = torch.empty(E, F, H, dtype=torch.bfloat16, device="cuda")
        for e in used:
            self.w1[e], self.w2[e] = weights(H, F, g)

    def tokens(self, T, K, used, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randint(-1, 2, (T, self.H), generator=g, device="cuda").to(torch.bfloat16)
        x[:, ::32] = x[:, 16:17] = 0
        x[:, 0] = 40
        idx = torch.stack([torch.tensor(used, device="cuda")[torch.randperm(len(used), generator=g, device="cuda")[:K]] for _ in range(T)])
        w = torch.randint(1, 4, (T, K), generator=g, device="cuda").float() * (1 - 2 * torch.randint(0, 2, (T, K), generator=g, device="cuda"))
        return x, idx.to(torch.int32), w

    def exact(self, x, idx, w):
        """In 64 bits; what makes it so is checked on the way."""
        out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        most = torch.zeros_like(out)
        for e in sorted(set(idx.flatten().tolist()) - {-1}):
            t, k = torch.nonzero(idx == e, as_tuple=True)
            gu, down = x[t].double() @ self.w1[e].double(), self.w2[e].double()
            g, u = gu[:, :self.F], gu[:, self.F:]
            a = g * u
            assert float(g.min()) >= 17 and float(a.abs().max()) <= 2 ** 17 and float((a.abs() @ down.abs()).max()) < 2 ** 23
            y = w[t, k].double()[:, None] * (a @ down)
            out.index_add_(0, t, y)
            most.index_add_(0, t, y.abs())
        assert float(most.max()) < 2 ** 24
        return out


def rounded(v):
    return v.float().to(torch.bfloat16)  # fp32 holds it


def in4(layer, used, group):
    w1 = torch.zeros(layer.E, 2, mep.w4_bytes(layer.H, layer.F, group), dtype=torch.uint8, device="cuda")
    w2 = torch.zeros(layer.E, 1, mep.w4_bytes(layer.F, layer.H, group), dtype=torch.uint8, device="cuda")
    for e in used:
        mep.mep_w4_save(layer.w1[e], group, parts=2, w4=w1[e])
        mep.mep_w4_save(layer.w2[e], group, w4=w2[e])
        assert torch.equal(mep.mep_w4_load(w1[e], layer.H, 2 * layer.F, group), layer.w1[e])
        assert torch.equal(mep.mep_w4_load(w2[e], layer.F, layer.H, group), layer.w2[e])
    return w1, w2


def run(x, idx, w, w1, w2, **kind):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mep.mep_expert_layer(x, idx, w, w1, w2, status, **kind)
    assert int(status) == 0
    return out


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("T,K,E,H,F", SIZES)
def test_whole_numbers(T, K, E, H, F, group):
    used = list(range(E))
    layer = Whole(E, H, F, used, 1)
    x, idx, w = layer.tokens(T, K, used, 2)
    if T > 4:
        idx[::5, 0] = -1
    kind, w1, w2 = {}, layer.w1, layer.w2
    if group:
        kind = dict(F=F, group=group)
        w1, w2 = in4(layer, used, group)
    got, want = run(x, idx, w, w1, w2, **kind), layer.exact(x, idx, w)
    assert torch.equal(got, rounded(want)), (int((got != rounded(want)).sum()), got.numel())


@pytest.mark.parametrize("group", [0, 128])
def test_whole_numbers_in_weights_beyond_2_31_elements(group):
    E, H, F, used = 256, 7168, 1408, [0, 1, 127, 150, 254, 255]
    layer = Whole(E, H, F, used, 3)
    kind, w1, w2 = {}, layer.w1, layer.w2
    if group:
        kind = dict(F=F, group=group)
        w1, w2 = in4(layer, used, group)
    for T, K in ((3, 2), (64, 3)):
        x, idx, w = layer.tokens(T, K, used, T)
        assert torch.equal(run(x, idx, w, w1, w2, **kind), rounded(layer.exact(x, idx, w)))


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T,H,F", [(1, 256, 128), (24, 2048, 1408), (2, 7168, 1408)])
def test_what_the_second_part_of_an_activation_holds(T, H, F, group):
    """Two activations whose first parts are (nearly) the same cancel: the result is the few bits that are left, each one
    right. Columns of the first product come in pairs whose ups differ by one row that x has at +-1."""
    layer = Whole(1, H, F, [0], 4)
    w1, w2 = layer.w1[0], layer.w2[0]
    up = w1[:, F:]
    w1[:, 1:F:2] = w1[:, 0:F:2]
    up[:, ::32] = up[:, 2 % F].unsqueeze(1)
    up[:, 1::2] = up[:, 0::2]
    up[5, 0::2], up[5, 1::2] = 0, 1
    w2.zero_()
    pairs, h = F // 2, torch.arange(H, device="cuda")
    w2[2 * (h % pairs), h], w2[2 * (h % pairs) + 1, h] = 7, -7
    x, idx, w = layer.tokens(T, 1, [0], 5)
    x[:, 5] = 1
    kind, q1, q2 = {}, layer.w1, layer.w2
    if group:
        kind = dict(F=F, group=group)
        q1, q2 = in4(layer, [0], group)
    got, want = run(x, idx, w, q1, q2, **kind), layer.exact(x, idx, w)
    gate = (x.double() @ w1.double())[:, :F:2][:, h % pairs]
    assert torch.equal(want, w.double() * -7 * gate)
    assert torch.equal(got, rounded(want))


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,K,E,H,F", [(1, 6, 64, 2048, 1408), (8, 6, 64, 2048, 1408), (64, 6, 64, 2048, 1408), (2, 2, 4, 7168, 1408), (64, 4, 8, 4096, 2048),
                                       (64, 8, 256, 2048, 512)])
def test_normal_inputs_in_the_norm(T, K, E, H, F, group):
    """One rounding to bf16 is off by 2^-8 of a value at most. Before it each of a sum's n additions is off by 2^-23 of the
    running sum, which is of the size of the result: n * 2^-23 if all went the same way, for gate, up and the second
    sum together (2 * 7168 + 1408) * 2^-23 < 2^-9."""
    g = torch.Generator(device="cuda").manual_seed(6)
    w1 = torch.empty(E, H, 2 * F, dtype=torch.bfloat16, device="cuda").normal_(0, H ** -0.5, generator=g)
    w2 = torch.empty(E, F, H, dtype=torch.bfloat16, device="cuda").normal_(0, F ** -0.5, generator=g)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]).to(torch.int32)
    w = torch.rand(T, K, generator=g, device="cuda")
    kind, v1, v2 = {}, w1, w2
    if group:
        kind, w1, w2 = dict(F=F, group=group), mep.mep_w4_save(w1, group, parts=2), mep.mep_w4_save(w2, group)
        v1, v2 = (lambda e: mep.mep_w4_load(w1[e], H, 2 * F, group, dtype=torch.float32)), (lambda e: mep.mep_w4_load(w2[e], F, H, group, dtype=torch.float32))
    got = run(x, idx, w, w1, w2, **kind).double()
    want, _ = ref.layer(x, idx, w, v1 if group else v1.__getitem__, v2 if group else v2.__getitem__)
    assert float((got - want).norm() / want.norm()) <= 2.0 ** -8 + 2.0 ** -9
