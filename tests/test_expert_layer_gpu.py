"""The layer for a few tokens against its formula in 64 bits (bounds in serve_ref), from weights in bf16 and in
4 bits, and against the path that plans, permutes and multiplies."""

import numpy as np
import pytest
import torch

import load_balancing_topk_gb300 as mep
import serve_ref as ref

pytestmark = pytest.mark.gpu
BAD = mep.STATUS_CODE["MEP_ERR_BAD_ROUTING"]


class Layer:
    def __init__(self, E, H, F, seed=0, group=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.H, self.F, self.group = E, H, F, group
        self.p1 = torch.empty(E, H, 2 * F, dtype=torch.bfloat16, device="cuda").normal_(0, H ** -0.5, generator=g)
        self.p2 = torch.empty(E, F, H, dtype=torch.bfloat16, device="cuda").normal_(0, F ** -0.5, generator=g)
        self.kind = {}
        self.w1, self.w2 = self.p1, self.p2
        if group:
            self.kind = dict(F=F, group=group)
            self.save()

    def save(self):
        self.w1, self.w2 = mep.mep_w4_save(self.p1, self.group, parts=2), mep.mep_w4_save(self.p2, self.group)

    def m1(self, e):
        return mep.mep_w4_load(self.w1[e], self.H, 2 * self.F, self.group, dtype=torch.float32) if self.group else self.w1[e]

    def m2(self, e):
        return mep.mep_w4_load(self.w2[e], self.F, self.H, self.group, dtype=torch.float32) if self.group else self.w2[e]

    def __call__(self, x, idx, w, **kw):
        return mep.mep_expert_layer(x, idx, w, self.w1, self.w2, **self.kind, **kw)


def tokens(T, K, E, H, seed=0, skew=0.5, empty=0):
    rng = np.random.default_rng([seed, T, K, E])
    logits = rng.normal(size=(T, E)) - skew * np.log(rng.permutation(E) + 1.0)
    idx = np.argsort(-logits, 1)[:, :K].astype(np.int32)
    if empty:
        idx[rng.choice(T, empty, replace=False)] = -1
        idx[rng.random((T, K)) < 0.2] = -1
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand(T, K, generator=g, device="cuda") - 0.2
    return x, torch.from_numpy(idx).cuda(), w


def agrees(layer, x, idx, w, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = layer(x, idx, w, status=status, **kw)
    want, bound = ref.layer(x, idx, w, layer.m1, layer.m2)
    assert int(status) == 0
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), (float(off.max()), float(want.abs().max()))
    return got


SIZES = [(1, 1, 1, 8, 8), (1, 2, 3, 16, 8), (4, 2, 8, 128, 64), (1, 6, 64, 2048, 1408), (8, 6, 64, 2048, 1408), (64, 8, 16, 264, 72),
         (64, 1, 1, 136, 200), (17, 64, 64, 72, 40), (5, 4, 4096, 64, 32), (64, 8, 256, 512, 128), (2, 2, 4, 7168, 1408), (33, 3, 5, 104, 88),
         (16, 2, 2, 640, 328), (64, 4, 4, 1000, 1000), (3, 3, 7, 4104, 8), (3, 3, 7, 8, 4104), (63, 5, 9, 200, 120), (48, 1, 2, 256, 256),
         (64, 8, 256, 2048, 512), (16, 8, 128, 2048, 520)]


@pytest.mark.parametrize("group", [0, 128, 64, 32])
@pytest.mark.parametrize("T,K,E,H,F", SIZES)
def test_sizes(T, K, E, H, F, group):
    if group in (32, 64) and E * H * F > 1 << 24:
        pytest.skip("one group size is enough at this size")
    agrees(Layer(E, H, F, 1, group), *tokens(T, K, E, H, 2))


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T,K,E,H,F,empty", [(4, 2, 8, 128, 64, 1), (64, 8, 32, 264, 72, 20), (7, 3, 5, 40, 24, 6), (9, 1, 4, 64, 64, 9)])
def test_places_without_an_expert(T, K, E, H, F, empty, group):
    x, idx, w = tokens(T, K, E, H, 3, empty=empty)
    x[(idx < 0).all(1)] = float("nan")  # what an empty place holds is not read
    w[idx < 0] = float("nan")
    got = agrees(Layer(E, H, F, 4, group), x, idx, torch.where(idx < 0, torch.full_like(w, 3.0), w))
    assert (got[(idx < 0).all(1)] == 0).all()
    assert torch.equal(got, Layer(E, H, F, 4, group)(x, idx, w))


@pytest.mark.parametrize("group", [0, 32])
def test_no_expert_at_all_and_no_token(group):
    layer = Layer(4, 64, 32, 5, group)
    x, idx, w = tokens(6, 2, 4, 64, 6)
    assert (layer(x, torch.full_like(idx, -1), w) == 0).all()
    assert layer(x[:0], idx[:0], w[:0]).shape == (0, 64)


@pytest.mark.parametrize("group", [0, 128])
def test_skewed(group):
    """Every token on the same experts, and the experts' tokens from one to all."""
    layer = Layer(16, 200, 136, 7, group)
    x, idx, w = tokens(64, 3, 16, 200, 8, skew=0.0)
    idx[:] = torch.tensor([3, 0, 15], dtype=torch.int32)
    agrees(layer, x, idx, w)
    for n in (1, 7, 8, 9, 16, 17, 24, 25, 32, 33, 40, 48, 56, 57, 63):
        idx[:] = torch.tensor([3, 0, 15], dtype=torch.int32)
        idx[n:] = torch.tensor([3, 1, 2], dtype=torch.int32)
        agrees(layer, x, idx, w)


@pytest.mark.parametrize("group", [0, 64])
def test_bad_routing(group):
    layer = Layer(8, 64, 32, 9, group)
    x, idx, w = tokens(9, 3, 8, 64, 10)
    for t, k, v in ((0, 0, 8), (8, 2, -2), (4, 1, 1 << 30), (5, 2, int(idx[5, 0])), (8, 1, int(idx[8, 2])), (3, 0, -(1 << 31))):
        bad = idx.clone()
        bad[t, k] = v
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(x, 3.0)
        layer(x, bad, w, status=status, out=out)
        assert int(status) == BAD and (out == 3).all()
        layer(x, idx, w, status=status, out=out)  # the status holds
        assert int(status) == BAD and (out == 3).all()
        layer(x, bad, w, out=out)  # no status word: refused all the same
        assert (out == 3).all()
    agrees(layer, x, idx, w)


@pytest.mark.parametrize("group", [0, 128])
def test_unused_experts_are_not_read_and_nan_stays_with_its_expert(group):
    layer = Layer(8, 136, 72, 11, group)
    layer.p1[5], layer.p2[5] = float("nan"), float("inf")
    layer.p2[2, 3, 7] = float("nan")
    if group:
        layer.save()
    x, idx, w = tokens(12, 2, 5, 136, 12)
    got = layer(x, idx, w)
    hit = (idx == 2).any(1)
    assert hit.any() and not hit.all()
    nan = torch.isnan(got)
    assert nan[hit][:, 7].all() and not nan[~hit].any() and int(nan.sum()) == int(hit.sum())


@pytest.mark.parametrize("group", [0, 64])
def test_infinities_and_large_gates(group):
    """Gates far out on both sides: silu is 0 or the gate itself, never NaN."""
    layer = Layer(4, 64, 64, 13, group)
    layer.p1[:, :, :64] *= 400
    if group:
        layer.save()
    x, idx, w = tokens(16, 2, 4, 64, 14)
    got = agrees(layer, x, idx, w)
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("group", [0, 32])
def test_any_workspace_and_repeated_bits(group):
    layer = Layer(16, 512, 264, 15, group)
    x, idx, w = tokens(40, 4, 16, 512, 16)
    ws = torch.full((mep.expert_layer_workspace_bytes(64, 4, 16, 512, 264, bool(group), group or 128),), 255, dtype=torch.uint8, device="cuda")
    for n in (40, 1, 17, 40):
        out = torch.full((n + 1, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        got = layer(x[:n], idx[:n].contiguous(), w[:n].contiguous(), workspace=ws, out=out[:n])
        assert torch.equal(got, layer(x[:n], idx[:n].contiguous(), w[:n].contiguous())) and (out[n] == 7).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,K,E,H,F,same", [(1, 1, 1, 4096, 8, 1), (64, 1, 1, 2048, 64, 1), (64, 8, 8, 2048, 512, 1), (16, 8, 128, 2048, 512, 0),
                                            (64, 8, 256, 2048, 512, 0), (64, 8, 256, 2048, 512, 1), (3, 8, 256, 1024, 512, 0),
                                            (64, 2, 64, 8, 4096, 0), (40, 4, 16, 1000, 328, 0), (64, 64, 64, 264, 72, 0)])
def test_nothing_is_written_behind_the_workspace(T, K, E, H, F, same, group):
    """As many experts as can be in use and as few; one byte less is refused."""
    layer = Layer(E, H, F, 26, group)
    x, idx, w = tokens(T, K, E, H, 27, skew=0.0)
    if same:
        idx[:] = idx[0].clone()
    need = mep.expert_layer_workspace_bytes(T, K, E, H, F, bool(group), group or 128)
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    agrees(layer, x, idx, w, workspace=ws[:need])
    assert (ws[need:] == 0xA5).all()
    with pytest.raises(ValueError):
        layer(x, idx, w, workspace=ws[:need - 1])


def test_against_the_planned_path():
    R, S, K, E, H, F = 4, 16, 3, 8, 256, 192
    layer = Layer(E, H, F, 17)
    x, idx, w = tokens(R * S, K, E, H, 18)
    p = mep.mep_plan(idx, R, S, K, E, E // R)
    buf = mep.mep_dispatch(x, p.dst_pos, p.status, R, S, K)

    def product(v, home):
        slot = torch.zeros(R, E // R, *home.shape[1:], dtype=torch.bfloat16, device="cuda")
        mep.mep_prefetch(p.slot_expert, home, slot, p.status, E)
        return mep.mep_grouped_gemm(v, p.cu_seqlens, home, slot, p.status, R, S, K)

    a = mep.mep_swiglu(product(buf, layer.p1))
    planned = mep.mep_combine(product(a, layer.p2), w, p.dst_pos, p.status, R, S, K)
    assert int(p.status) == 0
    got = agrees(layer, x, idx, w)
    # the planned path rounds the gates, the ups and the experts' outputs to bf16 as well
    assert float((got.double() - planned.double()).norm() / got.double().norm()) < 4 * 2.0 ** -8


@pytest.mark.parametrize("group", [0, 64])
def test_streams_at_once(group):
    layer = Layer(8, 512, 256, 19, group)
    calls = [tokens(T, 2, 8, 512, T) for T in (1, 5, 64)]
    want = [layer(*c) for c in calls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in calls], [[] for _ in calls]
    for _ in range(10):
        for i, (s, c) in enumerate(zip(streams, calls)):
            with torch.cuda.stream(s):
                got[i].append(layer(*c))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[i]) for i in range(3) for v in got[i])


@pytest.mark.parametrize("group", [0, 128])
def test_captured_step_with_new_tokens(group):
    """Two captured graphs with one workspace, replayed in turn on new routings, bad ones and empty places among them."""
    T, K, E, H, F = 12, 3, 10, 264, 136
    layer = Layer(E, H, F, 20, group)
    x, idx, w = tokens(T, K, E, H, 21)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(mep.expert_layer_workspace_bytes(T, K, E, H, F, bool(group), group or 128), dtype=torch.uint8, device="cuda")
    layer(x, idx, w, status=status, workspace=ws)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer(x, idx, w, status=status, workspace=ws)
        graphs.append((g, out))
    for seed in range(6):
        g, out = graphs[seed % 2]
        nx, ni, nw = tokens(T, K, E, H, 30 + seed, skew=seed / 2, empty=seed)
        for a, b in ((x, nx), (idx, ni), (w, nw)):
            a.copy_(b)
        status.zero_()
        g.replay()
        assert int(status) == 0 and torch.equal(out, layer(nx, ni, nw))
        idx[3, 1] = E
        before = out.clone()
        g.replay()
        assert int(status) == BAD and torch.equal(out, before)


def test_after_the_router_with_masked_experts():
    """Norm, router product, choice with masked experts and an empty row, layer: as a decoding step runs them."""
    T, K, E, H, F = 6, 3, 8, 256, 128
    layer = Layer(E, H, F, 22, 64)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    router = torch.randn(H, E, device="cuda") * H ** -0.5
    y, _, _ = mep.mep_layer_norm(x)
    logits = y.float() @ router
    logits[:, 5] = -float("inf")
    logits[4] = -float("inf")
    logits[1, 2:] = -float("inf")
    idx, w = mep.mep_route(logits, K, skip_masked=True)
    got = agrees(layer, y, idx, w)
    assert (got[4] == 0).all() and not (idx == 5).any() and int((idx[1] >= 0).sum()) == 2


def test_weights_beyond_2_31_elements():
    E, H, F = 256, 7168, 1408
    p1 = torch.empty(E, H, 2 * F, dtype=torch.bfloat16, device="cuda")
    p2 = torch.empty(E, F, H, dtype=torch.bfloat16, device="cuda")
    layer = Layer(1, 8, 8)
    layer.E, layer.H, layer.F, layer.w1, layer.w2 = E, H, F, p1, p2
    for e in (0, 150, 254, 255):
        p1[e].normal_(0, H ** -0.5)
        p2[e].normal_(0, F ** -0.5)
    x, _, w = tokens(3, 2, 4, H, 23)
    agrees(layer, x, torch.tensor([[255, 0], [150, 255], [254, 255]], dtype=torch.int32, device="cuda"), w)
    layer.group, layer.kind = 128, dict(F=F, group=128)
    layer.w1 = torch.empty(E, 2, mep.w4_bytes(H, F), dtype=torch.uint8, device="cuda")
    layer.w2 = torch.empty(E, 1, mep.w4_bytes(F, H), dtype=torch.uint8, device="cuda")
    for e in (0, 150, 254, 255):
        mep.mep_w4_save(p1[e], parts=2, w4=layer.w1[e])
        mep.mep_w4_save(p2[e], w4=layer.w2[e])
    agrees(layer, x, torch.tensor([[255, 0], [150, 255], [254, 255]], dtype=torch.int32, device="cuda"), w)


def test_the_binding_refuses():
    layer, four = Layer(4, 64, 32, 24), Layer(4, 64, 32, 24, 64)
    x, idx, w = tokens(3, 2, 4, 64, 25)
    call = mep.mep_expert_layer
    for f in (lambda: call(x.float(), idx, w, layer.w1, layer.w2), lambda: call(x, idx.long(), w, layer.w1, layer.w2),
              lambda: call(x, idx, w.double(), layer.w1, layer.w2), lambda: call(x, idx, w, layer.w1[:, :, :-1], layer.w2),
              lambda: call(x, idx, w, layer.w1, layer.w2[:3]), lambda: call(x, idx, w, layer.w1, four.w2),
              lambda: call(x, idx, w, four.w1, four.w2), lambda: call(x, idx, w, four.w1, four.w2, F=32, group=128),
              lambda: call(x, idx, w, four.w1, layer.w2, F=32, group=64), lambda: call(x, idx[:2], w, layer.w1, layer.w2),
              lambda: call(x, idx, w, layer.w1, layer.w2, F=33), lambda: call(x, idx, w, layer.w1, layer.w2, out=x[:2]),
              lambda: call(x, idx, w, layer.w1, layer.w2, workspace=torch.empty(1, dtype=torch.uint8, device="cuda")),
              lambda: call(x, idx, w, layer.w1.cpu(), layer.w2), lambda: call(x[:, :60].contiguous(), idx, w, layer.w1, layer.w2),
              lambda: call(x.repeat(30, 1), idx.repeat(30, 1), w.repeat(30, 1), layer.w1, layer.w2)):
        with pytest.raises((TypeError, ValueError, mep.MepError)):
            f()
