"""Weights in 4 bits: stored byte for byte as the definition says, read back exactly, and multiplied within
the bound of serve_ref (bit for bit where every sum is exact in fp32)."""

import numpy as np
import pytest
import torch

import load_balancing_topk_gb300 as mep
import serve_ref as ref

pytestmark = pytest.mark.gpu


def weights(K, N, seed, dtype, kind="normal"):
    rng = np.random.default_rng([seed, K, N])
    w = rng.normal(size=(K, N)).astype(np.float32)
    if kind == "special":
        w[:, ::5] = 0
        w[::3, 1::5] *= 1e-38
        w[:, 2 % N] = 1e-41
        w[:, 3 % N] = np.float32(3e38)
        w[0, 4 % N] = np.inf
        w[K // 2, 7 % N] = np.nan
        w[:, 8 % N] = rng.integers(-7, 8, K) * 0.5 + 0.25  # halves between steps
    return torch.from_numpy(w).to(dtype)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,N,kind", [(1, 1, "normal"), (128, 64, "normal"), (130, 66, "special"), (31, 70, "special"), (200, 17, "normal"),
                                      (257, 129, "special")])
def test_bytes(K, N, kind, dtype, group):
    w = weights(K, N, 1, dtype, kind)
    q, s = ref.w4_quantise(w.double().numpy(), group)
    got = mep.mep_w4_save(w.cuda(), group=group)
    assert got.shape == (1, mep.w4_bytes(K, N, group)) and mep.w4_bytes(K, N, group) == ref.w4_bytes(K, N, group)
    want = ref.w4_pack(q, s, group)
    g, nan = got[0].cpu().numpy(), np.isnan(s)
    if nan.any():  # a NaN's bits are free: compare them as values below
        q = np.where(np.repeat(nan, group, 0)[:K], 0, q)
        want = ref.w4_pack(q, s, group)
        block = 4096 + 128 // group * 128
        a, b = (torch.from_numpy(v.reshape(-1, block)[:, 4096:].copy()).view(torch.bfloat16).float() for v in (g, want))
        assert torch.equal(torch.nan_to_num(a, nan=-1.0), torch.nan_to_num(b, nan=-1.0))
        assert (g.reshape(-1, block)[:, :4096] == want.reshape(-1, block)[:, :4096]).all()
    else:
        assert (g == want).all()
    back = mep.mep_w4_load(got, K, N, group=group, dtype=torch.float32).cpu().double().numpy()
    v = ref.w4_values(q, s, group)
    assert (np.isnan(back) == np.isnan(v)).all() and (np.nan_to_num(back) == np.nan_to_num(v)).all()
    half = mep.mep_w4_load(got, K, N, group=group).cpu()
    assert torch.equal(torch.nan_to_num(half.float()), torch.nan_to_num(torch.from_numpy(v).float().to(torch.bfloat16).float()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("exponent", [0, 100, 117, -60, -90, -98, -100, -104, -115, -126, -130])
def test_quotients_next_to_half_steps(dtype, exponent):
    """w around (n + 1/2) s by single steps of fp32, scales of many sizes: q as the division in fp32 rounds it."""
    K, N, group = 128, 4096, 32
    g = torch.Generator(device="cuda").manual_seed(exponent + 200)
    top = (1 + torch.rand(K // group, 1, N, generator=g, device="cuda")) * 2.0 ** exponent
    scale = (top * (torch.ones(1, device="cuda") / 7)).to(torch.bfloat16).float()
    n = torch.randint(-7, 7, (K // group, group, N), generator=g, device="cuda").float() + 0.5
    w = n * scale
    step = torch.randint(-3, 4, w.shape, generator=g, device="cuda", dtype=torch.int32)
    w = torch.where(w.abs() > 2.0 ** -120, (w.view(torch.int32) + step).view(torch.float32), w)
    w = torch.minimum(torch.maximum(w, -top), top)
    w[:, 0] = top[:, 0]
    w = w.reshape(K, N).to(dtype).reshape(K // group, group, N)
    top = w.float().abs().amax(1, keepdim=True)
    scale = (top * (torch.ones(1, device="cuda") / 7)).to(torch.bfloat16).float()
    want = torch.round(w.float() / torch.where(scale > 0, scale, torch.ones_like(scale))).clamp(-7, 7) * scale
    got = mep.mep_w4_load(mep.mep_w4_save(w.reshape(K, N), group=group), K, N, group=group, dtype=torch.float32)
    assert torch.equal(got.reshape(w.shape), torch.where(scale > 0, want, torch.zeros_like(want)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_parts_and_batches(dtype):
    M, K, F, group = 3, 200, 72, 64
    w = torch.randn(M, K, 2 * F).to(dtype).cuda()
    got = mep.mep_w4_save(w, group=group, parts=2)
    assert got.shape == (M, 2, mep.w4_bytes(K, F, group))
    for m in range(M):
        for p in range(2):
            alone = mep.mep_w4_save(w[m, :, p * F:(p + 1) * F].contiguous(), group=group)
            assert torch.equal(got[m, p], alone[0])
    assert torch.equal(mep.mep_w4_load(got, K, 2 * F, group=group, dtype=dtype)[1],
                       mep.mep_w4_load(mep.mep_w4_save(w[1], group=group), K, 2 * F, group=group, dtype=dtype))


def test_weights_at_odd_addresses_and_given_outputs():
    base = torch.randn(65 * 77 + 1, device="cuda").to(torch.bfloat16)
    w = base[1:].view(65, 77)
    out = torch.zeros(1, mep.w4_bytes(65, 77), dtype=torch.uint8, device="cuda")
    mep.mep_w4_save(w, w4=out)
    assert torch.equal(out, mep.mep_w4_save(w.clone()))
    back = torch.zeros(65 * 77 + 2, dtype=torch.bfloat16, device="cuda")
    mep.mep_w4_load(out, 65, 77, w=back[1:-1].view(65, 77))
    assert torch.equal(back[1:-1].view(65, 77), mep.mep_w4_load(out, 65, 77)) and back[0] == 0 and back[-1] == 0


def test_more_than_2_31_weights():
    M, K, N = 9, 16384, 16384
    w = torch.zeros(M, K, N, dtype=torch.bfloat16, device="cuda")
    w[-1] = torch.randn(K, N, device="cuda")
    w4 = mep.mep_w4_save(w)
    assert torch.equal(w4[-1], mep.mep_w4_save(w[-1]))
    w.zero_()
    mep.mep_w4_load(w4, K, N, w=w)
    assert torch.equal(w[-1], mep.mep_w4_load(w4[-1], K, N))


PRODUCTS = [(1, 1, 1, 128), (1, 128, 64, 128), (3, 8, 5, 32), (5, 1001, 1407, 32), (8, 1000, 130, 64), (9, 256, 64, 128), (16, 384, 192, 64),
            (17, 2048, 700, 128), (33, 136, 1000, 32), (64, 512, 256, 64), (64, 1408, 2048, 128), (1, 7168, 7168, 128), (2, 7168, 100, 64),
            (40, 4104, 72, 32), (1, 65, 20000, 64), (64, 33, 3, 32), (24, 127, 129, 32), (25, 640, 65, 128), (32, 129, 127, 64)]


@pytest.mark.parametrize("T,K,N,group", PRODUCTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product(T, K, N, group, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + K + N)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    w4 = mep.mep_w4_save(torch.randn(K, N, generator=g, device="cuda"), group=group)
    got = mep.mep_w4_product(x, w4, N, group=group, dtype=dtype)
    want, mag = ref.product(x, mep.mep_w4_load(w4, K, N, group=group, dtype=torch.float32))
    assert got.dtype == dtype and got.shape == (T, N)
    assert ((got.double() - want).abs() <= ref.product_bound(want, mag, K, 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24)).all()


@pytest.mark.parametrize("T,K,N,group", PRODUCTS)
def test_product_of_whole_numbers_is_exact(T, K, N, group):
    """Scales 2^-1 .. 2^1 (a group's largest magnitude is 7 steps), |x| <= 2: sums stay whole halves below 2^23."""
    rng = np.random.default_rng([T, K, N])
    q = rng.integers(-7, 8, (K, N))
    q[::32] = 7
    s = np.repeat(2.0 ** rng.integers(-1, 2, (-(-K // group), N)), group, 0)[:K]
    w = torch.from_numpy(q * s).float().cuda()
    w4 = mep.mep_w4_save(w, group=group)
    assert torch.equal(mep.mep_w4_load(w4, K, N, group=group, dtype=torch.float32), w)
    x = torch.from_numpy(rng.integers(-2, 3, (T, K))).to(torch.bfloat16).cuda()
    got = mep.mep_w4_product(x, w4, N, group=group, dtype=torch.float32)
    assert torch.equal(got.double(), x.double() @ w.double())


def test_product_repeats_its_bits_and_takes_any_workspace():
    T, K, N = 20, 1408, 1000
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    w4 = mep.mep_w4_save(torch.randn(K, N, device="cuda"))
    want = mep.mep_w4_product(x, w4, N)
    ws = torch.full((mep.w4_product_workspace_bytes(64, K, N) + 64,), 255, dtype=torch.uint8, device="cuda")
    for t in (20, 1, 13):
        got = mep.mep_w4_product(x[:t], w4, N, workspace=ws)
        assert torch.equal(got, want[:t]) or t != 20
        assert torch.equal(got, mep.mep_w4_product(x[:t], w4, N))


@pytest.mark.parametrize("T,K,N", [(1, 7168, 256), (64, 7168, 200), (64, 2048, 40000), (5, 1001, 1407), (33, 257, 70000), (64, 40000, 8)])
def test_product_writes_nothing_behind_its_workspace(T, K, N):
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    w4 = mep.mep_w4_save(torch.randn(K, N, device="cuda"))
    need = mep.w4_product_workspace_bytes(T, K, N)
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = mep.mep_w4_product(x, w4, N, workspace=ws[:need], dtype=torch.float32)
    assert (ws[need:] == 0xA5).all()
    want, mag = ref.product(x, mep.mep_w4_load(w4, K, N, dtype=torch.float32))
    assert ((got.double() - want).abs() <= ref.product_bound(want, mag, K, 2.0 ** -24)).all()


def test_product_special_values():
    """A NaN or an infinity in one row or one column's group stays there; so does a group of zeros."""
    T, K, N = 11, 300, 100
    x = torch.randn(T, K, device="cuda")
    x[3, 7] = float("nan")
    x[5, 299] = float("inf")
    x = x.to(torch.bfloat16)
    w = torch.randn(K, N, device="cuda")
    w[:, 10] = 0
    w[17, 20] = float("nan")
    w[299, 30] = float("inf")
    w4 = mep.mep_w4_save(w, group=32)
    got = mep.mep_w4_product(x, w4, N, group=32).double()
    want = x.double() @ mep.mep_w4_load(w4, K, N, group=32, dtype=torch.float32).double()
    rows = [t for t in range(T) if t not in (3, 5)]
    cols = [n for n in range(N) if n not in (20, 30)]
    assert torch.isfinite(got[rows][:, cols]).all()
    assert torch.isnan(got[:, 20]).all() and torch.isnan(got[:, 30]).all() and torch.isnan(got[3]).all()
    assert not torch.isfinite(got[5]).any()
    keep = [n for n in cols if n != 10]
    assert torch.allclose(got[rows][:, keep], want[rows][:, keep], rtol=2.0 ** -7, atol=1e-3) and (got[rows][:, 10] == 0).all()


def test_product_rows_at_odd_addresses():
    T, K, N = 6, 77, 50
    base = torch.randn(10, K, device="cuda").to(torch.bfloat16)
    w4 = mep.mep_w4_save(torch.randn(K, N, device="cuda"))
    y = torch.full((10, N), -3.0, dtype=torch.bfloat16, device="cuda")
    mep.mep_w4_product(base[3:9], w4, N, y=y[1:7])
    assert torch.equal(y[1:7], mep.mep_w4_product(base[3:9].clone(), w4, N)) and (y[0] == -3).all() and (y[7:] == -3).all()


def test_product_status_streams_and_graph():
    T, K, N = 4, 512, 640
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    w4 = mep.mep_w4_save(torch.randn(K, N, device="cuda"))
    status = torch.full((1,), 4, dtype=torch.int32, device="cuda")
    y = torch.full((T, N), 5.0, dtype=torch.bfloat16, device="cuda")
    mep.mep_w4_product(x, w4, N, y=y, status=status)
    assert (y == 5).all() and int(status) == 4
    want = mep.mep_w4_product(x, w4, N)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([mep.mep_w4_product(x, w4, N) for _ in range(10)])
    torch.cuda.synchronize()
    assert all(torch.equal(v, want) for row in got for v in row)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mep.mep_w4_product(x, w4, N)
    for _ in range(3):
        x.copy_(torch.randn(T, K, device="cuda"))
        g.replay()
        assert torch.equal(out, mep.mep_w4_product(x, w4, N))


def test_no_rows():
    w4 = mep.mep_w4_save(torch.randn(64, 64, device="cuda"))
    assert mep.mep_w4_product(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w4, 64).shape == (0, 64)
    assert mep.mep_w4_save(torch.empty(0, 64, 64, device="cuda")).shape[0] == 0


def test_the_binding_refuses():
    x = torch.randn(2, 64, device="cuda").to(torch.bfloat16)
    w = torch.randn(64, 96, device="cuda")
    w4 = mep.mep_w4_save(w)
    for f in (lambda: mep.mep_w4_save(w, group=16), lambda: mep.mep_w4_save(w, parts=5), lambda: mep.mep_w4_save(w.t()),
              lambda: mep.mep_w4_save(w.half()), lambda: mep.mep_w4_save(w, w4=w4[:, :-1]), lambda: mep.mep_w4_load(w4, 64, 300),
              lambda: mep.mep_w4_load(w4, 64, 96, group=32), lambda: mep.mep_w4_load(w4, 64, 96, dtype=torch.float16),
              lambda: mep.mep_w4_product(x.float(), w4, 96), lambda: mep.mep_w4_product(x, w4, 300),
              lambda: mep.mep_w4_product(x, w4, 96, group=32), lambda: mep.mep_w4_product(x, w4, 96, dtype=torch.float16),
              lambda: mep.mep_w4_product(x.expand(2, 64).t(), w4, 96), lambda: mep.mep_w4_product(x.repeat(40, 1), w4, 96),
              lambda: mep.mep_w4_product(x, w4.cpu(), 96),
              lambda: mep.mep_w4_product(x, w4, 96, workspace=torch.empty(3, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((TypeError, ValueError, mep.MepError)):
            f()
