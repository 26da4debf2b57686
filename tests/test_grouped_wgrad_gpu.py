"""mep_grouped_wgrad against a plain 64-bit form.

* Integer rows (|x|, |dy| <= 2): every partial sum is an integer below 2^24,
  exact in fp32 in any order, and integers up to 2 are exact in 8 bits too:
  compared bit for bit.
* Normal rows: products of two bf16 are exact in fp32; each of the n additions
  of a sum over n rows is taken to be off by at most 2^-23 relatively (the
  tensor cores do not say how they round): n 2^-23 sum |x dy|.
"""

import numpy as np
import pytest
import torch

import load_balancing_topk_gb300 as mep
import train_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def _cu(sizes):
    return np.cumsum(np.asarray(sizes, np.int64), 1).astype(np.int32)


def _rows(n, C, seed, integer):
    g = torch.Generator().manual_seed(seed)
    if integer:
        return torch.randint(-2, 3, (n, C), generator=g).to(BF16)
    return torch.randn(n, C, generator=g).to(BF16)


def _case(cu, E, H, Hp, seed, integer, kept, accumulate=False, before=0.0):
    R, G = cu.shape
    SK, B = int(cu[0, -1]), G - E
    x, dy = _rows(R * SK, H, seed, integer), _rows(R * SK, Hp, seed + 1, integer)
    xd = x.to(DEV)
    xn = x.double().numpy()
    if kept:
        xd = mep.mep_ckpt_save(xd)
        xn = ref.kept(xn)
    home = torch.full((E, H, Hp), before, device=DEV)
    slot = torch.full((R, B, H, Hp), before, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mep.mep_grouped_wgrad(xd, dy.to(DEV), torch.from_numpy(cu).to(DEV), home, slot if B else None, status, R, SK, 1,
                          accumulate=accumulate)
    assert int(status.item()) == 0
    want = ref.wgrad(xn, dy.double().numpy(), cu, E)
    n = np.diff(np.concatenate([np.zeros((R, 1), np.int64), cu], 1), axis=1)
    nh, ns = n[:, :E].sum(0)[:, None, None], n[:, E:][:, :, None, None]
    add = before if accumulate else 0.0
    for got, w, mag, cnt, is_slot in ((home, want[0], want[2], nh, False), (slot, want[1], want[3], ns, True)):
        got = got.double().cpu().numpy()
        w = w + add
        if is_slot and not accumulate:
            w = np.where(cnt == 0, before, w)  # slots without rows are left alone
        tol = 0 if integer else (cnt * 2.0 ** -23 * mag + (np.abs(w) * 2.0 ** -23 if accumulate else 0))
        bad = ~(np.abs(got - w) <= tol)
        assert not bad.any(), f"{'slot' if is_slot else 'home'}: {bad.sum()} of {bad.size} off, first {np.argwhere(bad)[:4].tolist()}"


# E = 3, B = 2; group sizes [R, E + B]
TABLES = {
    "one_row": [[1, 0, 0, 0, 0]],
    "one_tile": [[64, 0, 0, 0, 0]],
    "under_and_over_a_step": [[15, 17, 63, 65, 1], [16, 33, 48, 0, 64]],
    "one_group_takes_all": [[0, 0, 300, 0, 0], [0, 0, 0, 300, 0]],
    "every_rank_has_rows_of_an_expert": [[40, 50, 10, 0, 3], [3, 97, 1, 2, 0], [0, 0, 100, 3, 0]],
    "long": [[700, 5, 295, 0, 24], [257, 255, 256, 256, 0]],
}
SIZES = [(64, 64), (128, 8), (8, 128), (136, 200), (256, 256), (264, 520)]


@pytest.mark.parametrize("kept", [False, True], ids=["as_it_was", "kept"])
@pytest.mark.parametrize("integer", [True, False], ids=["integer", "normal"])
@pytest.mark.parametrize("H,Hp", SIZES)
@pytest.mark.parametrize("table", list(TABLES))
def test_wgrad(table, H, Hp, integer, kept):
    _case(_cu(TABLES[table]), 3, H, Hp, H + Hp, integer, kept)


@pytest.mark.parametrize("kept", [False, True], ids=["as_it_was", "kept"])
@pytest.mark.parametrize("accumulate", [False, True], ids=["overwrite", "accumulate"])
@pytest.mark.parametrize("H,Hp", [(72, 136), (256, 384)])
def test_wgrad_over_what_is_there(H, Hp, accumulate, kept):
    """Home rows are overwritten even without rows, slots without rows are not; accumulate adds to both."""
    _case(_cu([[0, 70, 0, 0, 130], [90, 0, 0, 110, 0]]), 3, H, Hp, 3, True, kept, accumulate, before=7.0)


@pytest.mark.parametrize("seed", range(12))
def test_wgrad_random_tables(seed):
    rng = np.random.default_rng(seed)
    R, per, B = int(rng.integers(1, 5)), int(rng.integers(1, 4)), int(rng.integers(0, 4))
    E, SK = R * per, int(rng.integers(1, 900))
    cuts = np.sort(rng.integers(0, SK + 1, (R, E + B - 1)), 1)
    cu = np.concatenate([cuts, np.full((R, 1), SK)], 1).astype(np.int32)
    H, Hp = 8 * int(rng.integers(1, 60)), 8 * int(rng.integers(1, 60))
    _case(cu, E, H, Hp, seed, seed % 2 == 0, seed % 3 == 0)


@pytest.mark.parametrize("kept", [False, True], ids=["as_it_was", "kept"])
@pytest.mark.parametrize("sizes", [
    [[3000, 3, 0, 0, 40]],                                    # one group of 47 steps beside short ones
    [[0, 5000, 0, 0, 0], [0, 0, 700, 4300, 0]],               # three long ones, one of them of two parts' length
    [[17 * 64, 16 * 64, 64, 1, 17 * 64 + 1]],                 # at the shortest length that is cut, and beside it
    [[900, 100, 70, 130, 0], [950, 20, 30, 200, 0], [64, 0, 36, 1100, 0]],  # parts that begin inside a rank's rows
])
def test_wgrad_groups_in_parts(sizes, kept):
    _case(_cu(sizes), 3, 264, 136, 5, True, kept)
    _case(_cu(sizes), 3, 72, 520, 6, False, kept, accumulate=True, before=2.0)


def test_wgrad_more_weight_rows_than_a_block_of_threads():
    n = np.random.default_rng(0).integers(0, 3, (2, 1100))
    n[:, -1] += 3000 - n.sum(1)  # every rank has 3000 rows
    _case(_cu(n), 1090, 8, 16, 7, True, False)


def test_wgrad_wide():
    _case(_cu([[100, 28]]), 1, 7168, 72, 1, True, True)
    _case(_cu([[100, 28]]), 1, 72, 7168, 1, True, False)


@pytest.mark.parametrize("kept", [False, True], ids=["as_it_was", "kept"])
@pytest.mark.parametrize("rows,H,Hp", [
    (30000, 264, 136),   # one group in eight parts of 59 steps: from 8 bits every part empties its one accumulator twice
    (13000, 1160, 520),  # eight parts of 26 steps over 15 tiles
    (5000, 2048, 2560),  # 80 tiles, more than there are pairs: one part of 79 steps
])
def test_wgrad_of_more_steps_than_an_accumulator_takes(rows, H, Hp, kept):
    """Integers, bit for bit. (Sums of 30000 products of at most 4 stay below 2^24, so that the fp32 product compared
    with is exact as well.)"""
    x, dy = _rows(rows + 70, H, 1, True).to(DEV), _rows(rows + 70, Hp, 2, True).to(DEV)
    cu = torch.tensor([[30, 30 + rows, rows + 70]], dtype=torch.int32, device=DEV)
    home, slot = torch.zeros(2, H, Hp, device=DEV), torch.zeros(1, 1, H, Hp, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mep.mep_grouped_wgrad(mep.mep_ckpt_save(x) if kept else x, dy, cu, home, slot, status, 1, rows + 70, 1)
    assert int(status.item()) == 0
    for got, a, b in ((home[0], 0, 30), (home[1], 30, 30 + rows), (slot[0, 0], 30 + rows, rows + 70)):
        assert torch.equal(got, x[a:b].float().t() @ dy[a:b].float())


@pytest.mark.parametrize("kept", [False, True], ids=["as_it_was", "kept"])
def test_wgrad_sums_leave_the_tensor_cores_in_time(kept):
    """2-norm error over 3000 rows in one part (80 tiles, so that nothing is cut).

    The tensor cores' additions, one for 16 rows, cut off up to an ulp: half of one on average, and an ulp is 0.72 * 2^-23
    of a value on average; a running sum of random terms has on average 2/3 of its last size. After n additions that is
    n * 2^-25 of the sum: 32 (512 rows) 0.95e-6, 188 (all of them) 5.6e-6. From 8 bits there are fewer bits to cut off."""
    rows, H, Hp = 3000, 2048, 2560
    x, dy = _rows(rows, H, 1, False).to(DEV), _rows(rows, Hp, 2, False).to(DEV)
    cu = torch.tensor([[rows]], dtype=torch.int32, device=DEV)
    home = torch.zeros(1, H, Hp, device=DEV)
    ck = mep.mep_ckpt_save(x)
    mep.mep_grouped_wgrad(ck if kept else x, dy, cu, home, None, None, 1, rows, 1)
    want = (mep.mep_ckpt_load(ck, H) if kept else x).double().t() @ dy.double()
    assert float((home[0] - want).norm() / want.norm()) < 1e-6


def _room(nbytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 1.2 * nbytes:
        pytest.skip("not enough memory")


@pytest.mark.parametrize("kept", [False, True], ids=["as_it_was", "kept"])
def test_wgrad_of_more_than_2_31_elements(kept):
    """Two ranks of 150001 rows of 7168 columns (the second's rows lie beyond 2^31 bytes and elements), integers."""
    _room(8 << 30)
    R, S, E, H, Hp = 2, 150001, 2, 7168, 136
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.randint(-2, 3, (R * S, H), generator=g, device=DEV, dtype=torch.int8).to(BF16)
    dy = torch.randint(-2, 3, (R * S, Hp), generator=g, device=DEV, dtype=torch.int8).to(BF16)
    assert x.numel() > 2 ** 31
    ends = [[S - 70, S - 70, S], [100, S - 40, S]]
    cu = torch.tensor(ends, dtype=torch.int32, device=DEV)
    home, slot = torch.zeros(E, H, Hp, device=DEV), torch.zeros(R, 1, H, Hp, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mep.mep_grouped_wgrad(mep.mep_ckpt_save(x) if kept else x, dy, cu, home, slot, status, R, S, 1)
    assert int(status.item()) == 0

    def product(a, b):
        return x[a:b].float().t() @ dy[a:b].float()

    assert torch.equal(home[0], product(0, S - 70) + product(S, S + 100))
    assert torch.equal(home[1], product(S + 100, 2 * S - 40))
    assert torch.equal(slot[0, 0], product(S - 70, S)) and torch.equal(slot[1, 0], product(2 * S - 40, 2 * S))


def test_wgrad_gradients_of_more_than_2_31_elements():
    """The large workload's experts (256 of 7168 x 1408): the last ones' gradients lie beyond 2^31 elements."""
    E, H, Hp, SK = 256, 7168, 1408, 640
    _room(4 * E * H * Hp)
    home = torch.full((E, H, Hp), 7.0, device=DEV)
    assert home.numel() > 2 ** 31
    x, dy = _rows(2 * SK, H, 1, True).to(DEV), _rows(2 * SK, Hp, 2, True).to(DEV)
    n = torch.zeros(2, E, dtype=torch.int64)
    n[0, 0], n[0, 200], n[0, 254] = 300, 40, 300
    n[1, 1], n[1, 213], n[1, 255] = 17, 500, 123
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mep.mep_grouped_wgrad(x, dy, n.cumsum(1).int().to(DEV), home, None, status, 2, SK, 1)
    assert int(status.item()) == 0
    at = 0
    for e in range(E):  # (no expert has rows of both ranks)
        assert not n[0, e] or not n[1, e]
    for r in range(2):
        for e in n[r].nonzero().flatten().tolist():
            c = int(n[r, e])
            assert torch.equal(home[e], x[at:at + c].float().t() @ dy[at:at + c].float()), e
            at += c
    empty = (n.sum(0) == 0).nonzero().flatten()
    assert all(not home[e].any() for e in empty.tolist())


def test_wgrad_of_no_rows():
    home, slot = torch.full((2, 16, 8), 5.0, device=DEV), torch.full((1, 1, 16, 8), 5.0, device=DEV)
    cu = torch.zeros((1, 3), dtype=torch.int32, device=DEV)
    x, dy = torch.empty((0, 16), dtype=BF16, device=DEV), torch.empty((0, 8), dtype=BF16, device=DEV)
    mep.mep_grouped_wgrad(x, dy, cu, home, slot, None, 1, 0, 1)
    assert not home.any() and (slot == 5).all()


def test_wgrad_next_groups_rows_do_not_leak():
    """NaN and infinity in the rows right behind a group (inside its last tile) stay out of it."""
    cu = _cu([[70, 58, 0], [30, 0, 98]])
    R, E, SK, H, Hp = 2, 2, 128, 136, 72
    x, dy = _rows(R * SK, H, 1, True), _rows(R * SK, Hp, 2, True)
    want = ref.wgrad(x.double().numpy(), dy.double().numpy(), cu, E)
    for kept in (False, True):
        xb, db = x.clone(), dy.clone()
        xb[70:128], db[70:128] = float("nan"), float("inf")
        xb[SK + 30:], db[SK + 30:] = float("inf"), float("nan")
        home, slot = torch.zeros(E, H, Hp, device=DEV), torch.zeros(R, 1, H, Hp, device=DEV)
        xd = mep.mep_ckpt_save(xb.to(DEV)) if kept else xb.to(DEV)
        mep.mep_grouped_wgrad(xd, db.to(DEV), torch.from_numpy(cu).to(DEV), home, slot, None, R, SK, 1)
        assert (home[0].double().cpu().numpy() == want[0][0]).all()
        assert home[1].isnan().all() and slot[1, 0].isnan().all() and not slot[0].any()


def test_wgrad_rows_of_an_infinite_block_become_nan():
    cu = _cu([[64, 64]])
    x, dy = _rows(128, 256, 1, True), torch.ones(128, 64, dtype=BF16)
    x[70, 130] = float("inf")
    home, slot = torch.zeros(1, 256, 64, device=DEV), torch.zeros(1, 1, 256, 64, device=DEV)
    mep.mep_grouped_wgrad(mep.mep_ckpt_save(x.to(DEV)), dy.to(DEV), torch.from_numpy(cu).to(DEV), home, slot, None, 1, 128, 1)
    assert not home.isnan().any() and slot[0, 0, 128:].isnan().all() and not slot[0, 0, :128].isnan().any()


def test_wgrad_repeats_its_bits_on_another_stream_and_in_a_graph():
    cu = torch.from_numpy(_cu([[300, 20, 192], [100, 0, 412]])).to(DEV)
    x, dy = _rows(1024, 264, 1, False).to(DEV), _rows(1024, 328, 2, False).to(DEV)
    home, slot = torch.zeros(2, 264, 328, device=DEV), torch.zeros(2, 1, 264, 328, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        mep.mep_grouped_wgrad(x, dy, cu, home, slot, status, 2, 512, 1)

    step()
    want = home.clone(), slot.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        home.zero_()
        step()
    side.synchronize()
    assert torch.equal(home, want[0]) and torch.equal(slot, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    dy.mul_(2)
    graph.replay()
    assert torch.equal(home, 2 * want[0]) and torch.equal(slot, 2 * want[1]) and int(status.item()) == 0


def test_wgrad_gradient_against_differences():
    """The product is linear in the weights: the difference of the loss along a direction is exact but for the
    64-bit rounding, and the kernel's gradient is within its bound, here below n 2^-23 of the sum of magnitudes."""
    cu = _cu([[50, 31, 19]])
    x, dy = _rows(100, 64, 1, False), _rows(100, 40, 2, False)
    home, slot = torch.zeros(2, 64, 40, device=DEV), torch.zeros(1, 1, 64, 40, device=DEV)
    mep.mep_grouped_wgrad(x.to(DEV), dy.to(DEV), torch.from_numpy(cu).to(DEV), home, slot, None, 1, 100, 1)
    rng = np.random.default_rng(0)
    w, d = rng.normal(size=(3, 64, 40)), rng.normal(size=(3, 64, 40))
    xn, dn = x.double().numpy(), dy.double().numpy()

    def loss(w):
        return sum((xn[a:b] @ w[j] * dn[a:b]).sum() for j, (a, b) in enumerate([(0, 50), (50, 81), (81, 100)]))

    num = (loss(w + d) - loss(w - d)) / 2
    grad = np.concatenate([home.double().cpu().numpy(), slot[0].double().cpu().numpy()])
    mag = ref.wgrad(xn, dn, cu, 2)
    bound = 50 * 2.0 ** -23 * (np.concatenate([mag[2], mag[3][0]]) * np.abs(d)).sum()
    assert abs(num - (grad * d).sum()) <= bound + 1e-9 * np.abs(grad * d).sum()


@pytest.mark.parametrize("rows", [[[10, 5, 64]], [[10, 80, 64]], [[-1, 5, 64]], [[10, 20, 63]], [[10, 20, 65]]])
def test_wgrad_malformed_tables(rows):
    home, slot = torch.full((2, 16, 8), 5.0, device=DEV), torch.full((1, 1, 16, 8), 5.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    x, dy = torch.ones(64, 16, dtype=BF16, device=DEV), torch.ones(64, 8, dtype=BF16, device=DEV)
    cu = torch.tensor(rows, dtype=torch.int32, device=DEV)
    mep.mep_grouped_wgrad(x, dy, cu, home, slot, status, 1, 64, 1)
    assert int(status.item()) == mep.STATUS_CODE["MEP_ERR_BAD_SEQLENS"]
    assert (home == 5).all() and (slot == 5).all()
    # and an earlier step's error is obeyed
    cu = torch.tensor([[10, 20, 64]], dtype=torch.int32, device=DEV)
    mep.mep_grouped_wgrad(x, dy, cu, home, slot, status, 1, 64, 1)
    assert (home == 5).all() and int(status.item()) == mep.STATUS_CODE["MEP_ERR_BAD_SEQLENS"]


@pytest.mark.parametrize("E,B", [(3, 1), (2, 2), (1100, 0)], ids=["a_slot", "two_slots", "more_weight_rows_than_threads"])
def test_wgrad_malformed_tables_whose_differences_wrap(E, B):
    """Ends far apart: taken in 32 bits, every difference of this row is positive and its last end is S*K."""
    ends = [2 ** 31 - 1, -2 ** 31, -1, 64]
    differences = np.diff(np.array([0] + ends, np.int64)).astype(np.int32)
    assert (differences > 0).all()
    # (further groups without rows in front, where the table has more than four)
    cu = torch.tensor([[0] * (E + B - 4) + ends], dtype=torch.int32, device=DEV)
    home = torch.full((E, 16, 8), 5.0, device=DEV)
    slot = torch.full((1, B, 16, 8), 5.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    x, dy = torch.ones(64, 16, dtype=BF16, device=DEV), torch.ones(64, 8, dtype=BF16, device=DEV)
    mep.mep_grouped_wgrad(x, dy, cu, home, slot if B else None, status, 1, 64, 1)
    assert int(status.item()) == mep.STATUS_CODE["MEP_ERR_BAD_SEQLENS"]
    assert (home == 5).all() and (slot == 5).all()


def test_wgrad_refusals():
    x, dy = torch.ones(64, 16, dtype=BF16, device=DEV), torch.ones(64, 8, dtype=BF16, device=DEV)
    cu = torch.tensor([[10, 20, 64]], dtype=torch.int32, device=DEV)
    home, slot = torch.zeros(2, 16, 8, device=DEV), torch.zeros(1, 1, 16, 8, device=DEV)
    with pytest.raises(TypeError):
        mep.mep_grouped_wgrad(x.float(), dy, cu, home, slot, None, 1, 64, 1)
    with pytest.raises(TypeError):
        mep.mep_grouped_wgrad(x, dy, cu, home.bfloat16(), slot, None, 1, 64, 1)
    with pytest.raises(ValueError):
        mep.mep_grouped_wgrad(x, dy, cu, home, slot[:, :, :8], None, 1, 64, 1)
    with pytest.raises(ValueError):
        mep.mep_grouped_wgrad(x, dy, cu, home.view(2, 128), slot, None, 1, 64, 1)
    with pytest.raises(ValueError):
        mep.mep_grouped_wgrad(x, dy, cu, home, slot, None, 1, 65, 1)
    with pytest.raises(ValueError):                      # 8-bit rows of another width
        mep.mep_grouped_wgrad(x.view(torch.uint8), dy, cu, home, slot, None, 1, 64, 2)
    with pytest.raises(ValueError):
        mep.mep_grouped_wgrad(x, dy, cu, home.cpu(), slot, None, 1, 64, 1)
    with pytest.raises(mep.MepError):                    # H' not a multiple of 8
        mep.mep_grouped_wgrad(x, dy[:, :4].contiguous(), cu, torch.zeros(2, 16, 4, device=DEV),
                              torch.zeros(1, 1, 16, 4, device=DEV), None, 1, 64, 1)
