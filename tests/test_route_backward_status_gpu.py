"""mep_route_backward and its status word: a bad index counts as -1 and every row is written all the same, however many
blocks start after the one that met it; a status that was set before the call leaves dlogits alone."""

import pytest
import torch

import load_balancing_topk_gb300 as mep

pytestmark = pytest.mark.gpu
BAD = mep.STATUS_CODE["MEP_ERR_BAD_ROUTING"]


def make(N, E, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx, w = mep.mep_route(torch.randn(N, E, generator=g, device="cuda"), K)
    return torch.randn(N, K, generator=g, device="cuda"), w, idx


def bad_places(N, where):
    return {"first": [0], "last": [N - 1], "spread": list(range(0, N, 997)), "head": list(range(2048))}[where]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("where", ["first", "last", "spread", "head"])
@pytest.mark.parametrize("N,E,K", [(65536, 256, 8), (16411, 4096, 4), (300007, 43, 3), (40000, 100, 40)])
def test_every_row_is_written(N, E, K, where, dtype):
    """Far more blocks than fit the GPU at once, the earliest of them done long before the last begin."""
    dw, w, idx = make(N, E, K, 1)
    rows = torch.tensor(bad_places(N, where), device="cuda")
    left_out = idx.clone()
    left_out[rows, 1] = -1
    want = mep.mep_route_backward(dw, w, left_out, E, dtype=dtype)
    for n, value in enumerate((E, -2, 1 << 30, -(1 << 31), E)):
        bad = idx.clone()
        bad[rows, 1] = value
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = torch.full((N, E), float("nan"), dtype=dtype, device="cuda")
        mep.mep_route_backward(dw, w, bad, E, dlogits=got, status=status)
        assert int(status) == BAD, n
        assert torch.equal(got, want), (n, int((got != want).any(1).sum()))


def test_a_status_that_stands_is_kept():
    dw, w, idx = make(65536, 256, 8, 2)
    idx[5, 1] = 256
    for code in (BAD, mep.STATUS_CODE["MEP_ERR_TIMEOUT"], -BAD, -1, 1 << 30):
        status = torch.full((1,), code, dtype=torch.int32, device="cuda")
        keep = torch.full((65536, 256), 9.0, device="cuda")
        mep.mep_route_backward(dw, w, idx, 256, dlogits=keep, status=status)
        assert int(status) == code and bool((keep == 9).all())


def test_in_a_graph_and_for_the_next_step_on_the_stream():
    """Bad, good and bad again, replayed; what runs next on the stream finds the code and does nothing."""
    N, E, K = 65536, 64, 6
    dw, w, idx = make(N, E, K, 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mep.mep_route_backward(dw, w, idx, E, status=status)
    graph = torch.cuda.CUDAGraph()
    second = torch.zeros(N, E, device="cuda")
    with torch.cuda.graph(graph):
        first = mep.mep_route_backward(dw, w, idx, E, status=status)
        mep.mep_route_backward(dw, w, idx, E, dlogits=second, status=status)
    good = idx.clone()
    left_out = idx.clone()
    left_out[3, 2] = -1
    for bad in (True, False, True, True, False):
        idx.copy_(good)
        if bad:
            idx[3, 2] = E
        status.zero_()
        first.fill_(float("nan"))
        second.fill_(7.0)
        graph.replay()
        want = mep.mep_route_backward(dw, w, left_out if bad else good, E)
        assert int(status) == (BAD if bad else 0) and torch.equal(first, want)
        assert bool((second == 7).all()) if bad else torch.equal(second, want)


def test_streams_with_a_word_each():
    calls = [make(30000, 128, 4, s) for s in (4, 5, 6)]
    calls[1][2][7, 0] = -5
    words = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in calls]
    want = [mep.mep_route_backward(*c[:2], c[2].masked_fill(c[2] < 0, -1), 128) for c in calls]
    torch.cuda.synchronize()
    got, streams = [], [torch.cuda.Stream() for _ in calls]
    for s, c, word in zip(streams, calls, words):
        with torch.cuda.stream(s):
            got.append(mep.mep_route_backward(*c, 128, status=word))
    torch.cuda.synchronize()
    assert [int(v) for v in words] == [0, BAD, 0]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_row_and_none():
    for N in (1, 3, 5):
        dw, w, idx = make(N, 9, 2, 7)
        idx[0, 0] = 9
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = mep.mep_route_backward(dw, w, idx, 9, status=status)
        assert int(status) == BAD and torch.equal(got, mep.mep_route_backward(dw, w, idx.masked_fill(idx > 8, -1), 9))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw, w, idx = make(4, 9, 2, 8)
    assert mep.mep_route_backward(dw[:0], w[:0], idx[:0], 9, status=status).shape == (0, 9) and int(status) == 0
