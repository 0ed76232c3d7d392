"""Routed tokens' rows on the GPU: sort, permute, combine and the gradients against ``oracle.moe_rows``, and a whole
routed W8A8 layer.

Tolerances, from the roundings: combine adds top_k FP32 products with one rounding each (top_k 2^-24 of the sum of the
terms' magnitudes) and rounds once to the output type; a dot product over H has at most H + 16 roundings on any path
(2^-24 each, of the sum of the magnitudes); dYs is one FP32 product rounded again to its type."""

import numpy as np
import pytest

from oracle import moe_rows, w8a8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "these tests need a CUDA device"
    return torch


@pytest.fixture(scope="module")
def lbq():
    import bit_weight_only_pack_b200 as lbq
    return lbq


def dtype(torch, name):
    return torch.float16 if name == "f16" else torch.bfloat16


def routing(rng, T, top_k, E, dropped=0.0):
    if top_k <= E:
        ids = np.argsort(rng.random((T, E)) ** rng.uniform(0.3, 3, size=(1, E)), axis=1)[:, :top_k].astype(np.int32)
    else:
        ids = rng.integers(0, E, size=(T, top_k), dtype=np.int32)
    if dropped:
        gone = rng.random(ids.shape) < dropped
        ids[gone] = rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], size=int(gone.sum()))
    return ids


def near(y, ref, tol):
    bad = ~(np.abs(y - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} values off, first at {np.argwhere(bad)[0]}"


def f64(t):
    return t.double().cpu().numpy()


def rounding(torch, ref, t):
    return np.abs(ref) * torch.finfo(t).eps / 2 + (2.0 ** -25 if t == torch.float16 else 0.0)


@pytest.mark.parametrize("T,top_k,E,dropped", [
    (1, 1, 1, 0), (1, 8, 256, 0), (1, 1, 1, 1.0), (16, 8, 256, 0), (37, 2, 8, 0.3), (300, 1, 3, 0), (333, 3, 2048, 0.1),
    (5, 4, 2, 0), (1024, 4, 3, 0), (1025, 4, 3, 0.01), (2000, 8, 64, 0), (2048, 8, 40, 0), (4097, 7, 16, 0.5), (12289, 8, 5, 0),
])
@pytest.mark.parametrize("cluster", [False, True])
def test_sort(torch, lbq, T, top_k, E, dropped, cluster):
    """Both kernels (the library takes the clustered one for many pairs)."""
    ids = routing(np.random.default_rng(T + E), T, top_k, E, dropped)
    lbq.lbq_debug_sort_cluster(cluster)
    try:
        got = [x.cpu().numpy() for x in lbq.moe_sort(torch.from_numpy(ids).cuda(), E)]
    finally:
        lbq.lbq_debug_sort_cluster(False)
    for a, b in zip(got, moe_rows.sort(ids, E)):
        assert np.array_equal(a, b)


def test_sort_with_every_pair_at_one_expert(torch, lbq):
    for e in (0, 3, 6):
        ids = torch.full((777, 4), e, dtype=torch.int32, device="cuda")
        row, pair, offsets = lbq.moe_sort(ids, 7)
        every = torch.arange(777 * 4, dtype=torch.int32, device="cuda")
        assert torch.equal(row.view(-1), every) and torch.equal(pair, every)
        assert offsets.tolist() == [0] * (e + 1) + [777 * 4] * (7 - e)


@pytest.mark.parametrize("name,H", [("float16", 1), ("bfloat16", 7), ("float16", 1003), ("bfloat16", 2048), ("int8", 48),
                                    ("int8", 33), ("int8", 64), ("int8", 65), ("int8", 79), ("int8", 1001), ("float16", 36),
                                    ("bfloat16", 4130), ("float32", 19), ("float64", 9), ("uint8", 2), ("float32", 1), ("float32", 6), ("float64", 5)])
@pytest.mark.parametrize("T,top_k,E,dropped", [(1, 3, 8, 0), (50, 2, 7, 0.4), (333, 8, 64, 0)])
def test_permute(torch, lbq, T, top_k, E, dropped, name, H):
    rng = np.random.default_rng(H + T)
    ids = routing(rng, T, top_k, E, dropped)
    row, _, _ = moe_rows.sort(ids, E)
    X = torch.from_numpy(rng.integers(-100, 100, size=(T, H))).to(getattr(torch, name))
    flat = torch.full((64 + T * top_k * H + 64,), 101, dtype=X.dtype, device="cuda")
    Xs = flat[64:64 + T * top_k * H].view(T * top_k, H)
    got = lbq.moe_permute(X.cuda(), torch.from_numpy(row).cuda(), Xs=Xs)
    assert got is Xs
    ref = moe_rows.permute(X.double().numpy(), row, np.full((T * top_k, H), 101.0))
    assert np.array_equal(f64(got), ref)
    assert bool((flat[:64] == 101).all()) and bool((flat[64 + T * top_k * H:] == 101).all())


def test_rows_past_the_buffers_are_skipped(torch, lbq):
    """Entries that name no row of the buffers they are used with: nothing outside is read or written."""
    row = torch.tensor([[0, 5], [9, -3], [2 ** 31 - 1, 1]], dtype=torch.int32, device="cuda")
    X = torch.arange(24, dtype=torch.float16, device="cuda").view(3, 8) + 1
    big = torch.zeros((9, 8), dtype=torch.float16, device="cuda")
    lbq.moe_permute(X, row, Xs=big[:6])
    assert torch.equal(big[[0, 5, 1]], X[[0, 0, 2]]) and bool((big[[2, 3, 4, 6, 7, 8]] == 0).all())
    w = torch.ones((3, 2), device="cuda")
    out = lbq.moe_combine(big[:6], row, w)
    assert torch.equal(out, torch.stack([2 * X[0], 0 * X[1], X[2]]))
    dY = torch.full((9, 8), 7.0, dtype=torch.float16, device="cuda")
    _, dw = lbq.moe_combine_grad(X, big[:6], row, w, dYs=dY[:6])
    assert bool((dY[[2, 3, 4, 6, 7, 8]] == 7).all())
    assert dw[1].tolist() == [0, 0] and dw[2, 0].item() == 0


def guarded(torch, rows, H, t):
    """An output between two stretches of sevens, and a check that those are as they were."""
    flat = torch.full((64 + rows * H + 64,), 7.0, dtype=t, device="cuda")

    def untouched():
        assert bool((flat[:64] == 7).all()) and bool((flat[64 + rows * H:] == 7).all())
    return flat[64:64 + rows * H].view(rows, H), untouched


CASES = [(1, 1, 1, 1, 0), (1, 8, 256, 2048, 0), (16, 8, 64, 512, 0.2), (333, 2, 8, 1003, 0), (40, 5, 7, 6, 0.5),
         (9, 13, 4, 100, 0), (64, 4, 16, 4100, 0), (3, 6, 8, 16384, 0), (500, 8, 32, 264, 0.05),
         (7, 3, 5, 31, 0.2), (7, 3, 5, 33, 0.2), (21, 4, 5, 34, 0), (33, 8, 16, 77, 0.3), (50, 5, 9, 1001, 0.1), (4, 2, 3, 2047, 0),
         (6, 9, 12, 2050, 0)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,top_k,E,H,dropped", CASES)
def test_combine_and_permute_grad(torch, lbq, T, top_k, E, H, dropped, dt):
    rng = np.random.default_rng(T + H)
    row, _, _ = moe_rows.sort(routing(rng, T, top_k, E, dropped), E)
    t = dtype(torch, dt)
    Y = torch.from_numpy(rng.standard_normal((T * top_k, H))).to(t)
    w = rng.random((T, top_k)).astype(np.float32)
    drow = torch.from_numpy(row).cuda()
    out, untouched = guarded(torch, T, H, t)
    dX, untouched2 = guarded(torch, T, H, t)
    for weights, got in ((w, lbq.moe_combine(Y.cuda(), drow, torch.from_numpy(w).cuda(), out=out)),
                         (None, lbq.moe_permute_grad(Y.cuda(), drow, dX=dX))):
        ref = moe_rows.combine(f64(Y), row, weights)
        size = moe_rows.combine(np.abs(f64(Y)), row, weights)
        fp32 = top_k * 2.0 ** -24 * size
        near(f64(got), ref, fp32 + rounding(torch, np.abs(ref) + fp32, t))
    untouched()
    untouched2()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,top_k,E,H,dropped", CASES)
def test_combine_grad(torch, lbq, T, top_k, E, H, dropped, dt):
    rng = np.random.default_rng(T + H + 1)
    row, _, _ = moe_rows.sort(routing(rng, T, top_k, E, dropped), E)
    t = dtype(torch, dt)
    Y = torch.from_numpy(rng.standard_normal((T * top_k, H))).to(t)
    dout = torch.from_numpy(rng.standard_normal((T, H))).to(t)
    w = rng.random((T, top_k)).astype(np.float32)
    dY, untouched = guarded(torch, T * top_k, H, t)
    dY.fill_(7.0)
    _, dw = lbq.moe_combine_grad(dout.cuda(), Y.cuda(), torch.from_numpy(row).cuda(), torch.from_numpy(w).cuda(), dYs=dY)
    rY, rw = moe_rows.combine_grad(f64(dout), f64(Y), row, w, np.full((T * top_k, H), 7.0))
    near(f64(dY), rY, np.abs(rY) * 2.0 ** -24 + rounding(torch, np.abs(rY) * (1 + 2.0 ** -24), t))
    _, size = moe_rows.combine_grad(np.abs(f64(dout)), np.abs(f64(Y)), row, w, np.zeros((T * top_k, H)))
    near(f64(dw), rw, (H + 16) * 2.0 ** -24 * size)
    untouched()


def test_gradients_against_differences(torch, lbq):
    """The loss <out, g> is linear in the rows and in the weights: a difference is the gradient up to roundings.
    Small whole numbers make every sum exact, so the two are equal."""
    rng = np.random.default_rng(0)
    T, top_k, E, H = 6, 3, 4, 24
    row = torch.from_numpy(moe_rows.sort(routing(rng, T, top_k, E), E)[0]).cuda()
    Y = torch.from_numpy(rng.integers(-3, 4, size=(T * top_k, H))).half().cuda()
    w = torch.from_numpy(rng.integers(1, 4, size=(T, top_k)).astype(np.float32)).cuda()
    g = torch.from_numpy(rng.integers(-3, 4, size=(T, H))).half().cuda()
    loss = lambda y, ww: float((lbq.moe_combine(y, row, ww).double() * g.double()).sum())  # noqa: E731
    dY, dw = lbq.moe_combine_grad(g, Y, row, w)
    base = loss(Y, w)
    for t, j in ((0, 0), (3, 2), (5, 1)):
        w2 = w.clone()
        w2[t, j] += 1
        assert loss(Y, w2) - base == dw[t, j].item()
    for r, h in ((0, 0), (7, 23), (17, 5)):
        Y2 = Y.clone()
        Y2[r, h] += 1
        assert loss(Y2, w) - base == dY[r, h].item()
    X = torch.from_numpy(rng.integers(-3, 4, size=(T, H))).half().cuda()
    ploss = lambda x: float((lbq.moe_permute(x, row).double() * Y.double()).sum())  # noqa: E731
    dX = lbq.moe_permute_grad(Y, row)
    X2 = X.clone()
    X2[4, 11] += 1
    assert ploss(X2) - ploss(X) == dX[4, 11].item()


@pytest.mark.parametrize("H", [520, 521, 7])
def test_combine_grad_in_place_and_repeatable(torch, lbq, H):
    rng = np.random.default_rng(2)
    T, top_k, E = 300, 8, 32
    row = torch.from_numpy(moe_rows.sort(routing(rng, T, top_k, E), E)[0]).cuda()
    Y = torch.randn((T * top_k, H), device="cuda").bfloat16()
    dout, w = torch.randn((T, H), device="cuda").bfloat16(), torch.rand((T, top_k), device="cuda")
    dY, dw = lbq.moe_combine_grad(dout, Y, row, w)
    again = lbq.moe_combine_grad(dout, Y, row, w)
    assert torch.equal(dY, again[0]) and torch.equal(dw, again[1])
    same, dw2 = lbq.moe_combine_grad(dout, Y, row, w, dYs=Y)
    assert same is Y and torch.equal(Y, dY) and torch.equal(dw2, dw)


@pytest.mark.parametrize("H", [2304, 2305])
def test_offsets_past_32_bits(torch, lbq, H):
    """Sorted rows of more than 2^31 elements: copied out, combined and their gradient, on sampled tokens."""
    g = torch.Generator(device="cuda").manual_seed(13)
    T, top_k, E = 131072, 8, 16
    ids = torch.randint(0, E, (T, top_k), generator=g, device="cuda", dtype=torch.int32)
    X = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    row, pair, offsets = lbq.moe_sort(ids, E)
    Xs = lbq.moe_permute(X, row)
    assert Xs.numel() > 2 ** 31
    at = torch.tensor([0, 1, 2 ** 31 // H - 1, 2 ** 31 // H, 2 ** 31 // H + 1, T * top_k - 1], device="cuda")
    assert torch.equal(Xs[at], X[pair[at].long() // top_k])
    w = torch.rand((T, top_k), generator=g, device="cuda")
    out = lbq.moe_combine(Xs, row, w)
    ts = [0, T // 3, T - 1] + [int(t) for t in (pair[at].long() // top_k)]
    # every copy of a token's row is the row itself: the combine is the row times the sum of its weights
    want = X[ts].double() * w[ts].double().sum(1, keepdim=True)
    size = X[ts].double().abs() * w[ts].double().abs().sum(1, keepdim=True)
    near(f64(out[ts]), f64(want), f64(size) * (top_k + 1) * 2.0 ** -24 + rounding(torch, f64(size), torch.bfloat16))
    dY, dw = lbq.moe_combine_grad(X, Xs, row, w, dYs=Xs)
    ref = X[pair[at].long() // top_k].double() * w.view(-1)[pair[at].long(), None].double()
    near(f64(dY[at]), f64(ref), np.abs(f64(ref)) * 2.0 ** -24 + rounding(torch, f64(ref) * (1 + 2.0 ** -24), torch.bfloat16))
    sq = X[ts].double().square().sum(1, keepdim=True).expand(-1, top_k)
    near(f64(dw[ts]), f64(sq), f64(sq) * (H + 16) * 2.0 ** -24)


def test_nan_and_infinity_stay_in_their_rows(torch, lbq):
    row = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    Y = torch.ones((4, 16), dtype=torch.bfloat16, device="cuda")
    Y[1, 3] = float("nan")
    Y[3, 0] = float("inf")
    out = lbq.moe_combine(Y, row, torch.ones((2, 2), device="cuda"))
    assert bool(torch.isnan(out[0, 3])) and int(torch.isnan(out).sum()) == 1
    assert bool(torch.isinf(out[1, 0])) and int(torch.isinf(out).sum()) == 1


@pytest.mark.parametrize("T", [1, 5, 150])
def test_routed_layer(torch, lbq, T):
    """Quantise, sort, copy codes and scales, gate/up product, gated activation, quantise, down product, combine; each
    step checked on the values that it was given, then the whole as a graph."""
    g = torch.Generator(device="cuda").manual_seed(T)
    top_k, E, H, I = 4, 16, 256, 136
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    top, ids = torch.randn((T, E), generator=g, device="cuda").topk(top_k, dim=1)
    ids, w = ids.to(torch.int32), torch.softmax(top, 1)
    w1, s1 = zip(*(lbq.quantize_int8_weight(torch.randn((H, 2 * I), generator=g, device="cuda") * 0.05) for _ in range(E)))
    w2, s2 = zip(*(lbq.quantize_int8_weight(torch.randn((I + 8, H), generator=g, device="cuda") * 0.05) for _ in range(E)))
    w1, s1, w2, s2 = (torch.stack(v) for v in (w1, s1, w2, s2))

    def layer(x, ids, w):
        xq, sx = lbq.quantize_int8_rows(x)
        row, pair, offsets = lbq.moe_sort(ids, E)
        rq, rs = lbq.moe_permute(xq, row), lbq.moe_permute(sx.view(-1, 1), row).view(-1)
        h = lbq.moe_w8a8_gemm(rq, rs, offsets, w1, s1)
        a = torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()
        a = torch.nn.functional.pad(a, (0, 8)).bfloat16()
        aq, sa = lbq.quantize_int8_rows(a)
        y = lbq.moe_w8a8_gemm(aq, sa, offsets, w2, s2)
        return rq, rs, offsets, h, aq, sa, y, row, lbq.moe_combine(y, row, w)

    rq, rs, offsets, h, aq, sa, y, row, out = layer(x, ids, w)
    lbq.device_status()
    n = lambda t: t.cpu().numpy()  # noqa: E731
    xq, sx = w8a8.quantize_rows(x.float().cpu().numpy())
    rrow, rpair, roff = moe_rows.sort(n(ids), E)
    assert np.array_equal(n(row), rrow) and np.array_equal(n(offsets), roff)
    assert np.array_equal(n(rq), xq[rpair // top_k]) and np.array_equal(n(rs), sx[rpair // top_k])
    u = 2.0 ** -8 + 4 * 2.0 ** -24
    ref = w8a8.routed_matmul(n(rq), n(rs), roff, n(w1), n(s1))
    near(f64(h), ref, np.abs(ref) * u)
    ref = w8a8.routed_matmul(n(aq), n(sa), roff, n(w2), n(s2))
    near(f64(y), ref, np.abs(ref) * u)
    ref, size = moe_rows.combine(f64(y), rrow, n(w)), moe_rows.combine(np.abs(f64(y)), rrow, n(w))
    near(f64(out), ref, top_k * 2.0 ** -24 * size * 2 + rounding(torch, np.abs(ref), torch.bfloat16))
    graph = torch.cuda.CUDAGraph()
    xi = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        got = layer(xi, ids, w)[-1]
    xi.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out)
