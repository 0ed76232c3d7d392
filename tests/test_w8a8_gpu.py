"""W8A8 on the GPU: the quantisers bit for bit, the dense and the routed product against the exact integer sums.

Tolerance of a product, from the roundings it makes: the integer sum to FP32 (half a step, 2^-24 relative), two FP32
products (2^-24 each) and the output (half a step of its type, and for FP16 half its smallest step, 2^-25)."""

import numpy as np
import pytest

from oracle import w8a8

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


def codes(rng, shape):
    return rng.integers(-128, 128, size=shape, dtype=np.int8)


def scales(rng, n):
    return np.exp2(rng.uniform(-12, -8, size=n)).astype(np.float32)


def check(torch, Y, ref):
    y = Y.double().cpu().numpy()
    u = torch.finfo(Y.dtype).eps / 2
    tol = np.abs(ref) * ((1 + u) * (1 + 2.0 ** -24) ** 3 - 1) + (2.0 ** -25 if Y.dtype == torch.float16 else 0.0)
    bad = ~(np.abs(y - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, first at {np.argwhere(bad)[0]}"


def cuda(torch, *arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def guarded(torch, rows, N, dtype):
    """An output of `rows` rows between two guard rows, and a check that the guards are as they were. (The output
    starts 16-byte aligned: the guard in front is a whole number of 16-byte pieces.)"""
    front = 64
    flat = torch.full((front + rows * N + 64,), 7.0, dtype=dtype, device="cuda")

    def untouched():
        assert bool((flat[:front] == 7).all()) and bool((flat[front + rows * N:] == 7).all())
    return flat[front:front + rows * N].view(rows, N), untouched


def test_helpers_refuse_what_does_not_fit(torch, lbq):
    """Types, shapes, strides and outputs, before anything is launched."""
    z = lambda shape, t: torch.zeros(shape, dtype=t, device="cuda")  # noqa: E731
    f16, f32, i8, i32 = torch.float16, torch.float32, torch.int8, torch.int32
    x, xq, sx, wq, sw = z((4, 64), f16), z((4, 64), i8), z(4, f32), z((8, 64), i8), z(8, f32)
    rows, w, y = z((4, 2), i32), z((4, 2), f32), z((8, 64), f16)
    before = lbq.lbq_launch_count()
    for bad, call in [
        (TypeError, lambda: lbq.quantize_int8_rows(x.float())),
        (ValueError, lambda: lbq.quantize_int8_rows(x[0])),
        (ValueError, lambda: lbq.quantize_int8_rows(z((4, 128), f16)[:, ::2])),
        (TypeError, lambda: lbq.quantize_int8_weight(x)),
        (TypeError, lambda: lbq.w8a8_gemm(x, sx, wq, sw)),
        (TypeError, lambda: lbq.w8a8_gemm(xq, sx.double(), wq, sw)),
        (ValueError, lambda: lbq.w8a8_gemm(xq, sx[:3], wq, sw)),
        (ValueError, lambda: lbq.w8a8_gemm(xq, sx, z((8, 48), i8), sw)),
        (ValueError, lambda: lbq.w8a8_gemm(xq, sx, wq, sw, Y=z((4, 9), f16))),
        (TypeError, lambda: lbq.w8a8_gemm(xq, sx, wq, sw, Y=z((4, 8), f32))),
        (TypeError, lambda: lbq.w8a8_linear(x.float(), wq, sw)),
        (ValueError, lambda: lbq.w8a8_linear(x, wq.t(), sw)),
        (lbq.LbqError, lambda: lbq.w8a8_linear(x, wq, sw, ws=z(16, torch.uint8))),
        (lbq.LbqError, lambda: lbq.w8a8_gemm(xq.view(-1)[8:8 + 192].view(3, 64), sx[:3], wq, sw)),  # misaligned
        (ValueError, lambda: lbq.moe_w8a8_gemm(xq, sx, z(2, i32), z((2, 8, 64), i8), z((2, 8), f32))),
        (TypeError, lambda: lbq.moe_w8a8_gemm(xq, sx, z(3, torch.int64), z((2, 8, 64), i8), z((2, 8), f32))),
        (TypeError, lambda: lbq.moe_sort(rows.long(), 4)),
        (lbq.LbqError, lambda: lbq.moe_sort(rows, 0)),
        (ValueError, lambda: lbq.moe_permute(x, rows[:3])),
        (TypeError, lambda: lbq.moe_permute(x, rows, Xs=z((8, 64), torch.bfloat16))),
        (ValueError, lambda: lbq.moe_permute(x, rows, Xs=z((8, 63), f16))),
        (TypeError, lambda: lbq.moe_combine(y.float(), rows, w)),
        (ValueError, lambda: lbq.moe_combine(y, rows, w[:3])),
        (TypeError, lambda: lbq.moe_combine(y, rows, w.half())),
        (TypeError, lambda: lbq.moe_combine_grad(x.bfloat16(), y, rows, w)),
        (ValueError, lambda: lbq.moe_combine_grad(x[:3], y, rows, w)),
        (ValueError, lambda: lbq.moe_combine_grad(x, y, rows, w, dYs=y[:7])),
    ]:
        with pytest.raises(bad):
            call()
    assert lbq.lbq_launch_count() == before


# ---------------------------------------------------------------------------- quantisers

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (33, 256), (5, 4096), (2, 4112), (2, 14336), (1, 32768), (1, 65536)])
def test_quantize_rows_is_bit_exact(torch, lbq, M, K, dt):
    rng = np.random.default_rng(M * 7 + K)
    x = rng.standard_normal((M, K), dtype=np.float32) * np.exp2(rng.uniform(-6, 6, size=(M, 1))).astype(np.float32)
    if M > 2:
        x[1] = 0.0
        x[2] *= 2.0 ** -20  # FP16: subnormals
    X = torch.from_numpy(x).to(torch.float16 if dt == "f16" else torch.bfloat16)
    xq, sx = lbq.quantize_int8_rows(X.cuda())
    rq, rs = w8a8.quantize_rows(X.float().numpy())
    assert np.array_equal(sx.cpu().numpy(), rs)
    assert np.array_equal(xq.cpu().numpy(), rq)


def test_quantize_rows_of_the_smallest_and_largest_values(torch, lbq):
    """Scales whose reciprocal overflows (BF16 subnormals) and the largest finite values, bit for bit."""
    rng = np.random.default_rng(6)
    for top in (2.0 ** -133, 2.0 ** -130, 2.0 ** -126, 2.0 ** -120, 3.3e38):
        X = torch.from_numpy((rng.uniform(-1, 1, size=(6, 128)) * top).astype(np.float32)).bfloat16()
        xq, sx = lbq.quantize_int8_rows(X.cuda())
        rq, rs = w8a8.quantize_rows(X.float().numpy())
        assert np.array_equal(sx.cpu().numpy(), rs) and np.array_equal(xq.cpu().numpy(), rq), top


def test_quantize_rows_ties_go_to_even(torch, lbq):
    """amax 127 makes the scale exactly 1: every half-integer is a tie."""
    x = torch.arange(-127, 128).float() / 2  # -63.5 .. 63.5 in halves
    x = torch.cat([x, torch.tensor([127.0])]).view(1, 256)
    xq, sx = lbq.quantize_int8_rows(x.half().cuda())
    assert sx.item() == 1.0
    assert np.array_equal(xq.cpu().numpy(), np.rint(x.numpy()).astype(np.int8))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_rows_with_nan_or_infinity_have_nan_products(torch, lbq, dt):
    t = torch.float16 if dt == "f16" else torch.bfloat16
    x = torch.randn(4, 64).to(t)
    x[1, 5] = float("nan")
    x[2, 63] = float("-inf")
    xq, sx = lbq.quantize_int8_rows(x.cuda())
    s = sx.cpu().numpy()
    assert np.isnan(s[1]) and s[2] == np.inf and np.isfinite(s[[0, 3]]).all()
    assert bool((xq[1:3] == 0).all())
    wq = torch.ones((8, 64), dtype=torch.int8, device="cuda")
    y = lbq.w8a8_gemm(xq, sx, wq, torch.ones(8, device="cuda"))
    assert bool(torch.isnan(y[1:3]).all()) and bool(torch.isfinite(y[[0, 3]]).all())


@pytest.mark.parametrize("K,N", [(16, 1), (48, 33), (256, 100), (4112, 7)])
def test_quantize_weight_is_bit_exact(torch, lbq, K, N):
    rng = np.random.default_rng(K + N)
    W = (rng.standard_normal((K, N)) * 0.02).astype(np.float32)
    W[:, 0] = 0.0
    if N > 6:
        W[3, 5] = np.nan
        W[0, 6] = np.inf
    wq, sw = lbq.quantize_int8_weight(torch.from_numpy(W).cuda())
    rq, rs = w8a8.quantize_weight(W)
    assert np.array_equal(sw.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(wq.cpu().numpy(), rq)


# ---------------------------------------------------------------------------- dense product

SHAPES = [
    (1, 16, 1), (1, 4096, 1000), (2, 48, 7), (3, 2064, 90), (4, 128, 28), (5, 8208, 40), (8, 144, 129), (8, 14336, 70), (15, 256, 127), (16, 4112, 1003), (17, 2048, 300),
    (31, 512, 64), (33, 1024, 200), (64, 640, 513), (100, 400, 4099), (255, 128, 130), (256, 272, 257), (257, 384, 96),
    (300, 1040, 1003), (513, 256, 2000), (1000, 192, 77), (1025, 64, 3000),
]


@pytest.mark.parametrize("ydt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N,tensor", [(*s, False) for s in SHAPES] + [(*s, True) for s in SHAPES if s[0] <= 8])
def test_gemm_matches_the_integer_sums(torch, lbq, M, K, N, ydt, tensor):
    """The library's choice, and small batches on the tensor cores too."""
    lbq.lbq_debug_w8a8_gemv_max(0 if tensor else -1)
    try:
        check_gemm(torch, lbq, M, K, N, ydt)
    finally:
        lbq.lbq_debug_w8a8_gemv_max(-1)


def check_gemm(torch, lbq, M, K, N, ydt):
    rng = np.random.default_rng(M * 31 + K * 7 + N)
    xq, wq, sx, sw = codes(rng, (M, K)), codes(rng, (N, K)), scales(rng, M), scales(rng, N)
    t = torch.float16 if ydt == "f16" else torch.bfloat16
    Y, untouched = guarded(torch, M, N, t)
    dxq, dsx, dwq, dsw = cuda(torch, xq, sx, wq, sw)
    lbq.w8a8_gemm(dxq, dsx, dwq, dsw, Y=Y)
    torch.cuda.synchronize()
    lbq.device_status()
    check(torch, Y, w8a8.matmul(xq, sx, wq, sw))
    untouched()


@pytest.mark.parametrize("plan", [(1, 1, 16, 1), (1, 3, 32, 2), (1, 2, 16, 4), (1, 5, 128, 8), (1, 3, 48, 4), (1, 7, 256, 1),
                                  (2, 1, 32, 1), (2, 2, 96, 1), (2, 3, 256, 1)])
@pytest.mark.parametrize("M,K,N", [(5, 4096, 100), (40, 4112, 127), (77, 4224, 254), (130, 4096, 300), (300, 8192, 256)])
def test_gemm_plans(torch, lbq, M, K, N, plan):
    """Every form of the tensor-core kernel (pairs, shared K, token tiles that end inside) on shapes that the library
    would give another. Plans that a shape cannot take are refused."""
    cg, n_tiles, bn, splits = plan
    lbq.lbq_debug_w8a8_gemv_max(0)
    lbq.lbq_debug_w8a8_plan(cg, n_tiles, bn, splits)
    try:
        # too few channel tiles, or more tiles than clusters of `splits` blocks fit at once
        if n_tiles * cg * 128 < N or (splits > 1 and -(-M // bn) * n_tiles * splits > 148):
            with pytest.raises(lbq.LbqError):
                check_gemm(torch, lbq, M, K, N, "bf16")
        else:
            check_gemm(torch, lbq, M, K, N, "bf16")
            check_gemm(torch, lbq, M, K, N, "f16")
    finally:
        lbq.lbq_debug_w8a8_plan(0)
        lbq.lbq_debug_w8a8_gemv_max(-1)


@pytest.mark.parametrize("M", [1, 6, 20, 300])
def test_gemm_largest_sums_stay_exact(torch, lbq, M):
    """Every product at its largest, 2^14, over the longest K: 2^30."""
    K, N = 65536, 9
    xq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    wq[1] = 127
    sx, sw = torch.full((M,), 2.0 ** -20, device="cuda"), torch.ones(N, device="cuda")
    y = lbq.w8a8_gemm(xq, sx, wq, sw)
    ref = np.full((M, N), 2.0 ** 10)
    ref[:, 1] = -128.0 * 127 * K * 2.0 ** -20
    check(torch, y, ref)


@pytest.mark.parametrize("M,K,N", [(1, 4096, 4096), (16, 8192, 28672), (2048, 4096, 14336)])
def test_gemm_full_size_sampled(torch, lbq, M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M)
    xq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(M, generator=g, device="cuda") * 1e-2
    sw = torch.rand(N, generator=g, device="cuda") * 1e-2
    y = lbq.w8a8_gemm(xq, sx, wq, sw)
    rng = np.random.default_rng(M)
    rows = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 12)]))
    cols = np.unique(np.concatenate([[0, N - 1], rng.integers(0, N, 200)]))
    ref = w8a8.matmul(xq[rows].cpu().numpy(), sx[rows].cpu().numpy(), wq[cols].cpu().numpy(), sw[cols].cpu().numpy())
    check(torch, y[rows][:, cols], ref)
    assert torch.equal(y, lbq.w8a8_gemm(xq, sx, wq, sw))


def test_offsets_past_32_bits(torch, lbq):
    """Outputs of more than 2^31 elements and experts' weights of more than 2^32 bytes."""
    g = torch.Generator(device="cuda").manual_seed(12)
    M, K, N = 140000, 16, 16384
    xq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sx, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    y = lbq.w8a8_gemm(xq, sx, wq, sw)
    rows = torch.tensor([0, 1, 131071, 131072, 135000, M - 1], device="cuda")
    n = lambda t: t.cpu().numpy()  # noqa: E731
    check(torch, y[rows], w8a8.matmul(n(xq[rows]), n(sx[rows]), n(wq), n(sw)))
    del y, xq, wq
    E, K, N = 66, 8192, 8192
    wq = torch.randint(-127, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand((E, N), generator=g, device="cuda")
    xq = torch.randint(-127, 128, (E, K), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(E, generator=g, device="cuda")
    y = lbq.moe_w8a8_gemm(xq, sx, torch.arange(E + 1, dtype=torch.int32, device="cuda"), wq, sw)
    for e in (0, 31, 32, 63, 64, E - 1):
        check(torch, y[e:e + 1], w8a8.matmul(n(xq[e:e + 1]), n(sx[e:e + 1]), n(wq[e]), n(sw[e])))


def test_rows_do_not_depend_on_the_batch(torch, lbq):
    """Row m of a product is the same at every M (the sums are integers, the scaling is per element)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    xq = torch.randint(-127, 128, (700, 1024), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (555, 1024), generator=g, device="cuda", dtype=torch.int8)
    sx, sw = torch.rand(700, generator=g, device="cuda"), torch.rand(555, generator=g, device="cuda") * 1e-3
    y = lbq.w8a8_gemm(xq, sx, wq, sw)
    for M in (1, 3, 9, 40, 129, 300):
        assert torch.equal(y[:M], lbq.w8a8_gemm(xq[:M], sx[:M], wq, sw))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 1024), (1, 65536, 9), (2, 8192, 77), (2, 8208, 50), (3, 16, 5), (5, 1040, 333), (7, 14336, 256),
                                   (16, 64, 100), (200, 512, 130)])
def test_linear_is_the_two_calls(torch, lbq, M, K, N, dt):
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.float16 if dt == "f16" else torch.bfloat16)
    wq, sw = lbq.quantize_int8_weight(torch.randn((K, N), generator=g, device="cuda") * 0.02)
    xq, sx = lbq.quantize_int8_rows(x)
    y = lbq.w8a8_linear(x, wq, sw)
    assert y.dtype == x.dtype and torch.equal(y, lbq.w8a8_gemm(xq, sx, wq, sw, y_dtype=dt))


def test_linear_on_other_streams_and_in_graphs(torch, lbq):
    """A side stream, and two graphs with a workspace each, replayed on new inputs in both orders."""
    g = torch.Generator(device="cuda").manual_seed(3)
    wq, sw = lbq.quantize_int8_weight(torch.randn((2048, 600), generator=g, device="cuda") * 0.02)
    xs = [torch.randn((M, 2048), generator=g, device="cuda").half() for M in (1, 40)]
    want = [lbq.w8a8_linear(x, wq, sw) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [lbq.w8a8_linear(x, wq, sw) for x in xs]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, ins, outs = [], [], []
    for x in xs:
        xi = torch.zeros_like(x)
        ws = torch.empty(lbq.lbq_w8a8_workspace_size(*x.shape), dtype=torch.uint8, device="cuda")
        yo = torch.empty((x.shape[0], 600), dtype=x.dtype, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lbq.w8a8_linear(xi, wq, sw, ws=ws, Y=yo)
        graphs.append(graph), ins.append(xi), outs.append(yo)
    for order in ((0, 1), (1, 0)):
        for i in order:
            ins[i].copy_(xs[i])
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
    lbq.device_status()


def test_chain_with_programmatic_launches(torch, lbq):
    """Three layers back to back, each reading the last one's output, with overlapping launches allowed."""
    g = torch.Generator(device="cuda").manual_seed(4)
    ws = [lbq.quantize_int8_weight(torch.randn((1024, 1024), generator=g, device="cuda") * 0.03) for _ in range(3)]
    for M in (1, 12, 300):
        x = torch.randn((M, 1024), generator=g, device="cuda").bfloat16()
        want = x
        for wq, sw in ws:
            want = lbq.w8a8_linear(want, wq, sw)
        torch.cuda.synchronize()
        lbq.lbq_set_option(lbq.LBQ_OPT_PDL, 1)
        try:
            for _ in range(5):
                y = x
                for wq, sw in ws:
                    y = lbq.w8a8_linear(y, wq, sw)
                assert torch.equal(y, want)
        finally:
            lbq.lbq_set_option(lbq.LBQ_OPT_PDL, 0)


# ---------------------------------------------------------------------------- routed product

def runs(rng, E, rows, kind):
    if kind == "one":
        counts = np.zeros(E, dtype=np.int64)
        counts[E // 2] = rows
    elif kind == "even":
        counts = np.full(E, rows // E)
        counts[:rows - counts.sum()] += 1
    else:
        counts = rng.multinomial(rows, rng.dirichlet(np.full(E, 0.3)))
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


@pytest.mark.parametrize("ydt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,E,K,N,kind", [
    (1, 1, 16, 1, "even"), (1, 256, 128, 40, "one"), (8, 32, 2048, 1024, "uneven"), (128, 256, 256, 100, "uneven"),
    (100, 3, 144, 129, "uneven"), (300, 4, 512, 128, "one"), (700, 8, 400, 333, "uneven"), (900, 2, 128, 300, "even"),
    (513, 2048, 64, 24, "uneven"), (1500, 6, 256, 77, "uneven"),
])
def test_routed_product(torch, lbq, rows, E, K, N, kind, ydt):
    rng = np.random.default_rng(rows + E)
    offsets = runs(rng, E, rows, kind)
    xq, wq, sx, sw = codes(rng, (rows, K)), codes(rng, (E, N, K)), scales(rng, rows), scales(rng, (E, N))
    t = torch.float16 if ydt == "f16" else torch.bfloat16
    Y, untouched = guarded(torch, rows, N, t)
    dxq, dsx, doff, dwq, dsw = cuda(torch, xq, sx, offsets, wq, sw)
    lbq.moe_w8a8_gemm(dxq, dsx, doff, dwq, dsw, Y=Y)
    torch.cuda.synchronize()
    lbq.device_status()
    check(torch, Y, w8a8.routed_matmul(xq, sx, offsets, wq, sw))
    untouched()


def test_routed_rows_in_no_run_are_left(torch, lbq):
    """Rows before the first run and after the last one; all runs empty."""
    rng = np.random.default_rng(9)
    rows, E, K, N = 200, 5, 128, 72
    xq, wq, sx, sw = codes(rng, (rows, K)), codes(rng, (E, N, K)), scales(rng, rows), scales(rng, (E, N))
    dxq, dsx, dwq, dsw = cuda(torch, xq, sx, wq, sw)
    for offsets in ([3, 3, 20, 20, 21, 150], [0, 0, 0, 0, 0, 0], [200, 200, 200, 200, 200, 200]):
        off = np.array(offsets, dtype=np.int32)
        Y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
        lbq.moe_w8a8_gemm(dxq, dsx, cuda(torch, off)[0], dwq, dsw, Y=Y)
        ref = w8a8.routed_matmul(xq, sx, off, wq, sw)
        check(torch, Y, np.where(np.isnan(ref), 7.0, ref))


def test_routed_offsets_that_decrease_or_lie_outside(torch, lbq):
    """Whatever the array holds, rows stay inside and belong to one run: an offset counts as the largest before it."""
    rng = np.random.default_rng(10)
    rows, E, K, N = 90, 6, 64, 40
    xq, wq, sx, sw = codes(rng, (rows, K)), codes(rng, (E, N, K)), scales(rng, rows), scales(rng, (E, N))
    dxq, dsx, dwq, dsw = cuda(torch, xq, sx, wq, sw)
    for offsets in ([0, 20, 10, 30, 30, 90, 60], [-5, -2 ** 31, 7, 2 ** 31 - 1, 0, 91, 3], [89, 90, 0, 0, 0, 0, 0]):
        off = np.array(offsets, dtype=np.int64)
        Y, untouched = guarded(torch, rows, N, torch.bfloat16)
        Y.fill_(7.0)
        lbq.moe_w8a8_gemm(dxq, dsx, cuda(torch, off.astype(np.int32))[0], dwq, dsw, Y=Y)
        ref = w8a8.routed_matmul(xq, sx, np.maximum.accumulate(np.clip(off, 0, rows)), wq, sw)
        check(torch, Y, np.where(np.isnan(ref), 7.0, ref))
        untouched()


@pytest.mark.parametrize("plan", [(1, 2, 16, 1), (1, 2, 64, 4), (2, 1, 64, 1)])
def test_waits_run_out(torch, lbq, plan):
    """Copies that never come: the waits end, nothing is written, the flag is reported, and the next call is right."""
    rng = np.random.default_rng(11)
    M, K, N = 40, 4096, 200
    xq, wq, sx, sw = codes(rng, (M, K)), codes(rng, (N, K)), scales(rng, M), scales(rng, N)
    dxq, dsx, dwq, dsw = cuda(torch, xq, sx, wq, sw)
    Y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lbq.lbq_debug_w8a8_plan(*plan)
    try:
        lbq.lbq_debug_w8a8_hold(True)
        lbq.w8a8_gemm(dxq, dsx, dwq, dsw, Y=Y)
        lbq.lbq_debug_w8a8_hold(False)
        with pytest.raises(lbq.LbqError) as e:
            lbq.device_status()
        assert e.value.status == lbq.binding.LBQ_ERR_DEVICE
        assert bool((Y == 7).all())
        lbq.w8a8_gemm(dxq, dsx, dwq, dsw, Y=Y)
        lbq.device_status()
        check(torch, Y, w8a8.matmul(xq, sx, wq, sw))
    finally:
        lbq.lbq_debug_w8a8_hold(False)
        lbq.lbq_debug_w8a8_plan(0)


def test_routed_with_one_expert_is_the_dense_product(torch, lbq):
    g = torch.Generator(device="cuda").manual_seed(5)
    xq = torch.randint(-127, 128, (333, 512), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (1, 200, 512), generator=g, device="cuda", dtype=torch.int8)
    sx, sw = torch.rand(333, generator=g, device="cuda"), torch.rand((1, 200), generator=g, device="cuda") * 1e-3
    off = torch.tensor([0, 333], dtype=torch.int32, device="cuda")
    assert torch.equal(lbq.moe_w8a8_gemm(xq, sx, off, wq, sw), lbq.w8a8_gemm(xq, sx, wq[0], sw[0]))
