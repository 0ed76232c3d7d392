"""Forms of the W8A8 kernels that the library picks by size: the row quantiser's warp form (many short rows), bit for
bit, and the routed product in every token tile, chosen by the library and forced.

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


@pytest.mark.parametrize("dt", ["float16", "bfloat16"])
@pytest.mark.parametrize("K", [16, 128, 256, 272, 512, 528, 1024, 1040, 2032, 2048, 2064, 4112])
@pytest.mark.parametrize("extra", [0, 1, 409])
def test_quantize_many_rows_is_bit_exact(torch, lbq, K, dt, extra):
    """Just enough rows for the warp form (up to 2048 columns), the last block of eight rows full and part-filled, and
    the block form's two lengths past it. Rows of zeros, ties, extremes, NaN and infinities among them; guards behind
    both outputs."""
    M = 4 * torch.cuda.get_device_properties(0).multi_processor_count + extra
    t = getattr(torch, dt)
    g = torch.Generator().manual_seed(K + extra)
    X = (torch.randn((M, K), generator=g) * torch.exp2(torch.randint(-12, 8, (M, 1), generator=g).float())).to(t)
    X[0] = 0
    X[7] = torch.where(torch.arange(K) % 2 == 0, 127.0, 0.5).to(t)          # scale 1, every other quotient a tie
    X[8, :] = torch.finfo(t).max
    X[9, :] = torch.finfo(t).smallest_normal
    X[10, K - 1] = float("nan")
    X[11, 0] = float("inf")
    X[12, K // 2] = float("-inf")
    X[13] = 0
    X[13, K - 1] = -1.0
    X[M - 1, K - 1] = 300.0                                                # the last row's largest in its last place
    xq = torch.full((M * K + 64,), 77, dtype=torch.int8, device="cuda")
    sx = torch.full((M + 64,), 77.0, device="cuda")
    lbq.lbq_quantize_int8_rows(X.cuda().data_ptr(), int(t is torch.bfloat16), M, K, xq.data_ptr(), sx.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
    rq, rs = w8a8.quantize_rows(X.float().numpy())
    assert np.array_equal(sx[:M].cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(xq[:M * K].view(M, K).cpu().numpy(), rq)
    assert bool((xq[M * K:] == 77).all()) and bool((sx[M:] == 77).all())


def ragged(rng, E, mean):
    """Runs of about `mean` rows, some empty, one of a single row."""
    counts = rng.integers(0, 2 * mean + 1, size=E)
    counts[E // 2] = 0
    counts[-1] = 1
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def check_routed(torch, lbq, offsets, K, N, t, seed):
    rng = np.random.default_rng(seed)
    rows, E = int(offsets[-1]), len(offsets) - 1
    xq, wq = (rng.integers(-128, 128, size=s, dtype=np.int8) for s in ((rows, K), (E, N, K)))
    sx, sw = (np.exp2(rng.uniform(-12, -8, size=s)).astype(np.float32) for s in (rows, (E, N)))
    flat = torch.full((64 + rows * N + 64,), 7.0, dtype=t, device="cuda")
    Y = flat[64:64 + rows * N].view(rows, N)
    lbq.moe_w8a8_gemm(*(torch.from_numpy(a).cuda() for a in (xq, sx, offsets, wq, sw)), Y=Y)
    torch.cuda.synchronize()
    lbq.device_status()
    ref = w8a8.routed_matmul(xq, sx, offsets, wq, sw)
    u = torch.finfo(t).eps / 2
    tol = np.abs(ref) * ((1 + u) * (1 + 2.0 ** -24) ** 3 - 1) + (2.0 ** -25 if t == torch.float16 else 0.0)
    bad = ~(np.abs(Y.double().cpu().numpy() - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, first at {np.argwhere(bad)[0]}"
    assert bool((flat[:64] == 7).all()) and bool((flat[64 + rows * N:] == 7).all())


@pytest.mark.parametrize("dt", ["float16", "bfloat16"])
@pytest.mark.parametrize("K,N", [(256, 200), (400, 131), (1040, 64)])
@pytest.mark.parametrize("mean", [2, 4, 6, 10, 12, 20, 40, 48, 60, 90, 130, 300])
def test_routed_token_tiles(torch, lbq, mean, K, N, dt):
    """Mean runs on both sides of each of the library's choices of tile."""
    rng = np.random.default_rng(mean + K)
    check_routed(torch, lbq, ragged(rng, 12, mean), K, N, getattr(torch, dt), mean)


@pytest.mark.parametrize("cg,bn", [(1, 16), (1, 32), (1, 64), (1, 128), (1, 256), (2, 32), (2, 64), (2, 128), (2, 256)])
@pytest.mark.parametrize("mean,K,N", [(3, 400, 131), (9, 1040, 300), (70, 256, 520), (200, 144, 257)])
def test_routed_forced_tiles(torch, lbq, cg, bn, mean, K, N):
    """Every token tile, alone and in pairs of blocks, on runs that the library would give another."""
    rng = np.random.default_rng(mean + bn)
    offsets = ragged(rng, 9, mean)
    lbq.lbq_debug_w8a8_plan(cg, -(-N // (128 * cg)) + 1, bn, 1)
    try:
        check_routed(torch, lbq, offsets, K, N, torch.bfloat16, bn)
    finally:
        lbq.lbq_debug_w8a8_plan(0)


@pytest.mark.parametrize("T", [37, 150, 400])
def test_routed_layer_steps(torch, lbq, T):
    """The second quantisation of a routed layer, on rows that a product wrote, against the oracle."""
    g = torch.Generator(device="cuda").manual_seed(T)
    top_k, E, H, I = 4, 16, 256, 144
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    ids = torch.randn((T, E), generator=g, device="cuda").topk(top_k, dim=1)[1].int()
    w1 = torch.randint(-127, 128, (E, I, H), generator=g, device="cuda", dtype=torch.int8)
    s1 = torch.rand((E, I), generator=g, device="cuda") * 1e-3
    row, _, offsets = lbq.moe_sort(ids, E)
    rq, rs = lbq.quantize_int8_rows(lbq.moe_permute(x, row))
    xq, sx = lbq.quantize_int8_rows(x)
    assert torch.equal(rq, lbq.moe_permute(xq, row)) and torch.equal(rs, lbq.moe_permute(sx.view(-1, 1), row).view(-1))
    h = lbq.moe_w8a8_gemm(rq, rs, offsets, w1, s1)
    hq, sh = lbq.quantize_int8_rows(h)
    q, s = w8a8.quantize_rows(h.float().cpu().numpy())
    assert np.array_equal(hq.cpu().numpy(), q) and np.array_equal(sh.cpu().numpy(), s)


@pytest.mark.parametrize("tensor", [False, True])
@pytest.mark.parametrize("K,N", [(16, 5000), (512, 4100), (1024, 8200), (1520, 4097), (1536, 8200), (2048, 100), (25600, 40), (25616, 40)])
def test_one_to_five_tokens(torch, lbq, K, N, tensor):
    """Both products on both sides of the library's choice between them; a row is the same in either and at any batch."""
    g = torch.Generator(device="cuda").manual_seed(K)
    wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randn((5, K), generator=g, device="cuda").bfloat16()
    sw = torch.exp2(torch.rand(N, generator=g, device="cuda") * 4 - 12)
    xq, sx = lbq.quantize_int8_rows(x)
    n = lambda t: t.cpu().numpy()  # noqa: E731
    ref = w8a8.matmul(n(xq), n(sx), n(wq), n(sw))
    lbq.lbq_debug_w8a8_gemv_max(0 if tensor else -1)
    try:
        for M in (1, 2, 3, 4, 5):
            y = lbq.w8a8_gemm(xq[:M], sx[:M], wq, sw)
            assert torch.equal(y, lbq.w8a8_linear(x[:M], wq, sw))
            tol = np.abs(ref[:M]) * ((1 + 2.0 ** -8) * (1 + 2.0 ** -24) ** 3 - 1)
            assert (np.abs(y.double().cpu().numpy() - ref[:M]) <= tol).all()
    finally:
        lbq.lbq_debug_w8a8_gemv_max(-1)
