"""moe_combine_grad without a buffer from the caller: the rows that no entry names have the gradient zero, whatever the
memory held before. (Tolerances as in test_moe_rows_gpu: an FP32 product rounded again to its type.)"""

import numpy as np
import pytest

from oracle import moe_rows

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


def dirty(torch, rows, H, t):
    """Leave NaN in the memory that the allocator hands out next."""
    torch.cuda.synchronize()
    for _ in range(3):
        x = torch.full((rows, H), float("nan"), dtype=t, device="cuda")
        del x


def check(torch, lbq, row, rows, H, t, seed):
    rng = np.random.default_rng(seed)
    T, top_k = row.shape
    Y = torch.from_numpy(rng.standard_normal((rows, H))).to(t)
    dout = torch.from_numpy(rng.standard_normal((T, H))).to(t)
    w = rng.random((T, top_k)).astype(np.float32)
    args = dout.cuda(), Y.cuda(), torch.from_numpy(row).cuda(), torch.from_numpy(w).cuda()
    dirty(torch, rows, H, t)
    dY, dw = lbq.moe_combine_grad(*args)
    f64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    ref, rw = moe_rows.combine_grad(f64(dout), f64(Y), row, w, np.zeros((rows, H)))
    half = np.abs(ref) * (1 + 2.0 ** -24) * torch.finfo(t).eps / 2 + (2.0 ** -25 if t == torch.float16 else 0.0)
    got = f64(dY)
    assert (np.abs(got - ref) <= np.where(ref == 0, 0, np.abs(ref) * 2.0 ** -24 + half)).all()
    named = np.zeros(rows, dtype=bool)
    named[row[(row >= 0) & (row < rows)]] = True
    assert not got[~named].any()
    # the same as into zeros of the caller's
    again, dw2 = lbq.moe_combine_grad(*args, dYs=torch.zeros((rows, H), dtype=t, device="cuda"))
    assert torch.equal(dY, again) and torch.equal(dw, dw2)
    return f64(dw), rw


@pytest.mark.parametrize("dt", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,top_k,E,H,dropped", [
    (1, 1, 1, 8, 1.0), (1, 8, 16, 2048, 0.5), (5, 3, 4, 1, 0.4), (40, 5, 7, 7, 0.5), (64, 4, 16, 4100, 0.3), (300, 8, 32, 264, 0.05),
    (333, 2, 8, 1003, 0.2), (256, 4, 64, 1024, 0), (1500, 8, 8, 64, 0.7), (2000, 6, 5, 33, 0.1), (700, 8, 20, 520, 1.0),
])
def test_dropped_pairs(torch, lbq, T, top_k, E, H, dropped, dt):
    rng = np.random.default_rng(T + H)
    ids = rng.integers(0, E, size=(T, top_k), dtype=np.int32)
    ids[rng.random(ids.shape) < dropped] = -1
    check(torch, lbq, moe_rows.sort(ids, E)[0], T * top_k, H, getattr(torch, dt), T)


@pytest.mark.parametrize("H", [40, 1024])
@pytest.mark.parametrize("rows", [50, 96, 97, 5000])
def test_rows_named_in_any_order(torch, lbq, rows, H):
    """More rows than pairs and fewer, named out of order, some entries outside the rows."""
    rng = np.random.default_rng(rows)
    row = rng.permutation(max(rows + 20, 96))[:96].reshape(32, 3).astype(np.int32)
    row[3, 1], row[7, 0] = -5, 2 ** 31 - 1
    check(torch, lbq, row, rows, H, torch.bfloat16, rows)


@pytest.mark.parametrize("T,H", [(160000, 16), (160000, 7), (20000, 1024), (20000, 1001), (20000, 512), (20000, 136)])
def test_many_rows(torch, lbq, T, H):
    """Sampled on the device: half of the pairs dropped, rows beyond what one pass of the zeroing blocks takes too."""
    g = torch.Generator(device="cuda").manual_seed(T)
    top_k, E = 8, 16
    ids = torch.randint(0, 2 * E, (T, top_k), generator=g, device="cuda", dtype=torch.int32)
    row, pair, offsets = lbq.moe_sort(ids, E)
    Y = torch.randn((T * top_k, H), generator=g, device="cuda").half()
    dout, w = torch.randn((T, H), generator=g, device="cuda").half(), torch.rand((T, top_k), generator=g, device="cuda")
    dirty(torch, T * top_k, H, torch.float16)
    dY, dw = lbq.moe_combine_grad(dout, Y, row, w)
    n = int(offsets[-1])
    assert 0 < n < T * top_k and not bool(dY[n:].any())
    want, dw2 = lbq.moe_combine_grad(dout, Y, row, w, dYs=torch.zeros_like(Y))
    assert torch.equal(dY, want) and torch.equal(dw, dw2)


@pytest.mark.parametrize("overlap", [0, 1])
@pytest.mark.parametrize("T,H", [(90, 256), (2000, 64)])
def test_in_a_graph(torch, lbq, T, H, overlap):
    """Captured and replayed with other routings: rows named before are zero once nothing names them. (Zeroed beside the
    tokens and before them; with overlapping launches too.)"""
    g = torch.Generator(device="cuda").manual_seed(3)
    top_k, E = 8, 8
    Y, dout = (torch.randn((n, H), generator=g, device="cuda").bfloat16() for n in (T * top_k, T))
    w = torch.rand((T, top_k), generator=g, device="cuda")
    row = lbq.moe_sort(torch.zeros((T, top_k), dtype=torch.int32, device="cuda"), E)[0]
    graph = torch.cuda.CUDAGraph()
    lbq.lbq_set_option(lbq.LBQ_OPT_PDL, overlap)
    try:
        with torch.cuda.graph(graph):
            lbq.moe_permute_grad(Y, row)
            dY, dw = lbq.moe_combine_grad(dout, Y, row, w)
            dX = lbq.moe_permute_grad(dY, row)
    finally:
        lbq.lbq_set_option(lbq.LBQ_OPT_PDL, 0)
    for keep in (E, 1, E // 2, 0):
        ids = torch.randint(0, E, (T, top_k), generator=g, device="cuda", dtype=torch.int32)
        row.copy_(lbq.moe_sort(torch.where(ids < keep, ids, -1), E)[0])
        graph.replay()
        torch.cuda.synchronize()
        want, dw2 = lbq.moe_combine_grad(dout, Y, row, w, dYs=torch.zeros_like(Y))
        assert torch.equal(dY, want) and torch.equal(dw, dw2) and torch.equal(dX, lbq.moe_permute_grad(want, row))
