"""W8A8 and routed rows without a GPU: refusals of the C ABI and of the Python helpers, and the oracles."""

import numpy as np
import pytest

from oracle import moe_rows, w8a8


@pytest.fixture(scope="module")
def lbq():
    import bit_weight_only_pack_b200 as lbq
    return lbq


P = 4096  # a 16-byte aligned address that is never read: every call below is refused on the host


def gemm(lbq, M=4, K=64, N=8, xq=P, sx=P, wq=P, sw=P, Y=P, dt=0):
    lbq.lbq_w8a8_gemm(xq, sx, M, K, N, wq, sw, Y, dt, None)


def linear(lbq, M=4, K=64, N=8, X=P, xdt=0, wq=P, sw=P, Y=P, dt=0, ws=P, ws_bytes=1 << 20):
    lbq.lbq_w8a8_linear(X, xdt, M, K, N, wq, sw, Y, dt, ws, ws_bytes, None)


def routed(lbq, rows=4, K=64, N=8, E=2, xq=P, sx=P, offsets=P, wq=P, sw=P, Y=P, dt=0):
    lbq.lbq_moe_w8a8_gemm(xq, sx, rows, K, N, offsets, E, wq, sw, Y, dt, None)


def quant(lbq, M=4, K=64, X=P, dt=0, xq=P, sx=P):
    lbq.lbq_quantize_int8_rows(X, dt, M, K, xq, sx, None)


def quant_w(lbq, K=64, N=8, W=P, wq=P, sw=P):
    lbq.lbq_quantize_int8_weight(W, K, N, wq, sw, None)


def sort(lbq, ids=P, pairs=8, E=4, row=P, pair=P, offsets=P):
    lbq.lbq_moe_sort(ids, pairs, E, row, pair, offsets, None)


def permute(lbq, X=P, row_bytes=32, T=4, top_k=2, row=P, rows=8, Xs=P):
    lbq.lbq_moe_permute(X, row_bytes, T, top_k, row, rows, Xs, None)


def combine(lbq, Ys=P, dt=0, rows=8, H=16, row=P, weights=P, T=4, top_k=2, out=P):
    lbq.lbq_moe_combine(Ys, dt, rows, H, row, weights, T, top_k, out, None)


def grad(lbq, dout=P, Ys=P, dt=0, rows=8, H=16, row=P, weights=P, T=4, top_k=2, dYs=P, dw=P):
    lbq.lbq_moe_combine_grad(dout, Ys, dt, rows, H, row, weights, T, top_k, dYs, dw, None)


BAD = [  # (call, arguments, status): 1 = invalid argument, 2 = unsupported
    *[(f, {k: v}, 1) for f, k in ((gemm, "M"), (gemm, "N"), (gemm, "K"), (linear, "M"), (routed, "rows"), (quant, "M"),
                                  (quant, "K"), (quant_w, "N"), (sort, "pairs"), (sort, "E"), (permute, "T"),
                                  (permute, "top_k"), (permute, "rows"), (permute, "row_bytes"), (combine, "T"),
                                  (combine, "H"), (combine, "rows"), (grad, "H"), (grad, "top_k"), (routed, "E"))
      for v in (0, -1)],
    *[(f, {"K": 72}, 1) for f in (gemm, linear, routed, quant, quant_w)],
    *[(f, {"K": 65552}, 2) for f in (gemm, linear, routed, quant, quant_w)],
    *[(f, {k: v}, 1) for f, ks in ((gemm, ("xq", "sx", "wq", "sw", "Y")), (linear, ("X", "wq", "sw", "Y", "ws")),
                                   (routed, ("xq", "sx", "offsets", "wq", "sw", "Y")), (quant, ("X", "xq", "sx")),
                                   (quant_w, ("W", "wq", "sw")), (sort, ("ids", "row", "pair", "offsets")),
                                   (permute, ("X", "row", "Xs")), (combine, ("Ys", "row", "out")),
                                   (grad, ("dout", "Ys", "row", "weights", "dYs", "dw")))
      for k in ks for v in (None, P + 8)],
    (combine, {"weights": P + 4}, 1),
    *[(f, {"dt": 2}, 2) for f in (gemm, linear, routed, quant, combine, grad)],
    (linear, {"xdt": 5}, 2),
    (linear, {"ws_bytes": 4 * 64}, 1),
    (routed, {"E": 2049}, 1), (sort, {"E": 2049}, 1), (sort, {"pairs": 1 << 30}, 1),
    (routed, {"E": 2048, "N": 1 << 21}, 1),
    *[(f, {k: 2 ** 31 - 1024}, 2) for f, k in ((gemm, "M"), (gemm, "N"), (linear, "N"), (routed, "rows"), (routed, "N"))],
    *[(f, {"T": 1 << 20, "top_k": 1 << 10}, 1) for f in (permute, combine, grad)],
]


@pytest.mark.parametrize("call,args,status", BAD)
def test_refusals_come_before_any_launch(lbq, call, args, status):
    before = lbq.lbq_launch_count()
    with pytest.raises(lbq.LbqError) as e:
        call(lbq, **args)
    assert e.value.status == status and lbq.lbq_last_error()
    assert lbq.lbq_launch_count() == before


def test_workspace_size(lbq):
    assert lbq.lbq_w8a8_workspace_size(1, 16) == lbq.lbq_w8a8_workspace_size(2, 8192) == 0
    for M, K in ((1, 16400), (3, 4096), (8192, 14336)):
        assert M * (K + 4) <= lbq.lbq_w8a8_workspace_size(M, K) <= M * (K + 4) + 512
    with pytest.raises(lbq.LbqError):
        lbq.lbq_w8a8_workspace_size(0, 16)


def test_helpers_refuse_host_tensors(lbq):
    import torch
    x, i8, f32, i32 = (torch.zeros((4, 64), dtype=t) for t in (torch.float16, torch.int8, torch.float32, torch.int32))
    for call in (lambda: lbq.quantize_int8_rows(x), lambda: lbq.w8a8_linear(x, i8, f32[0]),
                 lambda: lbq.w8a8_gemm(i8, f32[0], i8, f32[0]), lambda: lbq.moe_sort(i32, 4),
                 lambda: lbq.moe_permute(x, i32), lambda: lbq.moe_combine(x, i32), lambda: lbq.quantize_int8_weight(f32),
                 lambda: lbq.moe_combine_grad(x, x, i32, f32), lambda: lbq.moe_permute_grad(x, i32),
                 lambda: lbq.moe_w8a8_gemm(i8, f32[0], i32[0], i8, f32)):
        with pytest.raises(ValueError):
            call()


def test_every_shape_has_a_plan(lbq):
    """The dense plan (host code) covers all channels and tokens, in tiles that the kernel takes."""
    sizes = [1, 2, 3, 7, 8, 9, 15, 16, 17, 64, 100, 128, 129, 255, 256, 257, 500, 1003, 4096, 8192, 28672, 65537, 10 ** 6]
    for M in sizes + [2 ** 31 - 1]:
        for N in sizes:
            for K in (16, 128, 144, 4096, 65536):
                cg, ht, n_tiles, bn, m_tiles, splits, sub = lbq.lbq_debug_w8a8_planned(M, K, N)
                if M * N > 2 ** 40:
                    continue  # more tiles than one launch counts: refused
                assert cg in (1, 2) and 1 <= ht <= 128 and bn % (16 * cg) == 0 and 16 <= bn <= 256, (M, K, N)
                assert m_tiles * bn >= M > (m_tiles - 1) * bn and n_tiles * ht * cg >= N, (M, K, N)
                assert 1 <= sub <= max(1, K // 128) and splits in (1, 2, 4, 8), (M, K, N)


# ---------------------------------------------------------------------------- the oracles

def test_oracle_row_quantiser_by_hand():
    x = np.array([[127.0, 0.5, 1.5, -2.5], [0, 0, 0, 0], [254.0, -254.0, 3.0, 1.0]], dtype=np.float32)
    q, s = w8a8.quantize_rows(x)
    assert s.tolist() == [1.0, 0.0, 2.0]
    assert q.tolist() == [[127, 0, 2, -2], [0, 0, 0, 0], [127, -127, 2, 0]]
    q, s = w8a8.quantize_rows(np.array([[1, np.nan], [1, -np.inf]], dtype=np.float32))
    assert np.isnan(s[0]) and s[1] == np.inf and not q.any()


def test_oracle_product_is_the_integer_sum():
    rng = np.random.default_rng(0)
    xq = rng.integers(-128, 128, size=(3, 40), dtype=np.int8)
    wq = rng.integers(-128, 128, size=(5, 40), dtype=np.int8)
    want = [[sum(int(a) * int(b) for a, b in zip(x, w)) for w in wq] for x in xq]
    assert w8a8.integer_sums(xq, wq).tolist() == want


def test_oracle_rows_by_hand():
    ids = np.array([[1, 0], [1, -1], [0, 2]])
    row, pair, offsets = moe_rows.sort(ids, 3)
    assert row.tolist() == [[2, 0], [3, -1], [1, 4]]
    assert pair.tolist() == [1, 4, 0, 2, 5, -1] and offsets.tolist() == [0, 2, 4, 5]
    X = np.array([[1.0], [2.0], [3.0]])
    Xs = moe_rows.permute(X, row, np.full((6, 1), 9.0))
    assert Xs.ravel().tolist() == [1, 3, 1, 2, 3, 9]
    w = np.array([[2.0, 3.0], [5.0, 7.0], [1.0, 10.0]])
    assert moe_rows.combine(Xs, row, w).ravel().tolist() == [5, 10, 33]
    dY, dw = moe_rows.combine_grad(np.array([[1.0], [1.0], [2.0]]), Xs, row, w, np.zeros((6, 1)))
    assert dY.ravel().tolist() == [3, 2, 2, 5, 20, 0] and dw.tolist() == [[1, 1], [2, 0], [6, 6]]


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(1)
    ids = rng.integers(-1, 4, size=(5, 3))
    row, _, _ = moe_rows.sort(ids, 4)
    Y, w, g = rng.standard_normal((15, 6)), rng.random((5, 3)), rng.standard_normal((5, 6))
    dY, dw = moe_rows.combine_grad(g, Y, row, w, np.zeros_like(Y))
    h = 1e-6
    for idx in ((0, 0), (2, 1), (4, 2)):
        w2 = w.copy()
        w2[idx] += h
        assert abs(((moe_rows.combine(Y, row, w2) - moe_rows.combine(Y, row, w)) * g).sum() / h - dw[idx]) < 1e-8
    for idx in ((0, 0), (7, 5), (14, 3)):
        Y2 = Y.copy()
        Y2[idx] += h
        assert abs(((moe_rows.combine(Y2, row, w) - moe_rows.combine(Y, row, w)) * g).sum() / h - dY[idx]) < 1e-8
