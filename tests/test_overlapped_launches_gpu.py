"""Launches that overlap (LBQ_OPT_PDL): buffers that are written and read again and again, against the same calls one
after another. Equality, bit for bit: the kernels and their orders are the same."""

import pytest

import workloads

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


def overlapped(lbq, run):
    lbq.lbq_set_option(lbq.LBQ_OPT_PDL, 1)
    try:
        return run()
    finally:
        lbq.lbq_set_option(lbq.LBQ_OPT_PDL, 0)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 12, 40, 300, 700])
def test_w8a8_with_two_buffers_in_turn(torch, lbq, M):
    """One layer writes buffer i mod 2, the next reads it, on new values every time: a reader that saw what lay there
    before, or read too early, would differ. (700 rows of 1024 take the quantiser's warp form, 5 and more the tensor
    cores, 3 and 4 the CUDA-core product of codes, 1 and 2 the one that quantises.)"""
    g = torch.Generator(device="cuda").manual_seed(M)
    K, n = 1024, 24
    w1, w2 = (lbq.quantize_int8_weight(torch.randn((K, N), generator=g, device="cuda") * 0.03) for N in (K, 520))
    xs = [torch.randn((M, K), generator=g, device="cuda").bfloat16() for _ in range(n)]
    buf = [torch.zeros((M, K), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = [torch.empty(max(16, lbq.lbq_w8a8_workspace_size(M, K)), dtype=torch.uint8, device="cuda") for _ in range(2)]

    def run(outs):
        for i in range(n):
            lbq.w8a8_linear(xs[i], *w1, ws=ws[0], Y=buf[i % 2])
            lbq.w8a8_linear(buf[i % 2], *w2, ws=ws[1], Y=outs[i])
        torch.cuda.synchronize()
        return outs

    want = run([torch.empty((M, 520), dtype=torch.bfloat16, device="cuda") for _ in range(n)])
    got = [torch.empty_like(y) for y in want]
    for _ in range(3):
        overlapped(lbq, lambda: run(got))
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    lbq.device_status()


@pytest.mark.parametrize("T,cluster", [(1, False), (9, False), (150, False), (150, True), (900, True)])
def test_routed_chain(torch, lbq, T, cluster):
    """Sort, copy, quantise, routed products, combine and the gradients, each on what the one before wrote, in the same
    buffers every round and with other routings and inputs each time; then captured once and replayed."""
    g = torch.Generator(device="cuda").manual_seed(T)
    top_k, E, H, I, n = 4, 16, 512, 144, 8
    w1, s1 = (torch.randint(-127, 128, (E, I, H), generator=g, device="cuda", dtype=torch.int8),
              torch.rand((E, I), generator=g, device="cuda") * 1e-3)
    w2, s2 = (torch.randint(-127, 128, (E, H, I), generator=g, device="cuda", dtype=torch.int8),
              torch.rand((E, H), generator=g, device="cuda") * 1e-3)
    ins = []
    for _ in range(n):
        top, ids = torch.randn((T, E), generator=g, device="cuda").topk(top_k, dim=1)
        ids = ids.int()
        ids[torch.rand((T, top_k), generator=g, device="cuda") < 0.1] = -1
        x, d = (torch.randn((T, H), generator=g, device="cuda").bfloat16() for _ in range(2))
        ins.append((ids, torch.softmax(top, 1), x, d))
    P, bf = T * top_k, torch.bfloat16
    # (buffers start as zeros: rows in no run keep what an earlier round left, the same on both sides)
    new = lambda rows, cols: torch.zeros((rows, cols), dtype=bf, device="cuda")  # noqa: E731

    def buffers():
        return [new(P, H), new(P, I), new(P, H), new(T, H), new(P, H), new(T, H)]

    def layer(v, b):
        ids, w, x, d = v
        Xs, h, y, out, dy, dx = b
        row, pair, offsets = lbq.moe_sort(ids, E)
        lbq.moe_permute(x, row, Xs=Xs)
        lbq.moe_w8a8_gemm(*lbq.quantize_int8_rows(Xs), offsets, w1, s1, Y=h)
        lbq.moe_w8a8_gemm(*lbq.quantize_int8_rows(h), offsets, w2, s2, Y=y)
        lbq.moe_combine(y, row, w, out=out)
        _, dw = lbq.moe_combine_grad(d, y, row, w, dYs=dy)
        lbq.moe_permute_grad(dy, row, dX=dx)
        return row, pair, offsets, dw

    def run():
        b, kept = buffers(), []
        torch.cuda.synchronize()
        for v in ins:
            kept.append([*layer(v, b), *(t.clone() for t in b)])
        torch.cuda.synchronize()
        return kept

    lbq.lbq_debug_sort_cluster(cluster)
    try:
        want = run()
        for _ in range(3):
            for a, b in zip(want, overlapped(lbq, run)):
                assert all(torch.equal(s, t) for s, t in zip(a, b))
        # captured with overlapping launches, replayed on each round's inputs in the same buffers
        b, held = buffers(), [t.clone() for t in ins[0]]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()

        def capture():
            with torch.cuda.graph(graph, stream=side):
                return layer(held, b)

        got = overlapped(lbq, capture)
        for v, a in zip(ins, want):
            for t, s in zip(held, v):
                t.copy_(s)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(s, t) for s, t in zip(a, [*got, *b]))
    finally:
        lbq.lbq_debug_sort_cluster(False)
    lbq.device_status()


# (name, batch, the test hook's kernel choice)
GEMVS = [*(("int4", 1, path) for path in (0, 1, 4, 5)), ("int4", 4, 2), ("int4", 4, 3), ("int4", 1, "registers"),
         ("lut3", 1, 0), ("lut3", 1, 4), ("lut3", 4, 0), ("lut3", 16, 0), ("lut3", 4, 2), ("affine", 1, 0),
         ("affine", 4, 0), ("w4a8", 1, 0), ("w4a8", 1, "tiled"), ("w4a8", 4, 0)]


@pytest.mark.parametrize("name,M,path", GEMVS)
def test_gemvs_with_two_buffers_in_turn(torch, lbq, name, M, path):
    """The low-bit GEMVs, as the W8A8 layers above (W4A8 with its quantiser between)."""
    K, N, n = 1024, 1032, 24
    g = torch.Generator(device="cuda").manual_seed(M)
    dt = torch.bfloat16 if name == "lut3" else torch.float16
    if name == "lut3":
        pack = lambda seed, k, m: lbq.pack_lut3(*(torch.from_numpy(v).cuda() for v in workloads.lut3_host(seed, k, m)))  # noqa: E731
        call = lambda x, img, m, ws, y: lbq.lut3_gemm(x, img, m, ws=ws, Y=y)  # noqa: E731
        space = lambda k, m: lbq.workspace(2, M, k, m, 0, "lut3")  # noqa: E731
    elif name == "affine":
        pack = lambda seed, k, m: lbq.pack_affine(torch.from_numpy(workloads.weights_host(seed, k, m)).cuda(), 64, 3)  # noqa: E731
        call = lambda x, img, m, ws, y: lbq.affine_gemv(x, img, m, 64, 3, Y=y)  # noqa: E731
        space = lambda k, m: None  # noqa: E731
    else:
        pack = lambda seed, k, m: lbq.pack(torch.from_numpy(workloads.weights_host(seed, k, m)).cuda(), 32, "asym")  # noqa: E731
        if name == "int4":
            call = lambda x, img, m, ws, y: lbq.gemv(x, img, m, 32, "asym", ws=ws, Y=y)  # noqa: E731
            space = lambda k, m: lbq.workspace(0, M, k, m, 32, "asym")  # noqa: E731
        else:
            call = lambda x, img, m, ws, y: lbq.w4a8_gemv(*lbq.quantize_int8(x), img, m, 32, "asym", Y=y)  # noqa: E731
            space = lambda k, m: None  # noqa: E731
    images = pack(1, K, K), pack(2, K, N)
    xs = [torch.randn((M, K), generator=g, device="cuda").to(dt) for _ in range(n)]
    if isinstance(path, int):
        lbq.lbq_debug_gemv_path(path)
    elif path == "registers":
        lbq.lbq_debug_direct_variant(0)
    else:
        lbq.lbq_debug_w4a8_tiled(True)
    try:
        buf = [torch.zeros((M, K), dtype=dt, device="cuda") for _ in range(2)]
        ws = space(K, K), space(K, N)

        def run(outs):
            for i in range(n):
                call(xs[i], images[0], K, ws[0], buf[i % 2])
                call(buf[i % 2], images[1], N, ws[1], outs[i])
            torch.cuda.synchronize()
            return outs

        want = run([torch.empty((M, N), dtype=dt, device="cuda") for _ in range(n)])
        got = [torch.empty_like(y) for y in want]
        for _ in range(3):
            overlapped(lbq, lambda: run(got))
            assert all(torch.equal(a, b) for a, b in zip(want, got))
    finally:
        lbq.lbq_debug_gemv_path(0)
        lbq.lbq_debug_direct_variant(-1)
        lbq.lbq_debug_w4a8_tiled(False)
    lbq.device_status()
