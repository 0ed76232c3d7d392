"""Operators of 8-bit and routed layers, in plain form and as the library's calls.

Five passes, named by a case's "op":

* ``linear``   -- W8A8 projection: every token's row of X is quantised to INT8 with one scale, multiplied with INT8
  weights that carry one scale per output channel, and scaled back.
* ``experts``  -- the same product on rows sorted by expert, each run of rows with its own expert's weights.
* ``dispatch`` -- the router's choices sorted by expert (stable), and every token's row copied to its places in that
  order.
* ``combine``  -- the experts' rows back in token order, weighted and summed over a token's choices.
* ``backward`` -- the gradients of the last two: of the experts' rows, of the router's weights and of the tokens.

``run`` computes a pass in elementary torch operations, or, where ``own`` is true, with the library's calls.
"""

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one token through a 4096 x 4096 projection: decode at batch 1, where latency counts
        dict(name="linear_decode_1", op="linear", M=1, K=4096, N=4096, dtype="f16"),
        # a decode batch through the widest projection of the batch sweep: the weights' bytes count
        dict(name="linear_batch_16", op="linear", M=16, K=8192, N=28672, dtype="bf16"),
        # a short prompt and odd sizes: nothing fits the tiles
        dict(name="linear_ragged_333", op="linear", M=333, K=4112, N=1003, dtype="f16"),
        # a long prefill through the gate projection: the tensor cores' rate counts
        dict(name="linear_prefill_8192", op="linear", M=8192, K=4096, N=14336, dtype="bf16"),
        # 16 tokens in the gate/up product of a layer of 256 experts: mostly one or two rows for each expert
        dict(name="experts_t16", op="experts", T=16, top_k=8, E=256, K=2048, N=1024, dtype="bf16"),
        # a prefill chunk in the same product: some 128 rows for each expert, unevenly
        dict(name="experts_t4096", op="experts", T=4096, top_k=8, E=256, K=2048, N=1024, dtype="bf16"),
        # the rows of a decode batch to their experts
        dict(name="dispatch_t16", op="dispatch", T=16, top_k=8, E=256, H=2048, dtype="bf16"),
        # the rows of a prefill chunk to their experts
        dict(name="dispatch_t4096", op="dispatch", T=4096, top_k=8, E=256, H=2048, dtype="bf16"),
        # an odd width that no vector load divides, and two choices of eight experts
        dict(name="combine_odd_t333", op="combine", T=333, top_k=2, E=8, H=1003, dtype="f16"),
        # the way back of a prefill chunk
        dict(name="combine_t4096", op="combine", T=4096, top_k=8, E=256, H=2048, dtype="bf16"),
        # a short training batch
        dict(name="backward_t256", op="backward", T=256, top_k=4, E=64, H=1024, dtype="f16"),
        # a training batch of the same layer as above
        dict(name="backward_t4096", op="backward", T=4096, top_k=8, E=256, H=2048, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "experts", "dispatch", "combine", "backward"))
    dtype = rng.choice(("f16", "bf16"))
    if op == "linear":
        while True:
            M, K, N = _spread(rng, 1, 8192), 16 * _spread(rng, 16, 896), _spread(rng, 128, 28672)
            if rng.random() < 0.7:
                N = -(-N // 8) * 8
            if M * K * N <= 8192 * 4096 * 14336 and K * N <= 8192 * 28672 and M * N <= 8192 * 14336:
                return dict(op=op, M=M, K=K, N=N, dtype=dtype)
    E = rng.choice((4, 8, 16, 64, 128, 256))
    top_k = min(E, rng.choice((1, 2, 4, 6, 8)))
    T = _spread(rng, 1, 4096)
    if op == "experts":
        while True:
            K, N = 16 * _spread(rng, 8, 256), _spread(rng, 64, 4096)
            if rng.random() < 0.7:
                N = -(-N // 8) * 8
            if E * K * N <= 256 * 2048 * 1024 and T * top_k * K * N <= 32768 * 2048 * 1024:
                return dict(op=op, T=T, top_k=top_k, E=E, K=K, N=N, dtype=dtype)
    H = _spread(rng, 64, 2048)
    if rng.random() < 0.7:
        H = -(-H // 8) * 8
    return dict(op=op, T=T, top_k=top_k, E=E, H=H, dtype=dtype)


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, cols, dtype):
    """Rows of different size, a few columns that stand out (as after a norm's gain)."""
    x = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    x *= 1 + 19 * (torch.rand((1, cols), generator=g, device="cuda") < 0.002)
    return x.to(DTYPES[dtype])


def _weights(g, shape):
    """INT8 codes of normal weights [.., N, K] and a scale for each output channel [.., N]."""
    q = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16).mul_(32).round_().clamp_(-127, 127)
    s = 0.02 / 32 * (0.5 + torch.rand(shape[:-1], generator=g, device="cuda"))
    return q.to(torch.int8), s


def _routing(g, T, top_k, E):
    """Each token's top_k different experts, some experts more popular than others, and its weights for them."""
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    top, ids = logits.topk(top_k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def _sorted_places(ids, E):
    """What a program keeps from sorting its routing: each pair's row and the experts' first rows."""
    order = torch.argsort(ids.reshape(-1), stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=order.device)
    offsets[1:] = torch.cumsum(torch.bincount(ids.reshape(-1).long(), minlength=E), 0)
    return row.to(torch.int32).reshape(ids.shape), offsets.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "linear":
        s["x"] = _activations(g, case["M"], case["K"], case["dtype"])
        s["wq"], s["sw"] = _weights(g, (case["N"], case["K"]))
        return s
    T, top_k, E = case["T"], case["top_k"], case["E"]
    s["ids"], s["weights"] = _routing(g, T, top_k, E)
    if case["op"] == "dispatch":
        s["x"] = _activations(g, T, case["H"], case["dtype"])
        return s
    s["row"], s["offsets"] = _sorted_places(s["ids"], E)
    if case["op"] == "experts":
        s["x"] = _activations(g, T * top_k, case["K"], case["dtype"])
        s["wq"], s["sw"] = _weights(g, (E, case["N"], case["K"]))
        return s
    s["y"] = _activations(g, T * top_k, case["H"], case["dtype"])
    if case["op"] == "backward":
        s["dout"] = _activations(g, T, case["H"], case["dtype"])
        s["dx"] = _activations(g, T * top_k, case["H"], case["dtype"])
    return s


# ---------------------------------------------------------------------------- plain forms

def _quantize_rows(x):
    """A scale for each row (its largest magnitude / 127) and the rounded quotients, as float32."""
    xf = x.float()
    s = xf.abs().amax(1, keepdim=True) / torch.full((1, 1), 127.0, device=x.device)
    q = torch.where(s == 0, torch.zeros_like(xf), torch.round(xf / s)).clamp(-127, 127)
    return q, s


def _plain_linear(x, wq, sw):
    q, s = _quantize_rows(x)
    return ((q @ wq.float().t()) * sw * s).to(x.dtype)


def _plain_experts(x, offsets, wq, sw):
    E, P = wq.shape[0], x.shape[0]
    q, s = _quantize_rows(x)
    r = torch.arange(P, device=x.device)
    e = torch.searchsorted(offsets[1:].long(), r, right=True)
    place = r - offsets.long()[e]
    room = int((offsets[1:] - offsets[:-1]).max())
    buf = torch.zeros((E, room, x.shape[1]), dtype=torch.float32, device=x.device)
    buf[e, place] = q
    y = torch.bmm(buf, wq.float().transpose(1, 2))
    return (y[e, place] * sw[e] * s).to(x.dtype)


def _plain_dispatch(x, ids, E):
    row, offsets = _sorted_places(ids, E)
    T, top_k = ids.shape
    pair = torch.empty(T * top_k, dtype=torch.int64, device=x.device)
    pair[row.reshape(-1).long()] = torch.arange(T * top_k, device=x.device)
    return {"row": row, "pair": pair.to(torch.int32), "offsets": offsets, "rows": x[pair // top_k]}


def _plain_combine(y, row, weights):
    return (y[row.long()].float() * weights[:, :, None]).sum(1).to(y.dtype)


def _plain_backward(dout, y, dx, row, weights):
    r = row.long()
    d = dout.float()[:, None, :]
    dy = torch.empty_like(y)
    dy[r.reshape(-1)] = (weights[:, :, None] * d).to(y.dtype).reshape(-1, y.shape[1])
    return {"dy": dy, "dweights": (d * y[r].float()).sum(-1), "dx": dx[r].float().sum(1).to(dx.dtype)}


def run(s):
    op = s["op"]
    if own:
        import bit_weight_only_pack_b200 as lbq
        if op == "linear":
            return lbq.w8a8_linear(s["x"], s["wq"], s["sw"])
        if op == "experts":
            xq, sx = lbq.quantize_int8_rows(s["x"])
            return lbq.moe_w8a8_gemm(xq, sx, s["offsets"], s["wq"], s["sw"], y_dtype=s["dtype"])
        if op == "dispatch":
            row, pair, offsets = lbq.moe_sort(s["ids"], s["E"])
            return {"row": row, "pair": pair, "offsets": offsets, "rows": lbq.moe_permute(s["x"], row)}
        if op == "combine":
            return lbq.moe_combine(s["y"], s["row"], s["weights"])
        dy, dweights = lbq.moe_combine_grad(s["dout"], s["y"], s["row"], s["weights"])
        return {"dy": dy, "dweights": dweights, "dx": lbq.moe_permute_grad(s["dx"], s["row"])}
    if op == "linear":
        return _plain_linear(s["x"], s["wq"], s["sw"])
    if op == "experts":
        return _plain_experts(s["x"], s["offsets"], s["wq"], s["sw"])
    if op == "dispatch":
        return _plain_dispatch(s["x"], s["ids"], s["E"])
    if op == "combine":
        return _plain_combine(s["y"], s["row"], s["weights"])
    return _plain_backward(s["dout"], s["y"], s["dx"], s["row"], s["weights"])


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N, "flops": 2 * M * N * K}
    T, top_k, E = case["T"], case["top_k"], case["E"]
    P = T * top_k
    if case["op"] == "experts":
        K, N = case["K"], case["N"]
        used = E * (1 - (1 - top_k / E) ** T)  # experts that have a row, on average
        return {"bytes": 2 * P * K + used * N * (K + 4) + 2 * P * N, "flops": 2 * P * N * K}
    H = case["H"]
    if case["op"] == "dispatch":
        return {"bytes": 12 * P + 4 * E + 2 * H * (T + P), "flops": 0}
    if case["op"] == "combine":
        return {"bytes": 8 * P + 2 * H * (T + P), "flops": 2 * P * H}
    return {"bytes": 12 * P + 2 * H * (2 * T + 3 * P), "flops": 4 * P * H}


# ---------------------------------------------------------------------------- the definitions in 64 bits

def _codes64(x):
    """Whole numbers nearest to 127 x / (the row's largest magnitude), and that magnitude / 127."""
    x = x.double()
    top = torch.linalg.vector_norm(x, ord=math.inf, dim=1)
    step = top / 127
    return torch.round(torch.nan_to_num(x / step[:, None], nan=0.0)), step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        q, step = _codes64(s["x"])
        y = torch.matmul(q, s["wq"].double().t())
        return y.mul_(step[:, None]).mul_(s["sw"].double()[None, :])
    if case["op"] == "experts":
        q, step = _codes64(s["x"])
        ends = s["offsets"].tolist()
        y = torch.empty((q.shape[0], case["N"]), dtype=torch.float64, device=q.device)
        for e in range(case["E"]):
            a, b = ends[e], ends[e + 1]
            if b > a:
                y[a:b] = torch.einsum("rk,nk->rn", q[a:b], s["wq"][e].double()) * s["sw"][e].double()
        return y * step[:, None]
    T, top_k = s["ids"].shape
    if case["op"] == "dispatch":
        ids = s["ids"].reshape(-1).tolist()
        order = sorted(range(len(ids)), key=lambda p: (ids[p], p))
        tokens = torch.tensor([p // top_k for p in order], device="cuda")
        return {"row": None, "pair": None, "offsets": None, "rows": s["x"].double()[tokens]}
    y, w, row = s["y"].double(), s["weights"].double(), s["row"].long()
    if case["op"] == "combine":
        out = torch.zeros((T, case["H"]), dtype=torch.float64, device="cuda")
        for j in range(top_k):
            out += w[:, j, None] * y[row[:, j]]
        return out
    dout, dx_rows = s["dout"].double(), s["dx"].double()
    dy = torch.empty_like(y)
    dw = torch.empty_like(w)
    dx = torch.zeros_like(dout)
    for j in range(top_k):
        dy[row[:, j]] = dout * w[:, j, None]
        dw[:, j] = torch.einsum("th,th->t", dout, y[row[:, j]])
        dx += dx_rows[row[:, j]]
    return {"dy": dy, "dweights": dw, "dx": dx}
