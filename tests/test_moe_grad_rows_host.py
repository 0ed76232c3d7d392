"""lbq_moe_combine_grad_full without a GPU: the refusals of lbq_moe_combine_grad, before any launch."""

import pytest

P = 4096  # a 16-byte aligned address that is never read


@pytest.mark.parametrize("args,status", [
    *[({k: v}, 1) for k in ("T", "top_k", "rows", "H") for v in (0, -1)],
    *[({k: v}, 1) for k in ("dout", "Ys", "row", "weights", "dYs", "dw") for v in (None, P + 8)],
    ({"Ys": P}, 1),  # dYs itself
    ({"dt": 2}, 2), ({"T": 1 << 20, "top_k": 1 << 10}, 1),
])
def test_refusals(args, status):
    import bit_weight_only_pack_b200 as lbq
    a = dict(dout=P, Ys=2 * P, dt=0, rows=8, H=16, row=P, weights=P, T=4, top_k=2, dYs=P, dw=P) | args
    before = lbq.lbq_launch_count()
    with pytest.raises(lbq.LbqError) as e:
        lbq.lbq_moe_combine_grad_full(a["dout"], a["Ys"], a["dt"], a["rows"], a["H"], a["row"], a["weights"], a["T"],
                                      a["top_k"], a["dYs"], a["dw"], None)
    assert e.value.status == status and lbq.lbq_last_error()
    assert lbq.lbq_launch_count() == before
