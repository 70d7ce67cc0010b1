"""GPU: a backward after a scored forward: the gradients that moe_route's rule gives where that rule made the
gates (whatever groups and balance decided the choice), a refusal where another one did."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_33_amd as moe
import oracle
from ops_util import DEV, gen, host, randn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
T, D, E, K, F = 96, 256, 16, 3, 128
TOL = {"bf16": 2e-2, "mxfp8": 6e-2}     # the tolerances of the two backwards' own parity tests


def setup(dtype):
    g = gen(31)
    x, dy, wr = randn(g, T, D, dtype=BF), randn(g, T, D, dtype=BF), randn(g, E, D) / 16
    ws = [randn(g, E, r, c, dtype=BF, scale=c ** -0.5) for r, c in ((F, D), (F, D), (D, F))]
    layer = moe.Layer.create(T, D, E, K, F, dtype=dtype)
    q = [moe.quantize_mx(w) for w in ws] if dtype == "mxfp8" else [(w, None) for w in ws]

    def forward(**kw):
        layer.forward(x, wr, None, *(c for c, _ in q), scales=tuple(s for _, s in q), save_au=True, **kw)

    def backward(**kw):
        if dtype == "mxfp8":
            return layer.backward_mx(dy, x, wr, *moe.quantize_mx_t_backward_weights(*ws), **kw)
        return layer.backward(dy, x, wr, *ws, **kw)
    return layer, forward, backward, (x, dy, wr, ws)


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_renormalised_softmax_in_groups(dtype):
    print(f"\n[case] {dtype} backward after a grouped, balanced softmax forward", flush=True)
    layer, forward, backward, (x, dy, wr, ws) = setup(dtype)
    bal = randn(gen(3), E, scale=0.02)
    forward(router=moe.make_router(groups=4, top_groups=2, group_top=2), balance=bal)
    got = [t.clone() for t in backward()]
    torch.cuda.synchronize()
    b = layer.bufs
    idx = b["topk_idx"].cpu().numpy().astype(np.int64)
    plain = oracle.route(host(x), host(wr), None, K)
    assert not np.array_equal(idx, plain.idx)      # groups and balance did move the choice
    r = oracle.Routing(idx, host(b["topk_gate"]), b["expert_count"].cpu().numpy(), host(b["logits"]), plain.probs)
    W = oracle.weights_from_arrays(*(host(w) for w in ws))
    if dtype == "mxfp8":
        ref = oracle.backward_mx(host(x), host(wr), r, W, host(dy), oracle.dispatch(idx, E, layer.shape.capacity, 0))
    else:
        ref = oracle.backward(host(x), host(wr), r, W, host(dy))
    for name, t in zip(("dx", "dw_gate", "dw_up", "dw_down", "dw_router"), got):
        off = oracle.max_abs_rel(host(t), getattr(ref, name))
        print(f"  {name} max-abs-rel {off:.2e}", flush=True)
        assert off <= TOL[dtype], name


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_other_gates_are_refused(dtype):
    print(f"\n[case] {dtype} backward of other gates", flush=True)
    layer, forward, backward, _ = setup(dtype)
    for rule in (dict(score="sigmoid"), dict(scale=2.0), dict(renormalise=False)):
        router = moe.make_router(**rule)
        forward(router=router)
        with pytest.raises(ValueError, match="router"):
            backward()
        if dtype == "bf16":
            with pytest.raises(ValueError, match="router"):
                backward(router=moe.make_router(score="sigmoid", scale=3.0))
            assert all(t.isfinite().all() for t in backward(router=router))
    forward()
    if dtype == "bf16":
        with pytest.raises(ValueError, match="router"):
            backward(router=moe.make_router("sigmoid"))
    assert all(t.isfinite().all() for t in backward())
    torch.cuda.synchronize()
