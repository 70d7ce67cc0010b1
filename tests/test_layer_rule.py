"""Layer's record of the rule that routed its tokens: a backward that would differentiate other gates than
those in its buffers is refused before anything runs (no GPU: the library's calls are replaced)."""
import pytest
import torch

import mixture_experts_layer_33_amd as moe

CALLS = ["moe_route", "moe_route_scored", "moe_dispatch", "moe_decode", "moe_forward", "moe_backward", "moe_backward_mx",
         "moe_backward_experts", "moe_route_scored_backward"]
T, D, E, K, F = 4, 512, 8, 2, 512
SIGMOID = dict(score="sigmoid", renormalise=True, scale=1.0)


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in CALLS:
        monkeypatch.setattr(moe, name, lambda *a, name=name, **k: seen.append(name))
    return seen


def layer(dtype="bf16"):
    a = moe.Layer.create(T, D, E, K, F, dtype=dtype, device="cpu")
    for name in ("ring_x", "expert_offset", "copy_slot", "slot_copy", "saved_au"):
        a.bufs[name] = torch.zeros(1)      # what forward(save_au=True) leaves besides its routing
    return a


def back(a, **kw):
    return a.backward(None, None, None, None, None, None, **kw)


def back_mx(a):
    return a.backward_mx(None, None, None, None, None, None, None)


@pytest.mark.parametrize("rule", [SIGMOID, dict(scale=2.0), dict(renormalise=False), dict(score="sigmoid", scale=2.5)], ids=str)
def test_scored_gates_need_their_router(calls, rule):
    router = moe.make_router(**rule)
    for dtype, grad in (("bf16", back), ("fp8", back), ("mxfp8", back_mx)):
        a = layer(dtype)
        a.route(None, None, router=router)
        del calls[:]
        with pytest.raises(ValueError, match="router"):
            grad(a)
        assert not calls
    a = layer()
    a.route(None, None, router=router)
    for other in (dict(rule, scale=3.0), dict(rule, groups=2), dict(rule, renormalise=not rule.get("renormalise", True))):
        with pytest.raises(ValueError, match="router"):
            back(a, router=moe.make_router(**other))
    back(a, router=moe.make_router(**rule))      # an equal one
    assert calls[-1] == "moe_route_scored_backward"
    a.route(None, None)                          # routed anew by moe_route
    back(a)
    assert calls[-1] == "moe_backward"


def test_the_rule_is_that_of_the_call(calls):
    """A router changed after the forward is another one."""
    a, router = layer(), moe.make_router("sigmoid")
    a.route(None, None, router=router)
    router.scale = 2.0
    with pytest.raises(ValueError, match="router"):
        back(a, router=router)


@pytest.mark.parametrize("how", ["route", "decode", "fused"])
def test_logits_of_an_older_call(calls, how):
    """After a call that routes by moe_route's rule, the logits are those of an older one."""
    a, router = layer(), moe.make_router("sigmoid")
    a.route(None, None, router=router)
    {"route": lambda: a.route(None, None), "decode": lambda: a.decode(None, None, None, None, None, None),
     "fused": lambda: a.forward_fused(None, None, None, None, None, None)}[how]()
    with pytest.raises(ValueError, match="router"):
        back(a, router=router)
    back(a)
    assert calls[-1] == "moe_backward"


def test_moe_route_s_own_rule_needs_no_router(calls):
    """Renormalised softmax gates of scale 1 have the gradient of moe_backward and moe_backward_mx, whatever groups
    and balance decided the choice."""
    for rule in (dict(), dict(groups=4, top_groups=2, group_top=2)):
        for dtype, grad, last in (("bf16", back, "moe_backward"), ("mxfp8", back_mx, "moe_backward_mx")):
            a = layer(dtype)
            a.route(None, None, router=moe.make_router(**rule), balance=torch.zeros(E))
            grad(a)
            assert calls[-1] == last


def test_gates_put_into_the_buffers_by_hand(calls):
    """A layer that has not routed knows nothing of its gates: either form runs."""
    for router in (None, moe.make_router("sigmoid")):
        a = layer()
        a._buf("topk_idx", (T, K), torch.int32)
        a._buf("topk_gate", (T, K), torch.float32)
        a._buf("logits", (T, E), torch.float32)
        back(a, router=router)


def test_a_refused_call_leaves_the_record(calls, monkeypatch):
    a = layer()
    a.route(None, None)

    def refuse(*args, **kw):
        raise moe.MoeError("moe_route_scored", 2)
    monkeypatch.setattr(moe, "moe_route_scored", refuse)
    with pytest.raises(moe.MoeError):
        a.route(None, None, router=moe.make_router("sigmoid"))
    back(a)
    assert calls[-1] == "moe_backward"
