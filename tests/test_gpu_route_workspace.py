"""GPU: moe_route in a workspace that holds its own logit planes and no more (moe_route_scored may
need more of them, and MOE_OP_ROUTE's size serves both)."""
import pytest
import torch

import mixture_experts_layer_33_amd as moe
from ops_util import DEV, gen, randn, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,d", [(256, 256, 7168), (9, 64, 4096)])
def test_own_planes_suffice(T, E, d):
    """Eight K splits at these sizes: eight planes [T, E] of floats, 256-byte aligned."""
    print(f"\n[case] route workspace T={T} E={E} d={d}", flush=True)
    own, k = 8 * T * E * 4, 8
    s = moe.make_shape(T, d, E, k, 128)
    need = moe.workspace_bytes(s, moe.OP_ROUTE)
    assert own % 256 == 0 and own < need
    x, w = randn(gen(1), T, d, dtype=torch.bfloat16), randn(gen(2), E, d, scale=d ** -0.5)
    outs = []
    for n in (own, need):
        buf = torch.full((n + 4096,), 7, dtype=torch.uint8, device=DEV)
        out = torch.zeros(T, k, dtype=torch.int32, device=DEV), torch.zeros(T, k, device=DEV), torch.zeros(E, dtype=torch.int32, device=DEV)
        moe.moe_route(s, x, w, None, *out, buf[:n])
        torch.cuda.synchronize()
        assert (buf[n:] == 7).all()
        outs.append(out)
    assert all(same_bits(a, b) for a, b in zip(*outs))
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_route(s, x, w, None, *outs[0], buf[:own - 256])
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_route_scored(s, moe.make_router(), x, w, None, None, *outs[0], None, buf[:own])
