"""GPU: the few-token layer with MXFP4 weights for every width and batch that has a kernel of its own, the rules that group experts,
both ends of the scale range, and stacks past 2^32 bytes.  Checked, with the tolerances, as in test_gpu_mxfp4."""
import pytest
import torch

import mixture_experts_layer_33_amd as moe
from oracle import mx4
from ops_util import DEV, gen, randn, same_bits
from test_gpu_mxfp4 import BF, GROUPED, U8, Decode, raw, weights

pytestmark = pytest.mark.gpu

FORMS = {   # by the pairs a wavefront holds (d) and sets of eight tokens
    "d4224_t3": dict(T=3, d=4224, E=5, k=2, f=128),
    "d5120_t1": dict(T=1, d=5120, E=6, k=3, f=256, fs=128),
    "d6144_t8": dict(T=8, d=6144, E=6, k=2, f=128, fs=256),
    "d2176_t9": dict(T=9, d=2176, E=10, k=2, f=256, fs=128),
    "d4096_t16": dict(T=16, d=4096, E=20, k=4, f=128),
    "d5120_t12": dict(T=12, d=5120, E=6, k=2, f=256, fs=128, bias=True),
    "d6144_t16": dict(T=16, d=6144, E=4, k=2, f=128),
    "d6272_t10": dict(T=10, d=6272, E=4, k=2, f=128, fs=128),
    "d7168_t16": dict(T=16, d=7168, E=16, k=4, f=128, fs=128, **dict(GROUPED, groups=4, top_groups=2)),
    "d8192_t16": dict(T=16, d=8192, E=3, k=2, f=256, fs=256),
    "e600_t12": dict(T=12, d=2304, E=600, k=4, f=128, bias=True),
    "e1024_t16": dict(T=16, d=512, E=1024, k=16, f=128, fs=128),
    "e520_t5_d7168": dict(T=5, d=7168, E=520, k=2, f=128),
}
RULES = {   # groups of which sizes, and how many experts a lane looks at (4, 8 or 16)
    "e12_g4": dict(T=5, d=256, E=12, k=3, f=128, groups=4, top_groups=2, group_top=2),
    "e12_g4_top1": dict(T=16, d=256, E=12, k=4, f=128, fs=128, score="sigmoid", groups=4, top_groups=3, group_top=1, balance=True),
    "e60_g3_plain": dict(T=9, d=384, E=60, k=6, f=128, groups=3, top_groups=2, group_top=2, renormalise=False, scale=1.5),
    "e300_g4": dict(T=8, d=256, E=300, k=8, f=128, score="sigmoid", groups=4, top_groups=2, group_top=2, balance=True),
    "e512_g8": dict(T=3, d=512, E=512, k=8, f=128, fs=128, **GROUPED),
    "e512_g8_softmax": dict(T=16, d=256, E=512, k=10, f=128, groups=8, top_groups=3, group_top=2, renormalise=False),
    "e640_g5": dict(T=4, d=256, E=640, k=5, f=128, bias=True, groups=5, top_groups=2, group_top=1),
    "e1000_g8": dict(T=2, d=256, E=1000, k=8, f=128, score="sigmoid", groups=8, top_groups=4, group_top=2, balance=True),
    "e1024_g64": dict(T=9, d=128, E=1024, k=16, f=128, score="sigmoid", groups=64, top_groups=4, group_top=2),
    "all_groups": dict(T=2, d=256, E=16, k=16, f=128, groups=4, top_groups=4, group_top=2, balance=True),
}


class Slices:
    """fp64 values of a stack's rows, made when they are asked for."""

    def __init__(self, c, s):
        self.c, self.s = c.view(-1, c.shape[-1]), s

    def __getitem__(self, rows):
        return mx4.values(raw(self.c[rows]), raw(self.s[:, rows].contiguous()))


def decode(T, d, E, k, f, fs=0, seed=0, make=None, **rule):
    """A Decode whose stacks' fp64 values are made a slice at a time.  make: (codes, scales) of a stack [E, rows, cols]."""
    c = Decode(T=T, d=128, E=E, k=k, f=128, seed=seed, **rule)
    g = gen(3000 + seed)
    c.shape = moe.make_shape(T, d, E, k, f, fs=fs, dtype="mxfp4")
    moe.check_shape(c.shape)
    c.x, c.w_r = randn(g, T, d, dtype=BF), randn(g, E, d, scale=d ** -0.5)
    for n, r, cols in (("gate", f, d), ("up", f, d), ("down", d, f)):
        w, s = moe.quantize_mxfp4(randn(g, E, r, cols, dtype=BF, scale=cols ** -0.5)) if make is None else make(g, E, r, cols)
        c.W[n] = (w, s, Slices(w, s))
    c.S = {n: weights(g, r, cols) if fs else (None, None, None) for n, r, cols in (("gate", fs, d), ("up", fs, d), ("down", d, fs))}
    c.ws = torch.full((moe.workspace_bytes(c.shape, moe.OP_DECODE),), 0xAB, dtype=U8, device=DEV)
    c.out = (torch.full((T, d), 7, dtype=BF, device=DEV), torch.full((T, k), -1, dtype=torch.int32, device=DEV),
             torch.full((T, k), -1.0, device=DEV))
    return c


@pytest.mark.parametrize("name", list(FORMS))
def test_decode_of_each_width(name):
    print(f"\n[case] decode_mxfp4 {name}", flush=True)
    decode(**FORMS[name], seed=200 + len(name)).check()


@pytest.mark.parametrize("name", list(RULES))
def test_decode_with_groups(name):
    print(f"\n[case] decode_mxfp4 {name}", flush=True)
    decode(**RULES[name], seed=300 + len(name)).check()


def test_decode_with_scales_at_both_ends():
    """W_down under the largest scales the quantiser writes (252), W_up under small ones; and W_up under 0."""
    print("\n[case] decode_mxfp4 scale ends", flush=True)
    for T in (2, 11):
        c = Decode(T=T, d=384, E=6, k=2, f=256, fs=128, seed=400 + T)
        for kind in (c.W, c.S):
            for n, by in (("down", None), ("up", -70)):
                w, s, _ = kind[n]
                s = (s.int() + (252 - int(s.max()) if by is None else by)).to(U8)
                kind[n] = (w, s, mx4.values(raw(w).reshape(-1, w.shape[-1]), raw(s)))
        assert max(int(k["down"][1].max()) for k in (c.W, c.S)) == 252
        c.check()
        for kind in (c.W, c.S):
            w, s, _ = kind["up"]
            kind["up"] = (w, torch.zeros_like(s), mx4.values(raw(w).reshape(-1, w.shape[-1]), raw(torch.zeros_like(s))))
        c.x *= 2.0 ** 40              # h stays among bf16's normal numbers, the logits what they were
        c.w_r *= 2.0 ** -40
        c.check()


def test_decode_of_a_stack_past_four_gib():
    """Expert stacks of 4.3 GB of codes each: the last experts, whose offsets pass 2^32, are as right as the first."""
    print("\n[case] decode_mxfp4 large stack", flush=True)
    def make(g, *shape):
        E, r, cols = shape
        w = torch.randint(0, 256, (E, r, cols // 2), generator=g, device=DEV, dtype=U8)
        assert w.numel() > 1 << 32
        return w, torch.randint(118, 122, (cols // 128, E * r, 4), generator=g, device=DEV, dtype=U8)

    E = 520
    c = decode(T=3, d=7680, E=E, k=3, f=2176, bias=True, seed=500, make=make)
    c.b_r[:] = -100.0
    c.b_r[[0, E // 2, E - 2, E - 1]] = 0.0
    c.check()
    assert int(c.out[1].max()) == E - 1


def test_layer_decode_with_a_shared_expert_and_a_balance_bias():
    """Layer.decode is the bare call, with its own buffers."""
    print("\n[case] Layer.decode shared, balance", flush=True)
    for T in (1, 6, 16):
        c = Decode(T=T, d=512, E=32, k=4, f=256, fs=384, bias=True, seed=600 + T, **dict(GROUPED, groups=4, top_groups=2))
        names = ("gate", "up", "down")
        layer = moe.Layer.create(T, 512, 32, 4, 256, fs=384, dtype="mxfp4", device=DEV)
        got = layer.decode(c.x, c.w_r, c.b_r, *(c.W[n][0] for n in names), *(c.S[n][0] for n in names),
                           scales=tuple(c.W[n][1] for n in names), shared_scales=tuple(c.S[n][1] for n in names), router=c.router,
                           balance=c.balance)
        want = c.run()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(got, want)) and layer.routed == bytes(c.router)
        c.check()
