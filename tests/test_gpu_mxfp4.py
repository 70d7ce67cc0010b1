"""GPU: MXFP4 weights: quantiser, the product of bf16 rows, the layer for a few tokens and the experts of a dispatched
batch, against the fp64 oracle.

Tolerances.  A product of a bf16 value and an E2M1 value under its scale is exact in fp32.  A sum over K of them on the bf16
matrix instruction is at most K additions (and K / 32 additions of the instruction's result), each counted with a
whole step, 2^-23, of a partial sum that is at most the sum of the terms' sizes: SUM(K) = (K + K / 32 + 40) 2^-23 of that
(40: joining the wavefronts' parts).  Then the output's own rounding, half a step.
  Logits are fp32 sums of d terms, off by at most (d + 40) 2^-23 of the sum of their sizes; the scores of the rule (at most
one exponential and one division more, a few steps) by at most that and 2^-20 of a logit of size below 16, and c =
score + balance alike: a choice that the oracle decides by more than twice the larger of these is the same.
  The layer: with A, U the gate and up sums and dA, dU their errors as above, h = silu(A) U is off by at most 1.1 |U| dA +
|silu(A)| dU (|silu'| < 1.1), 2^-19 of itself for the hardware exponential and reciprocal (about 2 ulp each), the products and
the gate, and 2^-16 for the second bf16 part's rounding; y adds SUM of the down products.  The gates that y is checked with
are the call's own; they are checked by themselves, off by the logits' error (a softmax score
changes by at most twice that of itself, a sigmoid's by at most that, a sum over the choice by as much again)."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_33_amd as moe
from oracle import mx, mx4, ops
from ops_util import DEV, HALF, codes, gen, host, randn, same_bits, within

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def SUM(K):
    return (K + K / 32 + 40) * 2.0 ** -23


def raw(t):
    return t.cpu().numpy()


def equal(got, want):
    assert got.shape == want.shape
    n = int((got != want).sum())
    assert n == 0, (n, np.argwhere(got != want)[:5].tolist())


def weights(g, *shape, scale=None):
    """bf16 weights quantised by the library: (codes, scales, fp64 values [rows, cols])."""
    w = randn(g, *shape, dtype=BF, scale=shape[-1] ** -0.5 if scale is None else scale)
    c, s = moe.quantize_mxfp4(w)
    return c, s, mx4.values(raw(c).reshape(-1, shape[-1] // 2), raw(s))


# ----------------------------------------------------------------------------- quantiser
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (127, 384), (300, 640)])
def test_quantiser(rows, cols):
    print(f"\n[case] quantize_mxfp4 {rows}x{cols}", flush=True)
    x = randn(gen(rows), rows, cols, dtype=BF)
    x[0, :128] = 0
    x[-1, -128:] *= 2.0 ** 90
    x[rows // 2, :32] *= 2.0 ** -125
    c, s = moe.quantize_mxfp4(x)
    torch.cuda.synchronize()
    want_c, want_s = mx4.quantise(host(x))
    equal(mx4.scale_rows(raw(s)), want_s)
    equal(mx4.unpack(raw(c)), want_c)


def test_quantiser_of_every_bf16_value():
    """Every finite bf16 value, in a block whose largest value sets each exponent around it."""
    print("\n[case] quantize_mxfp4 all", flush=True)
    bits = torch.arange(65536, dtype=torch.int32)
    v = bits.to(torch.int16).view(BF)
    v = v[torch.isfinite(v.float())]
    top = torch.exp2(torch.floor(torch.log2(v.abs().double().clamp_min(2.0 ** -126))))
    blocks = []
    for up in (1.0, 2.0, 8.0, 32.0):      # the block's maximum, in units of the value's power of two
        b = torch.zeros(v.numel(), 32, dtype=BF)
        b[:, 0] = (top * up).clamp_max(2.0 ** 127).to(BF)
        b[:, 1:] = v[:, None]
        b[:, 0] = torch.where(v.abs() > b[:, 0], v.abs(), b[:, 0])
        blocks.append(b)
    x = torch.cat(blocks)
    x = x[:x.shape[0] // 4 * 4].reshape(-1, 128).to(DEV)
    c, s = moe.quantize_mxfp4(x)
    torch.cuda.synchronize()
    want_c, want_s = mx4.quantise(host(x))
    equal(mx4.scale_rows(raw(s)), want_s)
    equal(mx4.unpack(raw(c)), want_c)


def test_quantiser_of_broken_blocks_stacks_and_nothing():
    print("\n[case] quantize_mxfp4 NaN", flush=True)
    x = randn(gen(1), 2, 64, 256, dtype=BF)
    x[0, 5, 3], x[1, 20, 130], x[1, 63, 255] = float("nan"), -float("inf"), float("inf")
    c, s = moe.quantize_mxfp4(x)
    torch.cuda.synchronize()
    want_c, want_s = mx4.quantise(host(x).reshape(128, 256))
    assert int((want_s == 255).sum()) == 3
    equal(mx4.scale_rows(raw(s)), want_s)
    equal(mx4.unpack(raw(c).reshape(128, 128)), want_c)
    c, s = moe.quantize_mxfp4(x[0, :0])
    assert c.shape == (0, 128) and s.shape == (2, 0, 4)


# ----------------------------------------------------------------------------- product
def matmul(x, w, s, ty):
    M, K, N = x.shape[0], x.shape[1], w.shape[0]
    out = torch.full((M + 1, N), 7, dtype=ty, device=DEV)     # the row behind stays as it was
    moe.moe_matmul_mxfp4(x, w, s, out[:M], moe.matmul_mxfp4_workspace(M, N, K, DEV))
    torch.cuda.synchronize()
    assert bool((out[M] == 7).all())
    return out[:M]


def check_product(out, x, W):
    X = host(x)
    ref = X @ W.T
    tol = HALF[out.dtype] * abs(ref) + SUM(X.shape[1]) * (abs(X) @ abs(W).T)
    within(host(out), ref, tol, "product")
    if out.dtype == BF:
        assert np.linalg.norm(host(out) - ref) <= 2.0 ** -8 * np.linalg.norm(ref) + 1e-30


SIZES = [(1, 1, 128), (1, 16, 256), (1, 7168, 512), (2, 40, 384), (3, 129, 640), (5, 1000, 2048), (8, 256, 1024), (9, 4100, 1152), (15, 72, 128),
         (16, 131, 7168), (2, 50, 8192), (1, 33, 8320), (7, 100, 12288), (17, 264, 640), (31, 512, 256), (33, 130, 128), (48, 2048, 1408), (64, 384, 384),
         (65, 128, 256), (100, 77, 512), (127, 256, 128), (128, 128, 256), (129, 257, 384), (200, 640, 1152), (255, 255, 128), (257, 1032, 256),
         (512, 512, 512), (700, 4168, 640), (1000, 128, 2048), (1536, 1544, 256), (2045, 4100, 256), (40, 1001, 7168), (61, 8, 4096), (300, 300, 4224)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("ty", [BF, F32])
def test_matmul(M, N, K, ty):
    print(f"\n[case] matmul_mxfp4 {M}x{N}x{K} {ty}", flush=True)
    g = gen(M + N)
    x = randn(g, M, K, dtype=BF)
    w, s, W = weights(g, N, K)
    out = matmul(x, w, s, ty)
    check_product(out, x, W)
    assert same_bits(out, matmul(x, w, s, ty))


def test_matmul_rows_are_independent():
    """A row of NaN and one of infinities leave the others as they were; a NaN scale spoils its column alone."""
    print("\n[case] matmul_mxfp4 NaN rows", flush=True)
    g = gen(3)
    for M in (4, 40):
        x = randn(g, M, 384, dtype=BF)
        w, s, _ = weights(g, 100, 384)
        clean = matmul(x, w, s, F32)
        y = x.clone()
        y[1, 5], y[2, 300] = float("nan"), float("inf")
        got = matmul(y, w, s, F32)
        keep = [0] + list(range(3, M))
        assert same_bits(got[keep], clean[keep]) and bool(torch.isnan(got[1]).all()) and not bool(torch.isfinite(got[2]).all())
        t = s.clone()
        t[1, 40, 2] = 255
        got = matmul(x, w, t, F32)
        cols = [n for n in range(100) if n != 40]
        assert bool(torch.isnan(got[:, 40]).all()) and same_bits(got[:, cols], clean[:, cols])


def test_matmul_of_extreme_scales():
    """Blocks whose scales differ by 2^100 and more: sums are dominated by the large ones to fp32's precision."""
    print("\n[case] matmul_mxfp4 scales", flush=True)
    g = gen(4)
    x = randn(g, 5, 512, dtype=BF)
    w, s, _ = weights(g, 64, 512)
    s = (s.int() + torch.randint(-60, 60, s.shape, generator=g, device=DEV)).clamp(1, 250).to(U8)
    W = mx4.values(raw(w), raw(s))
    check_product(matmul(x, w, s, F32), x, W)


def test_matmul_of_nothing():
    x, (w, s, _) = torch.zeros(0, 256, dtype=BF, device=DEV), weights(gen(5), 32, 256)
    out = torch.empty(0, 32, dtype=BF, device=DEV)
    moe.moe_matmul_mxfp4(x, w, s, out)
    moe.moe_matmul_mxfp4(torch.zeros(3, 256, dtype=BF, device=DEV), w[:0], s[:, :0].contiguous(), torch.empty(3, 0, dtype=F32, device=DEV))


def test_matmul_of_many_bytes():
    """Codes, rows and outputs whose offsets pass 2^31 and 2^32: the last ones are as right as the first."""
    print("\n[case] matmul_mxfp4 large", flush=True)
    g = gen(6)
    N, K = 262128, 16256                       # 2.1 GB of codes
    w, s = torch.zeros(N, K // 2, dtype=U8, device=DEV), torch.full((K // 128, N, 4), 127, dtype=U8, device=DEV)
    at = torch.tensor([0, 1, N // 2, N - 9, N - 2, N - 1], device=DEV)
    part, ps, W = weights(g, len(at), K)
    w[at], s[:, at] = part, ps
    for M in (1, 11, 20):
        x = randn(g, M, K, dtype=BF)
        out = matmul(x, w, s, F32)
        check_product(out[:, at], x, W)
        rest = torch.ones(N, dtype=torch.bool, device=DEV)
        rest[at] = False
        assert bool((out[:, rest] == 0).all())
    del w, s, out, rest
    M, K, N = 250007, 16384, 24                # 8.2 GB of rows
    x = torch.zeros(M, K, dtype=BF, device=DEV)
    at = torch.tensor([0, 127, M // 2, M - 3, M - 1], device=DEV)
    x[at] = randn(g, len(at), K, dtype=BF)
    w, s, W = weights(g, N, K)
    out = matmul(x, w, s, F32)
    check_product(out[at], x[at], W)
    out[at] = 0
    assert bool((out == 0).all())


def test_matmul_side_stream_and_graph():
    print("\n[case] matmul_mxfp4 graph", flush=True)
    for M, N, K in ((2, 512, 1024), (12, 512, 9216), (40, 520, 4096), (300, 520, 512), (2100, 1024, 256)):
        g = gen(M)
        x = randn(g, M, K, dtype=BF)
        w, s, _ = weights(g, N, K)
        want = matmul(x, w, s, BF)
        ws = moe.matmul_mxfp4_workspace(M, N, K, DEV)
        out = torch.zeros_like(want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        moe.moe_matmul_mxfp4(x, w, s, out, ws, stream=side)
        side.synchronize()
        assert same_bits(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_matmul_mxfp4(x, w, s, out, ws)
        for _ in range(4):
            x.mul_(-1.5)
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            assert same_bits(got, matmul(x, w, s, BF))


# ----------------------------------------------------------------------------- the layer for a few tokens
class Decode:
    def __init__(self, T, d, E, k, f, fs=0, seed=0, bias=False, balance=False, **rule):
        g = gen(1000 + seed)
        self.shape = moe.make_shape(T, d, E, k, f, fs=fs, dtype="mxfp4")
        moe.check_shape(self.shape)
        self.router = moe.make_router(**rule)
        self.x = randn(g, T, d, dtype=BF)
        self.w_r = randn(g, E, d, scale=d ** -0.5)
        self.b_r = randn(g, E, scale=0.1) if bias else None
        self.balance = randn(g, E, scale=0.05) if balance else None
        self.W = {n: weights(g, E, r, c) for n, r, c in (("gate", f, d), ("up", f, d), ("down", d, f))}
        self.S = {n: weights(g, r, c) if fs else (None, None, None) for n, r, c in (("gate", fs, d), ("up", fs, d), ("down", d, fs))}
        self.ws = torch.full((max(moe.workspace_bytes(self.shape, moe.OP_DECODE), 1),), 0xAB, dtype=U8, device=DEV)
        self.out = (torch.full((T, d), 7, dtype=BF, device=DEV), torch.full((T, k), -1, dtype=torch.int32, device=DEV),
                    torch.full((T, k), -1.0, device=DEV))

    def run(self, x=None, ws=None, out=None, stream=None):
        W, S = self.W, self.S
        names = ("gate", "up", "down")
        moe.moe_decode_mxfp4(self.shape, self.router, self.x if x is None else x, self.w_r, self.b_r, self.balance,
                             *(W[n][0] for n in names), *(W[n][1] for n in names), *(S[n][0] for n in names),
                             *(S[n][1] for n in names), *(self.out if out is None else out), self.ws if ws is None else ws, stream)
        return self.out if out is None else out

    def logit_error(self):
        """Largest error of an fp32 logit, and the logits in fp64."""
        X, W = host(self.x), host(self.w_r)
        l = X @ W.T + (0 if self.b_r is None else host(self.b_r))
        return (self.shape.hidden + 40) * 2.0 ** -23 * float(np.nanmax(abs(X) @ abs(W).T)) + 2.0 ** -20, l

    def check_choice(self, idx, gate):
        s, r = self.shape, self.router
        off, l = self.logit_error()
        rule = ops.Rule("sigmoid" if r.score else "softmax", r.groups, r.top_groups, r.group_top, bool(r.renormalise), r.scale)
        bal = None if self.balance is None else host(self.balance)
        sure = ops.margins(l, rule, s.top_k, bal) > 2 * off
        want = ops.choose(l, rule, s.top_k, bal)
        assert np.array_equal(idx[sure], want[sure])
        assert (np.diff(idx, axis=1) > 0).all() and (idx >= 0).all() and (idx < s.experts).all()
        if r.groups == 1:      # however near to a tie: what is chosen is at most the error below what is not
            c = l if bal is None else ops.scores(l, rule) + bal
            out = c.copy()
            np.put_along_axis(out, idx.astype(np.int64), -np.inf, axis=1)
            assert (np.take_along_axis(c, idx.astype(np.int64), axis=1).min(axis=1) >= out.max(axis=1) - 2 * off).all()
        g = ops.gates(l, idx.astype(np.int64), rule)
        within(gate, g, (4 * off + 2.0 ** -20) * abs(g) + 1e-30, "gates")

    def expect(self, idx, gate):
        """(y, tolerance) from the given choice and gates."""
        s = self.shape
        d, f, fs = s.hidden, s.ffn, s.shared_ffn
        X = host(self.x)
        y, tol = np.zeros_like(X), np.zeros_like(X)

        def add(t, g, wg, wu, wd, F):
            x = X[t:t + 1]
            A, U = x @ wg.T, x @ wu.T
            dA, dU = SUM(d) * (abs(x) @ abs(wg).T), SUM(d) * (abs(x) @ abs(wu).T)
            h = mx4.swiglu(A, U)
            dh = 1.1 * abs(U) * dA + abs(mx4.swiglu(A, np.ones_like(A))) * dU + (2.0 ** -19 + 2.0 ** -16) * abs(h)
            n = (s.top_k * f + fs)
            y[t] += g * (h @ wd.T)[0]
            tol[t] += abs(g) * ((dh + SUM(n) * abs(h)) @ abs(wd).T)[0]

        for t in range(s.tokens):
            for j in range(s.top_k):
                e = int(idx[t, j])
                add(t, float(gate[t, j]), self.W["gate"][2][e * f:(e + 1) * f], self.W["up"][2][e * f:(e + 1) * f],
                    self.W["down"][2][e * d:(e + 1) * d], f)
            if fs:
                add(t, 1.0, self.S["gate"][2], self.S["up"][2], self.S["down"][2], fs)
        return y, tol + HALF[BF] * (abs(y) + tol)

    def check(self):
        y, idx, gate = self.run()
        torch.cuda.synchronize()
        self.check_choice(idx.cpu().numpy(), host(gate))
        ref, tol = self.expect(idx.cpu(), gate.cpu().double())
        within(host(y), ref, tol, "y")
        err = np.linalg.norm(host(y) - ref) / max(np.linalg.norm(ref), 1e-30)
        assert err <= 2.0 ** -8, err
        first = [t.clone() for t in (y, idx, gate)]
        self.ws.fill_(0x3C)      # no initial contents needed
        again = self.run()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(first, again))


GROUPED = dict(score="sigmoid", groups=8, top_groups=4, group_top=2, scale=2.5, balance=True)
LAYERS = {
    "one": dict(T=1, d=256, E=8, k=2, f=128),
    "one_column": dict(T=1, d=128, E=1, k=1, f=128),
    "three": dict(T=3, d=1152, E=24, k=3, f=384, fs=256),
    "eight": dict(T=8, d=768, E=64, k=8, f=256, fs=128, **GROUPED),
    "nine": dict(T=9, d=512, E=16, k=4, f=384, fs=640, bias=True, score="sigmoid"),
    "sixteen": dict(T=16, d=640, E=40, k=5, f=128, renormalise=False, scale=1.5),
    "all_chosen": dict(T=5, d=384, E=16, k=16, f=256, fs=128),
    "every_pair": dict(T=16, d=256, E=300, k=16, f=128, fs=128),
    "same_expert": dict(T=16, d=512, E=1, k=1, f=640),
    "wide": dict(T=4, d=4096, E=4, k=2, f=256, fs=384),
    "widest": dict(T=2, d=8192, E=3, k=2, f=128),
    "odd_wide": dict(T=7, d=7296, E=4, k=3, f=128, bias=True),
    "tall": dict(T=6, d=256, E=4, k=2, f=2176, fs=1408),
    "many_experts": dict(T=2, d=128, E=1024, k=10, f=128, bias=True),
}


@pytest.mark.parametrize("name", list(LAYERS))
def test_decode(name):
    print(f"\n[case] decode_mxfp4 {name}", flush=True)
    Decode(**LAYERS[name], seed=len(name)).check()


@pytest.mark.parametrize("T", range(1, 17))
def test_decode_of_each_batch(T):
    print(f"\n[case] decode_mxfp4 T {T}", flush=True)
    Decode(T=T, d=384, E=12, k=3, f=256, fs=128, seed=T).check()


def test_decode_tokens_are_independent():
    """A token of NaN leaves the others' results as they were, bit for bit."""
    print("\n[case] decode_mxfp4 NaN token", flush=True)
    for T in (4, 12):
        c = Decode(T=T, d=384, E=6, k=2, f=256, fs=128, seed=50 + T)
        clean = [t.clone() for t in c.run()]
        c.x[2, 7] = float("nan")
        y, idx, gate = c.run()
        torch.cuda.synchronize()
        keep = [t for t in range(T) if t != 2]
        assert bool((idx[2] >= 0).all()) and bool((idx[2] < 6).all())
        assert same_bits(y[keep], clean[0][keep]) and torch.equal(idx[keep], clean[1][keep])
        assert bool(torch.isnan(y[2]).all())


def test_decode_in_graphs_that_share_a_workspace():
    """Two captured calls of different shapes with one workspace, replayed in turn, and calls on two streams with a workspace each."""
    print("\n[case] decode_mxfp4 graphs", flush=True)
    cases = [Decode(T=3, d=640, E=24, k=3, f=256, fs=128, seed=80), Decode(T=12, d=384, E=300, k=4, f=128, seed=81)]
    big = torch.full((max(c.ws.numel() for c in cases),), 0x5A, dtype=U8, device=DEV)
    graphs = []
    for c in cases:
        c.run(ws=big)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run(ws=big)
        graphs.append(graph)
    for i in range(3):
        for c, graph in zip(cases, graphs):
            c.x.copy_(randn(gen(90 + i), *c.x.shape, dtype=BF))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in c.out]
            eager = tuple(torch.empty_like(t) for t in c.out)
            c.run(out=eager)
            torch.cuda.synchronize()
            assert all(same_bits(a, b) for a, b in zip(got, eager))
    want = [[t.clone() for t in c.run()] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, stream in zip(cases, streams):
            c.run(stream=stream)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert all(same_bits(a, b) for a, b in zip(c.out, w))


def test_decode_experts_that_are_taken_out():
    """A bias of -inf takes experts out; a token that keeps none has gates 0 and the shared expert's output alone."""
    print("\n[case] decode_mxfp4 -inf", flush=True)
    c = Decode(T=3, d=256, E=8, k=2, f=128, fs=128, bias=True, seed=60)
    c.b_r[:] = -float("inf")
    y, idx, gate = c.run()
    torch.cuda.synchronize()
    assert bool((gate == 0).all())
    ref, tol = c.expect(idx.cpu(), gate.cpu().double())
    within(host(y), ref, tol, "shared alone")


# ----------------------------------------------------------------------------- the experts of a dispatched batch
TO_E4M3 = torch.tensor([0x00, 0x30, 0x38, 0x3C, 0x40, 0x44, 0x48, 0x4C], dtype=U8)
TO_E4M3 = torch.cat([TO_E4M3, TO_E4M3 | 0x80])


def as_e4m3(c):
    """Packed E2M1 codes as the E4M3 codes of the same values."""
    t = TO_E4M3.to(c.device)
    return torch.stack([t[(c & 15).long()], t[(c >> 4).long()]], -1).flatten(-2).contiguous()


class Experts:
    def __init__(self, T, d, E, k, f, C=None, head=0, seed=0, crowd=None):
        g = gen(2000 + seed)
        self.layer = moe.Layer.create(T, d, E, k, f, C, dtype="mxfp4", device=DEV)
        self.head = head
        self.x = randn(g, T, d, dtype=BF)
        pick = torch.rand(T, E, generator=g, device=DEV)
        if crowd is not None:
            pick[:, crowd] += 1
        self.idx = pick.topk(k, dim=1).indices.sort(1).values.to(torch.int32).contiguous()
        self.W = {n: weights(g, E, r, c) for n, r, c in (("gate", f, d), ("up", f, d), ("down", d, f))}

    def run(self):
        L = self.layer
        ring, rs, off, cs, sc = L.dispatch(self.x, self.idx, self.head)
        L._buf("ring_y", (L.shape.capacity, L.shape.hidden), BF).fill_(7)
        y, _ = L.expert_ffn(ring, rs, off, self.head, *(self.W[n][0] for n in self.W), tuple(self.W[n][1] for n in self.W))
        return ring, rs, off, y


def mx_round(h, X):
    return mx.DECODE_TABLE[mx.encode_e4m3(np.ldexp(h, -X))] * 2.0 ** X


def h_bounds(h, e):
    """h as the MX rows hold it, and how far a value off by up to e may land from that."""
    def per_block(v):
        return np.repeat(mx.block_exponent(v.reshape(v.shape[0], -1, 32).max(2)), 32, axis=1)
    X = per_block(abs(h))
    q = mx_round(h, X)
    off = np.zeros_like(h)
    for Y in (per_block(np.maximum(abs(h) - e, 0)), per_block(abs(h) + e)):
        for v in (h - e, h + e):
            off = np.maximum(off, abs(mx_round(v, Y) - q))
    return q, off


def cut(A, W):
    """What the 8-bit matrix instruction may cut off: for eight consecutive products a grid of 2^-13 of the largest one's
    binade, seven times."""
    top = lambda v: abs(v).reshape(v.shape[0], -1, 8).max(2)  # noqa: E731
    return 7 * 2.0 ** -13 * (top(A) @ top(W).T)


EXPERTS = {
    "one_row": dict(T=1, d=128, E=4, k=1, f=128),
    "few": dict(T=9, d=256, E=8, k=2, f=384),
    "ragged": dict(T=77, d=384, E=5, k=3, f=256, C=300, head=250),
    "crowded": dict(T=200, d=256, E=12, k=2, f=128, crowd=5),
    "tiles": dict(T=300, d=640, E=2, k=1, f=512, C=320, head=100),
    "many_rows": dict(T=700, d=384, E=2, k=2, f=256),      # 256-row tiles
    "one_expert": dict(T=513, d=256, E=1, k=1, f=384),
    "empty_experts": dict(T=4, d=256, E=64, k=2, f=128),
    "whole_lines": dict(T=190, d=512, E=2, k=1, f=768, crowd=1),
    "long_rows": dict(T=90, d=2048, E=3, k=2, f=1280),
}


@pytest.mark.parametrize("name", list(EXPERTS))
def test_experts(name):
    print(f"\n[case] experts mxfp4 {name}", flush=True)
    c = Experts(**EXPERTS[name], seed=len(name))
    s = c.layer.shape
    ring, rs, off, y = c.run()
    torch.cuda.synchronize()
    d, f, C = s.hidden, s.ffn, s.capacity
    scale = np.repeat(2.0 ** (mx4.scale_rows(raw(rs)).astype(int) - 127), 32, axis=1)
    X, got, o = codes(ring) * scale, host(y), off.cpu().numpy()
    used = np.zeros(C, dtype=bool)
    for e in range(s.experts):
        at = (c.head + np.arange(o[e], o[e + 1])) % C
        used[at] = True
        if at.size == 0:
            continue
        x = X[at]
        wg, wu, wd = (c.W[n][2][e * r:(e + 1) * r] for n, r in (("gate", f), ("up", f), ("down", d)))
        A, U = x @ wg.T, x @ wu.T
        dA, dU = (SUM(d) * (abs(x) @ abs(w).T) + cut(x, w) for w in (wg, wu))
        h = mx4.swiglu(A, U)
        q, dq = h_bounds(h, 1.1 * abs(U) * dA + abs(mx4.swiglu(A, np.ones_like(A))) * dU + 2.0 ** -19 * abs(h))
        ref = q @ wd.T
        tol = dq @ abs(wd).T + cut(q, wd) + SUM(f) * (abs(q) @ abs(wd).T)
        within(got[at], ref, tol + HALF[BF] * (abs(ref) + tol), f"expert {e}")
    assert (got[~used] == 7).all()


@pytest.mark.parametrize("name", ["few", "ragged", "many_rows"])
def test_experts_are_the_mxfp8_layers(name):
    """The same weights as E4M3 codes through the MXFP8 layer: results agree to the roundings of H and y."""
    print(f"\n[case] experts mxfp4 = mxfp8 {name}", flush=True)
    c = Experts(**EXPERTS[name], seed=len(name))
    s = c.layer.shape
    ring, rs, off, y = c.run()
    y = y.clone()
    L8 = moe.Layer.create(s.tokens, s.hidden, s.experts, s.top_k, s.ffn, s.capacity, dtype="mxfp8", device=DEV)
    L8._buf("ring_y", (s.capacity, s.hidden), BF).fill_(7)
    y8, _ = L8.expert_ffn(ring, rs, off, c.head, *(as_e4m3(c.W[n][0]) for n in c.W), tuple(c.W[n][1] for n in c.W))
    torch.cuda.synchronize()
    print("  bits equal:", same_bits(y, y8), flush=True)
    assert np.linalg.norm(host(y) - host(y8)) <= 2.0 ** -7 * np.linalg.norm(host(y8))


def test_experts_in_a_graph():
    print("\n[case] expert_ffn mxfp4 graph", flush=True)
    c = Experts(**EXPERTS["long_rows"], seed=5)
    want = c.run()[3].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = c.run()[3]
    for _ in range(3):
        y.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(y, want)


def test_layer_serves_a_prompt_and_then_tokens():
    """Norm, routing, dispatch of the norm's 8-bit rows, experts and combine of a prompt, then decoded tokens, one layer's weights."""
    print("\n[case] mxfp4 layer", flush=True)
    g = gen(70)
    T, d, E, k, f = 60, 512, 16, 4, 256
    W = {n: weights(g, E, r, c) for n, r, c in (("gate", f, d), ("up", f, d), ("down", d, f))}
    w_r = randn(g, E, d, scale=d ** -0.5)
    router = moe.make_router(score="sigmoid", groups=4, top_groups=2, group_top=2, scale=2.0)
    norm_w = 1 + 0.1 * randn(g, d)
    x = randn(g, T, d, dtype=BF)
    prompt = moe.Layer.create(T, d, E, k, f, dtype="mxfp4", device=DEV)
    h, n, n8, n8s = prompt.add_rmsnorm(x, None, norm_w)
    names = ("gate", "up", "down")
    args = [w_r, None] + [W[m][0] for m in names]
    y = prompt.forward(n, *args, tuple(W[m][1] for m in names), router=router, x8=n8, x8_scale=n8s).clone()
    few = moe.Layer.create(8, d, E, k, f, dtype="mxfp4", device=DEV)
    for t0 in (0, 8, 52):
        rows = n[t0:t0 + 8].contiguous()
        yd, idx, gate = few.decode(rows, *args, scales=tuple(W[m][1] for m in names), router=router)
        torch.cuda.synchronize()
        assert torch.equal(idx, prompt.bufs["topk_idx"][t0:t0 + 8])      # (far from any tie)
        # the prompt's rows and H are rounded to 8 bits (2^-4 a value, averaged over d and f of them), the tokens' are not
        a, b = host(yd), host(y[t0:t0 + 8])
        assert np.linalg.norm(a - b) <= 2.0 ** -4 * np.linalg.norm(b)
    with pytest.raises(ValueError):
        moe.Layer.create(8, d, E, k, f, device=DEV).decode(n[:8], w_r, None, None, None, None, router=router)
