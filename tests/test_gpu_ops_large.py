"""GPU: the norm, scored router and FP8 calls at sizes where 32-bit offsets, grids or launches end:
sampled rows against fp64.  Tolerances as in test_gpu_norm.py, test_gpu_score.py and test_gpu_fp8.py."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_33_amd as moe
from oracle import ops
from ops_util import DEV, HALF, codes, gen, host, randn, same_bits, within
from test_gpu_fp8 import check_product, expert_case, experts, ffn_within, matmul
from test_gpu_score import R, backward, make, run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows_of(n, seed=0):
    """The ends, the places around 2^31 / 384 and 2^31 / 128 rows, and a few others."""
    near = [m for c in (0, (1 << 31) // 384, (1 << 31) // 128, n - 1) for m in (c - 1, c, c + 1) if 0 <= m < n]
    return torch.from_numpy(np.unique(near + list(np.random.default_rng(seed).integers(0, n, 24)))).to(DEV)


@pytest.mark.parametrize("ty", [BF, torch.float32])
def test_matmul_offsets_past_31_bits(ty):
    print(f"\n[case] matmul_fp8 large operands {ty}", flush=True)
    n, K, few = 8_500_000, 384, 24
    g = gen(1)
    big = torch.randint(0, 0x70, (n, K), generator=g, device=DEV, dtype=torch.uint8)
    big[::2] |= 0x80
    small, ss = moe.quantize_fp8(randn(g, few, K, dtype=BF), 1)
    sb = torch.rand((n + 127) // 128, K // 128, generator=g, device=DEV) + 0.5
    at = rows_of(n)
    # many weight rows: A few tokens, W the large one
    out = matmul(small, ss, big, sb, ty)
    sub = out[:, at]
    W = codes(big[at]) * np.repeat(host(sb[at // 128]), 128, axis=1)
    A = ops.spread_rows(codes(small), host(ss).T)
    ref, size = A @ W.T, abs(A) @ abs(W).T
    top = lambda v: abs(v).reshape(v.shape[0], -1, 8).max(2)  # noqa: E731
    cut = 7 * 2.0 ** -13 * (top(A) @ top(W).T) if ty == BF else 0
    within(host(sub), ref, HALF[ty] * abs(ref) + (132 + K / 128) * 2.0 ** -24 * size + cut, "large W")
    del out
    # many token rows: the same matrix as A, a scale per row
    sr = torch.rand(K // 128, n, generator=g, device=DEV) + 0.5
    w, sw = moe.quantize_fp8(randn(g, few, K, dtype=BF), 128)
    out = matmul(big, sr, w, sw, ty)
    check_product(out[at], big[at], sr[:, at], w, sw)


@pytest.mark.parametrize("counts,f", [([2, 0, 3], 128), ([1700, 1, 1803], 128)])
def test_experts_in_a_long_ring(counts, f):
    """Slots whose rows lie past 2^31 bytes, and the wrap to the ring's start."""
    print(f"\n[case] expert_ffn fp8 long ring {counts}", flush=True)
    C, n = 26_000_000, sum(counts)
    s, q, qs, slot, ring, rs, off, wt = expert_case(counts, 128, f, C - n // 2, 5, C=C)
    y, au = experts(s, ring, rs, off, C - n // 2, wt)
    lo = 0
    for e, c in enumerate(counts):
        if c:
            m = np.unique([0, c - 1, *np.random.default_rng(e).integers(0, c, 8)]) + lo
            W = [ops.spread_blocks(codes(w[e]), host(sw[e])) for w, sw in wt]
            ffn_within(host(y[slot[m]]), ops.spread_rows(codes(q[m]), host(qs[:, m]).T), W, f"expert {e}")
        lo += c
    other = torch.ones(C, dtype=torch.bool, device=DEV)
    other[slot] = False
    assert bool((y[other] == 7).all())


# a few rows; some hundreds (row tiles found from the offsets); many workgroups (row tiles from a list)
@pytest.mark.parametrize("rows,f,most", [(32, 128, 20), (330, 128, 70), (1500, 512, 130)])
def test_1024_experts(rows, f, most):
    print(f"\n[case] expert_ffn fp8 of 1,024 experts, {rows} rows", flush=True)
    rng = np.random.default_rng(rows)
    counts = np.zeros(1024, dtype=int)
    counts[[0, 15, 16, 500, 1023]] = 1, 2, 3, most, 5
    np.add.at(counts, rng.integers(0, 1024, rows - most), 1)
    s, q, qs, slot, ring, rs, off, wt = expert_case(list(counts), 128, f, 9, 6)
    y, _ = experts(s, ring, rs, off, 9, wt)
    starts = np.concatenate([[0], np.cumsum(counts)])
    for e in (0, 1, 15, 16, 63, 64, 499, 500, 501, 777, 1022, 1023):
        r = slice(starts[e], starts[e + 1])
        if counts[e]:
            W = [ops.spread_blocks(codes(w[e]), host(sw[e])) for w, sw in wt]
            ffn_within(host(y[slot[r]]), ops.spread_rows(codes(q[r]), host(qs[:, r]).T), W, f"expert {e}")
    # every row was written, and nothing else
    other = torch.ones(s.capacity, dtype=torch.bool, device=DEV)
    other[slot] = False
    assert bool((y[other] == 7).all()) and bool(y[slot].isfinite().all()) and bool((y[slot] != 7).any(1).all())


def test_norm_of_more_than_2_31_elements():
    print("\n[case] add_rmsnorm large", flush=True)
    T, d = 600_001, 4096
    s = moe.make_shape(T, d, 1, 1, 8, dtype="f32")
    x = torch.empty(T, d, device=DEV).normal_(generator=gen(1))
    w = 1 + randn(gen(2), d, scale=0.1)
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=DEV)
    moe.moe_add_rmsnorm(s, x, None, w, 1e-6, h, y, None, None, rstd)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, (1 << 31) // d - 1, (1 << 31) // d, (1 << 31) // d + 1, T - 1], device=DEV)
    X = host(x[at])
    y64, r64 = ops.add_rmsnorm(X, host(w), 1e-6)
    u = (d / 512 + 14) * 2.0 ** -24
    assert same_bits(h[at], x[at])
    within(host(rstd[at]), r64, u * r64, "rstd")
    within(host(y[at]), y64, (u + 2.0 ** -24) * abs(y64), "y")
    del h
    dx, dw = y, torch.empty(d, device=DEV)     # dy is y itself, in place
    dy = y[at].clone()
    moe.moe_add_rmsnorm_backward(s, y, None, x, w, rstd, dx, dw, moe.workspace(s, moe.OP_NORM_BACKWARD, DEV))
    torch.cuda.synchronize()
    r, q, xh = host(rstd[at])[:, None], host(dy) * host(w), X * host(rstd[at])[:, None]
    want = r * (q - xh * (q * xh).mean(1, keepdims=True))
    within(host(dx[at]), want, 2.0 ** -24 * r * (8 * abs(q) + (d / 256 + 30) * abs(xh) * abs(q * xh).mean(1, keepdims=True)), "dx")


@pytest.mark.parametrize("dtype,T,d,E,k", [("bf16", (1 << 18) + 77, 64, 8, 2), ("f32", (1 << 21), 8, 4, 1)])
def test_routing_of_many_tokens(dtype, T, d, E, k):
    print(f"\n[case] route_scored {dtype} {T} tokens", flush=True)
    act = torch.float32 if dtype == "f32" else BF
    rule = R("sigmoid", renormalise=False, scale=2.0)
    x, w = randn(gen(1), T, d, dtype=act), randn(gen(2), E, d) / 8
    s, idx, gate, cnt, logits = run(dtype, x, w, None, None, k, rule)
    l = x.double() @ w.double().T
    assert int(cnt.sum()) == T * k and torch.equal(cnt.long(), torch.bincount(idx.view(-1).long(), minlength=E))
    D = (d / 16 + 16) * 2.0 ** -24 * (x.double().abs() @ w.double().abs().T) + 2.0 ** -23 * l.abs()
    assert bool(((logits.double() - l).abs() <= D).all())
    picked = l.gather(1, idx.long())
    assert bool(((gate.double() - 2 * torch.sigmoid(picked)).abs() <= 2.0 ** -14).all())
    dg = randn(gen(3), T, k)
    dx, dw, db, _ = backward(dtype, s, rule, dg, None, x, w, logits, idx, None)
    sg = torch.sigmoid(logits.double().gather(1, idx.long()))
    dl = torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter_add_(1, idx.long(), 2 * dg.double() * sg * (1 - sg))
    want = dl @ w.double()
    tol = HALF[act] * want.abs() + 2.0 ** -13 * (dl.abs() @ w.double().abs()) + 1e-30
    assert bool(((dx.double() - want).abs() <= tol).all())
    # sums over T: some fp32 sum adds at most T / 16 + 80 terms in a row
    seq = 2.0 ** -16 + (T / 16 + 80) * 2.0 ** -24
    assert bool(((dw.double() - dl.T @ x.double()).abs() <= seq * (dl.abs().T @ x.double().abs())).all())
    assert bool(((db.double() - dl.sum(0)).abs() <= seq * dl.abs().sum(0)).all())
