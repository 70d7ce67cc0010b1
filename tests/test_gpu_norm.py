"""GPU: residual add + RMS norm and its gradient against the fp64 oracle.

Tolerances.  A row's sum of squares adds, in some thread, at most d / 256 + 8 terms one after
another, then a tree over 64 lanes and 4 wavefronts, each step off by at most 2^-24 of the (positive) sum; the
root halves that, and mean, root, reciprocal and the two products of y add at most five more:
y and rstd are within (d / 512 + 14) 2^-24 of the oracle's, relative, before y's own rounding."""
import pytest
import torch

import mixture_experts_layer_33_amd as moe
from oracle import ops
from ops_util import DEV, HALF, codes, gen, host, randn, same_bits, within

pytestmark = pytest.mark.gpu
EPS = 1e-6


def shape(T, d, dtype):
    return moe.make_shape(T, d, 8, 1, 128, dtype=dtype)


def u(d):
    return (d / 512 + 14) * 2.0 ** -24


def forward(dtype, T, d, seed=0, residual=True, y8=True, x=None, alias=None):
    g = gen(seed)
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    x = randn(g, T, d, dtype=act) if x is None else x
    r = randn(g, T, d, dtype=act, scale=3.0) if residual else None
    w = 1 + randn(g, d, scale=0.1)
    s = shape(T, d, dtype)
    keep = (x.clone(), None if r is None else r.clone())
    h = {"x": x, "r": r}.get(alias, torch.full_like(x, 7))
    y, rstd = torch.full_like(x, 7), torch.full((T,), 7.0, device=DEV)
    q = qs = None
    if y8 and dtype in ("fp8", "mxfp8"):
        q = torch.full((T, d), 7, dtype=torch.uint8, device=DEV)
        qs = torch.zeros((d // 128, T) if dtype == "fp8" else (d // 128, T, 4), device=DEV,
                         dtype=torch.float32 if dtype == "fp8" else torch.uint8)
    moe.moe_add_rmsnorm(s, x, r, w, EPS, h, y, q, qs, rstd)
    torch.cuda.synchronize()
    return keep, w, h, y, q, qs, rstd


SIZES = [("bf16", 1, 64), ("bf16", 3, 448), ("bf16", 5, 512), ("bf16", 7, 576), ("bf16", 33, 2048), ("bf16", 4, 4096),
         ("bf16", 9, 7168), ("bf16", 2, 8192), ("bf16", 3, 8256), ("bf16", 2, 32768), ("f32", 1, 8), ("f32", 5, 40), ("f32", 6, 520),
         ("f32", 3, 2056), ("f32", 2, 4104), ("f32", 2, 12288), ("fp8", 1, 128), ("fp8", 5, 640), ("fp8", 66, 2176), ("fp8", 9, 7168),
         ("fp8", 2, 16512), ("mxfp8", 3, 128), ("mxfp8", 65, 1152), ("mxfp8", 3, 7168), ("mxfp8", 2, 8320)]


@pytest.mark.parametrize("dtype,T,d", SIZES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward(dtype, T, d, residual):
    print(f"\n[case] add_rmsnorm {dtype} {T}x{d} residual={residual}", flush=True)
    (x, r), w, h, y, q, qs, rstd = forward(dtype, T, d, residual=residual)
    want_h = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert same_bits(h, want_h)
    y64, rstd64 = ops.add_rmsnorm(host(want_h), host(w), EPS)
    within(host(rstd), rstd64, u(d) * rstd64, "rstd")
    within(host(y), y64, (u(d) + HALF[y.dtype]) * abs(y64), "y")
    if q is None:
        return
    if dtype == "fp8":
        s64 = host(qs).T
        _, want = ops.quantise_rows(y64)
        within(s64, want, (u(d) + 2.0 ** -23) * want, "scales")
        # half an E4M3 step (2^-10 of the scale below the normal range), the scale's own error
        within(ops.spread_rows(codes(q), s64), y64, (2.0 ** -4 + 2 * u(d) + 2.0 ** -22) * abs(y64) + 2.0 ** -9.9 * s64.repeat(128, 1), "y8")
    else:
        X = 2.0 ** (host(qs).transpose(1, 0, 2).reshape(T, d // 32) - 127)
        am = abs(y64).reshape(T, d // 32, 32).max(2)
        # E8M0: 2^floor(log2 amax) / 256, one binade either way only where amax is next to a power of two
        lo, hi = am * (1 - 2 * u(d)), am * (1 + 2 * u(d))
        import numpy as np
        assert ((X >= 2.0 ** (np.floor(np.log2(lo)) - 8)) & (X <= 2.0 ** (np.floor(np.log2(hi)) - 8))).all()
        X = X.repeat(32, 1)
        got = codes(q) * X
        # a block's largest values saturate at 448 X: up to 511 X is cut by 64 X, an eighth of it
        tol = np.where(abs(y64) > 448 * X, abs(y64) - 448 * X + 2.0 ** -18 * abs(y64), (2.0 ** -4 + 2 * u(d)) * abs(y64) + 2.0 ** -9.9 * X)
        within(got, y64, tol, "y8")


@pytest.mark.parametrize("dtype,d", [("bf16", 448), ("bf16", 2048), ("bf16", 8256), ("f32", 520)])
@pytest.mark.parametrize("alias", ["x", "r"])
def test_h_in_place(dtype, d, alias):
    """h written over x or over the residual gives what a buffer of its own gives."""
    print(f"\n[case] add_rmsnorm in place {dtype} {d} {alias}", flush=True)
    a, b = forward(dtype, 5, d), forward(dtype, 5, d, alias=alias)
    for i in (2, 3, 6):
        assert same_bits(a[i], b[i])


def test_outputs_left_out():
    print("\n[case] add_rmsnorm without y / h / rstd", flush=True)
    (x, r), w, h, y, q, qs, rstd = forward("fp8", 6, 640)
    s = shape(6, 640, "fp8")
    q2, qs2 = torch.empty_like(q), torch.empty_like(qs)
    moe.moe_add_rmsnorm(s, x, r, w, EPS, None, None, q2, qs2, None)
    y2 = torch.empty_like(y)
    moe.moe_add_rmsnorm(s, x, r, w, EPS, None, y2, None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and same_bits(qs, qs2) and same_bits(y, y2)


@pytest.mark.parametrize("dtype", ["fp8", "mxfp8"])
def test_zero_tiny_and_broken_rows(dtype):
    """A row of zeros, a subnormal one, one with a NaN, one with an infinity: the other rows are untouched."""
    print(f"\n[case] add_rmsnorm special rows {dtype}", flush=True)
    d = 384
    x = randn(gen(3), 6, d, dtype=torch.bfloat16)
    x[1] = 0
    x[2] = 2.0 ** -130
    x[3, 200] = float("nan")
    x[4, 300] = float("inf")
    (x0, _), w, h, y, q, qs, rstd = forward(dtype, 6, d, x=x.clone(), residual=False)
    assert same_bits(h, x0)
    assert (y[1] == 0).all() and (q[1] & 0x7f == 0).all()
    assert rstd[1].item() == pytest.approx(EPS ** -0.5, rel=1e-6)
    assert torch.isnan(y[3]).all() and y[2].isfinite().all()
    assert y[4, 300].isnan() and (y[4, :300] == 0).all()         # inf * 0 of the row's rstd = 0
    scale = qs if dtype == "fp8" else qs.float()
    nan = torch.isnan(scale) if dtype == "fp8" else (qs == 255)
    rows = nan.any(0) if dtype == "fp8" else nan.any(0).any(-1)
    assert rows.tolist() == [False, False, False, True, True, False]
    good = [0, 5]
    _, _, _, y1, q1, qs1, _ = forward(dtype, 2, d, x=x0[good].clone(), residual=False)
    assert same_bits(y[good], y1) and torch.equal(q[good], q1)


BWD = [("bf16", 1, 64), ("bf16", 7, 576), ("bf16", 600, 2048), ("bf16", 33, 4096), ("bf16", 1030, 7168), ("bf16", 5, 8256),
       ("bf16", 700, 16448), ("f32", 1, 8), ("f32", 513, 520), ("f32", 40, 4104), ("f32", 3, 12288)]


@pytest.mark.parametrize("dtype,T,d", BWD)
@pytest.mark.parametrize("with_dh", [True, False])
def test_backward(dtype, T, d, with_dh):
    """dx: its own rounding, and the fp32 terms (the mean of q xh is off by at most (d / 256 + 16)
    steps of its terms' sizes).  dw: each of at most 512 partials adds T / 512 rows, then a quarter
    of them are added one after another: at most T / 512 + 132 steps of the terms' sizes."""
    print(f"\n[case] rmsnorm backward {dtype} {T}x{d} dh={with_dh}", flush=True)
    g = gen(T + d)
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    h, dy = randn(g, T, d, dtype=act, scale=3.0), randn(g, T, d, dtype=act)
    dh = randn(g, T, d, dtype=act) if with_dh else None
    w = 1 + randn(g, d, scale=0.1)
    s = shape(T, d, dtype)
    rstd = torch.from_numpy(ops.add_rmsnorm(host(h), host(w), EPS)[1]).float().to(DEV)
    dx, dw = torch.full_like(h, 7), torch.full((d,), 7.0, device=DEV)
    ws = moe.workspace(s, moe.OP_NORM_BACKWARD, DEV)
    moe.moe_add_rmsnorm_backward(s, dy, dh, h, w, rstd, dx, dw, ws)
    H, DY, W, R = host(h), host(dy), host(w), host(rstd)
    dx64, dw64 = ops.add_rmsnorm_backward(DY, None if dh is None else host(dh), H, W, R)
    xh, q = H * R[:, None], DY * W
    size = 0 if dh is None else abs(host(dh))
    size = size + R[:, None] * (abs(q) + abs(xh) * abs(q * xh).mean(1, keepdims=True))
    within(host(dx), dx64, HALF[act] * abs(dx64) + (d / 256 + 16) * 2.0 ** -24 * size, "dx")
    within(host(dw), dw64, (T / 512 + 136) * 2.0 ** -24 * abs(DY * xh).sum(0) + 1e-30, "dw")
    # the same in place, twice, and without dw
    dx2, dw2 = dy.clone(), torch.empty_like(dw)
    moe.moe_add_rmsnorm_backward(s, dx2, dh, h, w, rstd, dx2, dw2, ws)
    assert same_bits(dx, dx2) and same_bits(dw, dw2)
    dx3 = torch.empty_like(dx)
    moe.moe_add_rmsnorm_backward(s, dy, dh, h, w, rstd, dx3, None, ws)
    torch.cuda.synchronize()
    assert same_bits(dx, dx3)


def test_gradient_against_differences():
    """fp32 layer: the gradient along random directions against central differences of the fp64 oracle."""
    print("\n[case] rmsnorm gradient against differences", flush=True)
    g = gen(11)
    T, d = 6, 40
    x, r, dy, dh, w = (randn(g, T, d) for _ in range(4)), None, None, None, 1 + randn(g, d, scale=0.1)
    x, r, dy, dh = x
    s = shape(T, d, "f32")
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=DEV)
    moe.moe_add_rmsnorm(s, x, r, w, EPS, h, y, None, None, rstd)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    moe.moe_add_rmsnorm_backward(s, dy, dh, h, w, rstd, dx, dw, moe.workspace(s, moe.OP_NORM_BACKWARD, DEV))
    H, W = host(x) + host(r), host(w)
    f = lambda a, b: (ops.add_rmsnorm(a, b, EPS)[0] * host(dy)).sum() + (a * host(dh)).sum()  # noqa: E731
    for k in range(3):
        a, b = host(randn(g, T, d)), host(randn(g, d))
        e = 1e-6
        want = (f(H + e * a, W + e * b) - f(H - e * a, W - e * b)) / (2 * e)
        got = (host(dx) * a).sum() + (host(dw) * b).sum()
        assert got == pytest.approx(want, rel=1e-5, abs=1e-4)


def test_no_rows():
    print("\n[case] rmsnorm of no rows", flush=True)
    s = shape(0, 256, "bf16")
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    w, dw = torch.ones(256, device=DEV), torch.full((256,), 7.0, device=DEV)
    moe.moe_add_rmsnorm(s, e, None, w, EPS, None, e, None, None, None)
    moe.moe_add_rmsnorm_backward(s, e, None, e, w, torch.empty(0, device=DEV), e, dw, None)
    assert (dw == 0).all()


def test_other_stream_and_graph():
    """A call on a side stream, and replays of a captured forward and backward between eager ones."""
    print("\n[case] rmsnorm side stream and graph", flush=True)
    T, d = 40, 2048
    (x, r), w, h, y, q, qs, rstd = forward("fp8", T, d)
    s = shape(T, d, "fp8")
    ws = moe.workspace(s, moe.OP_NORM_BACKWARD, DEV)
    h2, y2, q2, qs2, rstd2 = (torch.zeros_like(t) for t in (h, y, q, qs, rstd))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_add_rmsnorm(s, x, r, w, EPS, h2, y2, q2, qs2, rstd2, stream=side)
    side.synchronize()
    assert same_bits(y, y2) and torch.equal(q, q2)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_add_rmsnorm(s, x, r, w, EPS, h2, y2, q2, qs2, rstd2)
        moe.moe_add_rmsnorm_backward(s, y2, None, h2, w, rstd2, dx, dw, ws)
    for k in range(4):
        x.copy_(randn(gen(100 + k), T, d, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h2, y2, q2, qs2, dx, dw)]
        moe.moe_add_rmsnorm(s, x, r, w, EPS, h2, y2, q2, qs2, rstd2)
        moe.moe_add_rmsnorm_backward(s, y2, None, h2, w, rstd2, dx, dw, ws)
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(got, (h2, y2, q2, qs2, dx, dw)))
