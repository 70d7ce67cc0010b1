"""GPU: scored routing (softmax / sigmoid, balance, groups, renormalisation) and its gradient
against the fp64 oracle.

Tolerances.  A logit's d products are exact (bf16 times three bf16 planes of W_r) or off by one step
(fp32 x), and some fp32 sum adds at most d / 16 + 16 of them one after another: it is off by at most
(d / 16 + 16) 2^-24 sum |x w| =: D.  A score's relative error is then at most 2 D (softmax; its
sum moves too) or D, a renormalised gate's at most 4 D, and exp, sums over E and divisions add
fewer than 2^8 steps of 2^-24."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_33_amd as moe
from oracle import ops
from ops_util import DEV, HALF, gen, host, randn, same_bits, within

pytestmark = pytest.mark.gpu


def make(rule):
    return moe.make_router(rule.score, rule.groups, rule.top_groups, rule.group_top, rule.renormalise, rule.scale)


def draw(dtype, T, d, E, k, rule, seed, balanced, biased=False):
    """Tokens whose choice is clear of a tie by 1e-4 of the deciding values' size."""
    g = gen(seed)
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    w = randn(g, E, d) / d ** 0.5
    b = randn(g, E, scale=0.3) if biased else None
    bal = randn(g, E) * (0.05 if rule.score == "sigmoid" else 0.3 / E) if balanced else None
    x = randn(g, 2 * T + 32, d, dtype=act)
    l = host(x) @ host(w).T + (0 if b is None else host(b))
    near = ops.margins(l, rule, k, None if bal is None else host(bal))
    floor = 1e-4 if rule.score == "sigmoid" or not (balanced or rule.top_groups < rule.groups) else 1e-4 / E
    take = np.nonzero(near > floor)[0][:T]
    assert take.size == T
    return x[torch.from_numpy(take).to(DEV)].contiguous(), w, b, bal, l[take]


def run(dtype, x, w, b, bal, k, rule, ws=None, want_logits=True):
    T, d = x.shape
    E = w.shape[0]
    s = moe.make_shape(T, d, E, k, 128, dtype=dtype)
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    gate = torch.full((T, k), -7.0, device=DEV)
    cnt = torch.full((E,), -7, dtype=torch.int32, device=DEV)
    logits = torch.full((T, E), -7.0, device=DEV) if want_logits else None
    moe.moe_route_scored(s, make(rule), x, w, b, bal, idx, gate, cnt, logits, moe.workspace(s, moe.OP_ROUTE, DEV) if ws is None else ws)
    torch.cuda.synchronize()
    return s, idx, gate, cnt, logits


R = ops.Rule
CASES = [  # dtype, T, d, E, k, rule
    ("bf16", 1, 64, 8, 2, R()), ("bf16", 5, 256, 8, 8, R(renormalise=False, scale=2.0)), ("bf16", 70, 512, 60, 6, R("sigmoid", scale=2.5)),
    ("bf16", 130, 256, 64, 4, R("softmax", 8, 3, 1, False)), ("bf16", 33, 512, 160, 6, R("softmax", 8, 3, 1, False, 16.0)),
    ("bf16", 9, 1024, 256, 8, R("sigmoid", 8, 4, 2, True, 2.5)), ("bf16", 300, 256, 256, 8, R("sigmoid", 8, 4, 2, True, 2.5)),
    ("fp8", 17, 256, 256, 8, R("sigmoid", 8, 4, 2, True, 2.5)), ("mxfp8", 6, 128, 72, 5, R("sigmoid", 3, 2, 2, False)),
    ("bf16", 2, 192, 1024, 32, R("softmax", 64, 17, 2)), ("bf16", 64, 64, 1, 1, R()), ("bf16", 40, 128, 33, 32, R("sigmoid", 11, 11, 2)),
    ("bf16", 7, 128, 500, 10, R("sigmoid", 50, 7, 1)), ("f32", 19, 72, 16, 4, R("sigmoid", 4, 2, 2, True, 2.5)), ("f32", 66, 128, 130, 3, R(renormalise=False)),
]
CASES += [("bf16", 9, 7168, 256, 8, R("sigmoid", 8, 4, 2, True, 2.5)), ("bf16", 100, 4096, 512, 10, R(renormalise=False)),
          ("bf16", 65, 2048, 1000, 16, R("sigmoid", 10, 5, 2, True)), ("bf16", 31, 1024, 70, 4, R("softmax", 7, 3, 2, False))]
IDS = [f"{c[0]}-{c[1]}x{c[2]}-E{c[3]}k{c[4]}-{c[5].score}{c[5].groups}.{c[5].top_groups}.{c[5].group_top}{'r' if c[5].renormalise else ''}" for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("balanced", [False, True])
def test_forward(case, balanced):
    dtype, T, d, E, k, rule = case
    print(f"\n[case] route_scored {case} balanced={balanced}", flush=True)
    x, w, b, bal, l = draw(dtype, T, d, E, k, rule, 5 + E, balanced, biased=E % 2 == 0)
    _, idx, gate, cnt, logits = run(dtype, x, w, b, bal, k, rule)
    D = (d / 16 + 16) * 2.0 ** -24 * (abs(host(x)) @ abs(host(w)).T) + 2.0 ** -23 * abs(l)
    within(host(logits), l, D, "logits")
    want = ops.choose(l, rule, k, None if bal is None else host(bal))
    assert np.array_equal(idx.cpu().numpy(), want)
    assert np.array_equal(cnt.cpu().numpy(), np.bincount(want.ravel(), minlength=E))
    g = ops.gates(l, want, rule)
    within(host(gate), g, abs(g) * (4 * D.max() + 2.0 ** -16), "gates")
    _, idx2, gate2, cnt2, _ = run(dtype, x, w, b, bal, k, rule, want_logits=False)
    assert torch.equal(idx, idx2) and same_bits(gate, gate2) and torch.equal(cnt, cnt2)


# 128 x 128 tiles of the logits: one to many slices of 64, with K splits, ragged tiles
LOTS = [("bf16", 16500, 64, 130, 4, R("sigmoid")), ("bf16", 8200, 128, 257, 3, R()), ("bf16", 8200, 192, 260, 6, R("sigmoid", 4, 2, 2)),
        ("bf16", 8321, 320, 300, 2, R(renormalise=False)), ("bf16", 5000, 1088, 300, 8, R("sigmoid", 10, 5, 1)), ("bf16", 2048, 3136, 256, 8, R("sigmoid", 8, 4, 2, True, 2.5))]


@pytest.mark.parametrize("case", LOTS, ids=[f"{c[1]}x{c[2]}-E{c[3]}" for c in LOTS])
def test_forward_of_many_tokens(case):
    test_forward(case, True)


def test_softmax_without_groups_is_the_plain_router():
    """The rule that moe_route has gives its choice bit for bit, and its gates within rounding."""
    print("\n[case] route_scored against route", flush=True)
    for T, d, E, k in ((50, 256, 64, 8), (300, 512, 256, 8)):
        x, w, _, _, _ = draw("bf16", T, d, E, k, R(), E, False)
        s, idx, gate, cnt, _ = run("bf16", x, w, None, None, k, R())
        layer = moe.Layer.create(T, d, E, k, 128)
        i, g, c = layer.route(x, w)
        torch.cuda.synchronize()
        assert torch.equal(i, idx) and torch.equal(c, cnt)
        assert torch.allclose(g, gate, rtol=1e-5, atol=0)


def exact_logits(l, E):
    """x, W_r whose logits are l exactly (l in halves): W_r = identity rows."""
    T = l.shape[0]
    x = torch.zeros(T, 64 * ((E + 63) // 64), dtype=torch.bfloat16, device=DEV)
    x[:, :E] = torch.from_numpy(l).to(DEV).bfloat16()
    return x, torch.eye(E, x.shape[1], device=DEV)


@pytest.mark.parametrize("rule", [R(), R("sigmoid"), R("sigmoid", 4, 2, 2), R("softmax", 4, 2, 1, False), R("sigmoid", 8, 3, 1)], ids=str)
def test_ties(rule):
    """Logits drawn from three values: nearly every choice is a tie, of experts and of groups."""
    print(f"\n[case] route_scored ties {rule}", flush=True)
    l = np.random.default_rng(1).choice([-0.5, 0.0, 1.0], size=(200, 32))
    l[0] = 0
    x, w = exact_logits(l, 32)
    _, idx, gate, _, logits = run("bf16", x, w, None, None, 4, rule)
    assert np.array_equal(host(logits), l)
    # the fp32 scores of equal logits are equal, and sums of two of these three values tie only if the values do
    want = ops.choose(np.float32(l).astype(np.float64), rule, 4)
    assert np.array_equal(idx.cpu().numpy(), want)
    g = ops.gates(l, want, rule)
    within(host(gate), g, abs(g) * 2.0 ** -16, "gates")


def test_masks_and_what_is_not_a_number():
    print("\n[case] route_scored masks", flush=True)
    E, k, inf, nan = 16, 3, float("inf"), float("nan")
    x, w, _, _, l = draw("bf16", 12, 64, E, k, R(), 3, False)
    lowest = torch.finfo(torch.float32).min
    for rule in (R(), R("sigmoid", scale=2.0), R(renormalise=False), R("sigmoid", renormalise=False), R("sigmoid", 4, 2, 2)):
        # -inf in the bias takes experts out; all but two out leaves a place that nothing can fill: gate 0
        for out in (inf, -lowest):
            b = torch.zeros(E, device=DEV)
            b[2:] = -out
            _, idx, gate, _, _ = run("bf16", x, w, b, None, k, rule)
            assert idx[:, :2].tolist() == [[0, 1]] * 12
            if out == inf:
                assert (gate[:, 2] == 0).all()
                lm = l + host(b)
                g = ops.gates(lm, idx.cpu().numpy().astype(np.int64), rule)
                within(host(gate), g, abs(g) * 2.0 ** -12, "gates")
            assert gate.isfinite().all()
        # every expert out: valid ids, gates 0
        _, idx, gate, cnt, _ = run("bf16", x, w, torch.full((E,), -inf, device=DEV), None, k, rule)
        assert idx.tolist() == [[0, 1, 2]] * 12 and (gate == 0).all() and int(cnt.sum()) == 36
        # a balance of -inf moves the choice only: the gate is still the score's
        bal = torch.zeros(E, device=DEV)
        bal[5:] = -inf
        _, idx, gate, _, _ = run("bf16", x, w, None, bal, k, rule)
        assert (idx < 5).all() if rule.groups == 1 else True
        assert (gate > 0).all()
        # NaN: valid distinct ids whatever the row holds, the other rows as before
        y = x.clone()
        y[4, 0] = nan
        y[7, 1] = inf
        _, i1, g1, c1, _ = run("bf16", y, w, None, None, k, rule)
        _, i0, g0, _, _ = run("bf16", x, w, None, None, k, rule)
        assert (i1 >= 0).all() and (i1 < E).all() and (i1[:, 1:] > i1[:, :-1]).all() and int(c1.sum()) == 36
        rest = [t for t in range(12) if t not in (4, 7)]
        assert torch.equal(i1[rest], i0[rest]) and same_bits(g1[rest], g0[rest])


def backward(dtype, s, rule, dg, dlog, x, w, logits, idx, dx_in, db=True):
    T, d = x.shape
    E = w.shape[0]
    dx = torch.full_like(x, 7)
    dw, dbv = torch.full((E, d), 7.0, device=DEV), torch.full((E,), 7.0, device=DEV) if db else None
    ws = moe.workspace(s, moe.OP_ROUTE_BACKWARD, DEV)
    moe.moe_route_scored_backward(s, make(rule), dg, dlog, x, w, logits, idx, dx_in, dx, dw, dbv, ws)
    torch.cuda.synchronize()
    return dx, dw, dbv, ws


BCASES = CASES + [("bf16", 16, 320, 1000, 32, R(renormalise=False)), ("bf16", 16, 128, 64, 2, R("sigmoid")), ("bf16", 17, 128, 128, 2, R()),
                  ("bf16", 3000, 128, 72, 4, R(renormalise=False)), ("bf16", 700, 512, 160, 6, R(renormalise=False)), ("bf16", 257, 320, 512, 10, R("sigmoid")), ("f32", 300, 72, 40, 4, R("sigmoid"))]
BIDS = [f"{c[0]}-{c[1]}x{c[2]}-E{c[3]}k{c[4]}-{c[5].score}{'r' if c[5].renormalise else ''}" for c in BCASES]


@pytest.mark.parametrize("case", BCASES, ids=BIDS)
@pytest.mark.parametrize("more", [False, True])
def test_backward(case, more):
    """dl: within 2^-16 of its terms' sizes (exp, sums over E, divisions: fewer than 2^8 steps).
    dx: that error through W_r, dl and W_r taken to 2^-16 each (two bf16 parts, a bf16 rounding being off by
    2^-8 at most, or fp32) and the product of the two second parts (2^-16) left out, fp32 sums over E,
    its own rounding.  dW_r and db: dl's error, and fp32 sums over T (at most T / 16 + 80 in a row)."""
    dtype, T, d, E, k, rule = case
    print(f"\n[case] route_scored backward {case} more={more}", flush=True)
    x, w, _, _, l = draw(dtype, T, d, E, k, rule, 9 + E, False)
    g = gen(T)
    s = moe.make_shape(T, d, E, k, 128, dtype=dtype)
    idx = torch.from_numpy(ops.choose(l, rule, k)).to(DEV, torch.int32)
    logits = torch.from_numpy(l).float().to(DEV)
    dg = randn(g, T, k)
    dlog = randn(g, T, E, scale=0.01) if more else None
    dx_in = randn(g, T, d, dtype=x.dtype) if more else None
    dx, dw, db, ws = backward(dtype, s, rule, dg, dlog, x, w, logits, idx, dx_in)
    L, I = host(logits), idx.cpu().numpy().astype(np.int64)
    dl = ops.gates_backward(host(dg), L, I, rule)
    size = np.abs(ops.gates_backward(np.abs(host(dg)), L, I, rule)) + 2 * np.abs(rule.scale) * np.abs(host(dg)).max(1, keepdims=True) * (
        ops.scores(L, rule) if rule.score == "softmax" and not rule.renormalise else 0)
    if rule.renormalise or rule.score == "sigmoid":
        big = np.zeros_like(dl)
        np.put_along_axis(big, I, 2 * np.abs(ops.gates(L, I, rule)) * np.abs(host(dg)).max(1, keepdims=True), axis=1)
        size = size + big
    err = 2.0 ** -16 * size
    if more:
        dl = dl + host(dlog)
        size = size + abs(host(dlog))
    X, W = host(x), host(w)
    dx64, dw64 = dl @ W, dl.T @ X
    tol = (err + 3 * 2.0 ** -16 * size + (E / 16 + 16) * 2.0 ** -24 * size) @ abs(W)
    if more:
        dx64 = dx64 + host(dx_in)
        tol = tol + 2.0 ** -22 * abs(host(dx_in))
    within(host(dx), dx64, HALF[x.dtype] * abs(dx64) + tol + 1e-30, "dx")
    seq = (T / 16 + 80) * 2.0 ** -24
    within(host(dw), dw64, (err + seq * size).T @ abs(X) + 1e-30, "dw")
    within(host(db), dl.sum(0), (err + seq * size).sum(0) + 1e-30, "db")
    if more:   # in place, again, without db
        dx2, dw2 = dx_in.clone(), torch.empty_like(dw)
        moe.moe_route_scored_backward(s, make(rule), dg, dlog, x, w, logits, idx, dx2, dx2, dw2, None, ws)
        torch.cuda.synchronize()
        assert same_bits(dx, dx2) and same_bits(dw, dw2)


# sizes at which dx is built from taller tiles
MANY = [("bf16", 4100, 1024, 64, 6, R("sigmoid")), ("bf16", 5000, 1600, 40, 4, R()), ("bf16", 6001, 2112, 64, 4, R(renormalise=False))]


@pytest.mark.parametrize("case", MANY, ids=[f"{c[1]}x{c[2]}" for c in MANY])
def test_backward_of_many_tokens(case):
    test_backward(case, True)


def test_vectors_at_an_element_s_alignment():
    """Biases, counts, gates and ids may start at any element."""
    print("\n[case] route_scored alignment", flush=True)
    rule = R("sigmoid", 4, 2, 2, True, 2.5)
    for T in (3, 70):
        d, E, k = 128, 160, 3
        x, w, b, bal, _ = draw("bf16", T, d, E, k, rule, 6, True, biased=True)
        s, idx, gate, cnt, logits = run("bf16", x, w, b, bal, k, rule)
        dg, dlog = randn(gen(1), T, k), randn(gen(2), T, E)
        want = backward("bf16", s, rule, dg, dlog, x, w, logits, idx, None)

        def shift(t):
            buf = torch.full((t.numel() + 8,), 7, dtype=t.dtype, device=DEV)
            o = buf[1:1 + t.numel()].view(t.shape)
            o.copy_(t)
            return o, buf
        (b1, _), (bal1, _), (dg1, _) = shift(b), shift(bal), shift(dg)
        out = [shift(torch.zeros_like(t)) for t in (idx, gate, cnt)]
        moe.moe_route_scored(s, make(rule), x, w, b1, bal1, *(o for o, _ in out), None, moe.workspace(s, moe.OP_ROUTE, DEV))
        torch.cuda.synchronize()
        for (o, buf), ref in zip(out, (idx, gate, cnt)):
            assert torch.equal(o, ref) and buf[0] == 7 and (buf[1 + o.numel():] == 7).all()
        db, buf = shift(torch.zeros(E, device=DEV))
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        moe.moe_route_scored_backward(s, make(rule), dg1, dlog, x, w, logits, out[0][0], None, dx, dw, db, moe.workspace(s, moe.OP_ROUTE_BACKWARD, DEV))
        torch.cuda.synchronize()
        assert same_bits(dx, want[0]) and same_bits(dw, want[1]) and same_bits(db, want[2]) and buf[0] == 7 and (buf[1 + E:] == 7).all()


def test_two_routers_at_once():
    """Two calls on two streams, each with its own workspace, forward and backward."""
    print("\n[case] route_scored two streams", flush=True)
    rule = R("sigmoid", 8, 4, 2, True, 2.5)
    work = []
    for T in (5, 300):
        x, w, _, bal, _ = draw("bf16", T, 256, 64, 6, rule, T, True)
        s, idx, gate, cnt, logits = run("bf16", x, w, None, bal, 6, rule)
        dg = randn(gen(T), T, 6)
        want = (idx, gate, cnt, logits, *backward("bf16", s, rule, dg, None, x, w, logits, idx, x)[:3])
        work.append((s, x, w, bal, dg, want, [torch.zeros_like(t) for t in want], moe.workspace(s, moe.OP_ROUTE, DEV),
                     moe.workspace(s, moe.OP_ROUTE_BACKWARD, DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, x, w, bal, dg, _, o, ws, wb, st in work:
            moe.moe_route_scored(s, make(rule), x, w, None, bal, *o[:4], ws, stream=st)
            moe.moe_route_scored_backward(s, make(rule), dg, None, x, w, o[3], o[0], x, *o[4:], wb, stream=st)
    torch.cuda.synchronize()
    for v in work:
        assert all(same_bits(a, c) for a, c in zip(v[5], v[6]))


@pytest.mark.parametrize("rule", [R(), R(renormalise=False), R("sigmoid"), R("sigmoid", renormalise=False, scale=2.5)], ids=str)
def test_gradient_against_differences(rule):
    """fp32 layer: x, W_r and b_r along random directions against central differences of the oracle's gates."""
    print(f"\n[case] route_scored differences {rule}", flush=True)
    T, d, E, k = 6, 24, 16, 3
    x, w, b, _, l = draw("f32", T, d, E, k, rule, 21, False, biased=True)
    s, idx, gate, _, logits = run("f32", x, w, b, None, k, rule)
    dg = randn(gen(5), T, k)
    dx, dw, db, _ = backward("f32", s, rule, dg, None, x, w, logits, idx, None)
    X, W, B, I = host(x), host(w), host(b), idx.cpu().numpy().astype(np.int64)
    f = lambda a, c, e: (ops.gates(a @ c.T + e, I, rule) * host(dg)).sum()  # noqa: E731
    r = np.random.default_rng(2)
    for _ in range(3):
        a, c, e = r.normal(size=X.shape), r.normal(size=W.shape), r.normal(size=E)
        h = 1e-5
        want = (f(X + h * a, W + h * c, B + h * e) - f(X - h * a, W - h * c, B - h * e)) / (2 * h)
        got = (host(dx) * a).sum() + (host(dw) * c).sum() + (host(db) * e).sum()
        assert got == pytest.approx(want, rel=2e-4, abs=2e-4)


def test_backward_of_masked_rows_and_odd_ids():
    print("\n[case] route_scored backward masks", flush=True)
    T, d, E, k = 10, 64, 16, 3
    for rule in (R(), R("sigmoid"), R(renormalise=False), R("sigmoid", renormalise=False)):
        x, w, _, _, l = draw("bf16", T, d, E, k, rule, 4, False)
        s = moe.make_shape(T, d, E, k, 128)
        l = l.copy()
        l[3] = -np.inf
        l[4, 2:] = -np.inf
        idx = ops.choose(l, rule, k)
        logits = torch.from_numpy(l).float().to(DEV)
        dg = randn(gen(1), T, k)
        it = torch.from_numpy(idx).to(DEV, torch.int32)
        dx, dw, db, _ = backward("bf16", s, rule, dg, None, x, w, logits, it, None)
        assert dx.isfinite().all() and dw.isfinite().all() and (dx[3] == 0).all()
        want = ops.gates_backward(host(dg), l, idx, rule) @ host(w)
        within(host(dx), want, 2.0 ** -7 * abs(want) + 1e-4, "dx")
        # ids outside [0, E) are left out (the gate is then another one: only that nothing else is touched)
        it2 = it.clone()
        it2[5, 0], it2[6, 2] = -1, E
        dx2, dw2, _, _ = backward("bf16", s, rule, dg, None, x, w, logits, it2, None)
        rest = [t for t in range(T) if t not in (5, 6)]
        assert same_bits(dx[rest], dx2[rest]) and dx2.isfinite().all() and dw2.isfinite().all()


def test_no_tokens():
    print("\n[case] route_scored of no tokens", flush=True)
    s = moe.make_shape(0, 64, 16, 2, 128)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(16, 64, device=DEV)
    idx, f = torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV)
    cnt, dw, db = torch.full((16,), 7, dtype=torch.int32, device=DEV), torch.full((16, 64), 7.0, device=DEV), torch.full((16,), 7.0, device=DEV)
    r = moe.make_router()
    moe.moe_route_scored(s, r, e, w, None, None, idx, f, cnt, None, None)
    moe.moe_route_scored_backward(s, r, f, None, e, w, torch.empty(0, 16, device=DEV), idx, None, e, dw, db, None)
    assert (cnt == 0).all() and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T,d", [(3, 256), (12, 2048), (70, 256)])
def test_side_stream_graph_and_repeats(T, d):
    print(f"\n[case] route_scored graph {T}x{d}", flush=True)
    rule = R("sigmoid", 8, 4, 2, True, 2.5)
    E, k = 64, 6
    x, w, _, bal, _ = draw("bf16", T, d, E, k, rule, 8, True)
    s, idx, gate, cnt, logits = run("bf16", x, w, None, bal, k, rule)
    ws, wb = moe.workspace(s, moe.OP_ROUTE, DEV), moe.workspace(s, moe.OP_ROUTE_BACKWARD, DEV)
    out = [torch.zeros_like(t) for t in (idx, gate, cnt, logits)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_route_scored(s, make(rule), x, w, None, bal, *out, ws, stream=side)
    side.synchronize()
    assert all(same_bits(a, b) for a, b in zip(out, (idx, gate, cnt, logits)))
    dg, dx, dw, db = randn(gen(2), T, k), torch.empty_like(x), torch.empty_like(w), torch.empty(E, device=DEV)

    def both():
        moe.moe_route_scored(s, make(rule), x, w, None, bal, *out, ws)
        moe.moe_route_scored_backward(s, make(rule), dg, None, x, w, out[3], out[0], x, dx, dw, db, wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for j in range(4):
        x.copy_(randn(gen(50 + j), T, d, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, dx, dw, db)]
        both()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(got, (*out, dx, dw, db)))


@pytest.mark.parametrize("case", [("bf16", 1, 128, 64, 4), ("bf16", 16, 256, 500, 8), ("bf16", 17, 256, 500, 8), ("bf16", 4100, 256, 72, 4),
                                  ("f32", 30, 64, 20, 3), ("f32", 3000, 64, 20, 3)], ids=str)
def test_backward_keeps_to_its_workspace(case):
    dtype, T, d, E, k = case
    print(f"\n[case] route_scored backward workspace {case}", flush=True)
    rule = R("sigmoid", renormalise=False)
    x, w, _, _, _ = draw(dtype, T, d, E, k, rule, 8, False)
    s, idx, gate, _, logits = run(dtype, x, w, None, None, k, rule)
    dg = randn(gen(2), T, k)
    n = moe.workspace_bytes(s, moe.OP_ROUTE_BACKWARD)
    outs = []
    for fill in (0, 255):
        buf = torch.full((n + 65536,), fill, dtype=torch.uint8, device=DEV)
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(E, device=DEV)
        moe.moe_route_scored_backward(s, make(rule), dg, None, x, w, logits, idx, None, dx, dw, db, buf[:n])
        torch.cuda.synchronize()
        assert (buf[n:] == fill).all()
        outs.append((dx, dw, db))
    assert all(same_bits(a, b) for a, b in zip(*outs))


def test_balance_masks_inside_groups():
    """A balance of -inf leaves group 0 and one expert of group 1: every group but the first then scores -inf (group 1
    for want of a second), the tie goes to the lower id, and the choice is of the experts that are left.  With as many
    experts left as are chosen, the choice is theirs whatever the logits."""
    E, inf = 16, float("inf")
    for rule in (R("sigmoid", 4, 2, 2), R("softmax", 4, 2, 2, False), R("sigmoid", 4, 2, 1)):
        for k, left in ((3, 5), (5, 5), (2, 5)):
            print(f"\n[case] route_scored balance masks {rule} k={k}", flush=True)
            x, w, _, _, l = draw("bf16", 12, 64, E, k, rule, 3, False)
            bal = torch.zeros(E, device=DEV)
            bal[left:] = -inf
            _, idx, gate, cnt, _ = run("bf16", x, w, None, bal, k, rule)
            assert (idx < left).all() and (idx[:, 1:] > idx[:, :-1]).all() and int(cnt[:left].sum()) == 12 * k and (cnt[left:] == 0).all()
            want = ops.choose(l, rule, k, host(bal))
            assert np.array_equal(idx.cpu().numpy(), want)
            g = ops.gates(l, want, rule)
            within(host(gate), g, abs(g) * 2.0 ** -12, "gates")
            assert (gate > 0).all()
