"""CPU pins of the oracle's norm, scored routing and FP8 (oracle/ops.py): torch autograd and
central differences for every gradient, an independent dense selection, torch's own E4M3 cast."""
import numpy as np
import pytest
import torch

from oracle import ops


def rng(seed):
    return np.random.default_rng(seed)


def difference(f, x, d, eps=1e-6):
    """Central difference of the scalar f along d."""
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


def test_norm_gradient_against_differences():
    r = rng(0)
    h, w, dy, dh = r.normal(size=(5, 24)), r.normal(size=24), r.normal(size=(5, 24)), r.normal(size=(5, 24))
    _, rstd = ops.add_rmsnorm(h, w, 1e-5)
    dx, dw = ops.add_rmsnorm_backward(dy, dh, h, w, rstd)
    d = r.normal(size=h.shape)
    f = lambda v: (ops.add_rmsnorm(v, w, 1e-5)[0] * dy).sum() + (v * dh).sum()  # noqa: E731
    assert difference(f, h, d) == pytest.approx((dx * d).sum(), rel=1e-7)
    d = r.normal(size=w.shape)
    assert difference(lambda v: (ops.add_rmsnorm(h, v, 1e-5)[0] * dy).sum(), w, d) == pytest.approx((dw * d).sum(), rel=1e-7)
    assert np.allclose(ops.add_rmsnorm_backward(dy, None, h, w, rstd)[0] + dh, dx, rtol=0, atol=1e-15)


def test_norm_by_hand():
    y, rstd = ops.add_rmsnorm(np.array([[3.0, 4.0], [0.0, 0.0]]), np.array([2.0, 1.0]), 0.0 + 1e-300)
    assert rstd[0] == pytest.approx(1 / np.sqrt(12.5)) and np.allclose(y[0], [6 / np.sqrt(12.5), 4 / np.sqrt(12.5)])
    assert (y[1] == 0).all()


RULES = [ops.Rule(), ops.Rule(renormalise=False, scale=1.7), ops.Rule("sigmoid", scale=2.5), ops.Rule("sigmoid", renormalise=False),
         ops.Rule("sigmoid", 4, 2, 2, True, 2.5), ops.Rule("softmax", 4, 3, 1, False)]


@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("balanced", [False, True])
def test_choice_against_torch(rule, balanced):
    r = rng(1)
    l, b = r.normal(size=(40, 16)), 0.1 * r.normal(size=16) if balanced else None
    idx = ops.choose(l, rule, 3, b)
    lt = torch.from_numpy(l)
    c = torch.sigmoid(lt) if rule.score == "sigmoid" else torch.softmax(lt, 1)
    if balanced:
        c = c + torch.from_numpy(b)
    per = c.view(40, rule.groups, -1)
    top = per.topk(rule.group_top, 2).values.sum(2).topk(rule.top_groups, 1).indices
    mask = torch.zeros(40, rule.groups, dtype=torch.bool).scatter_(1, top, True)
    c = per.masked_fill(~mask[:, :, None], -9.0).reshape(40, 16)
    assert np.array_equal(idx, c.topk(3, 1).indices.sort(1).values.numpy())
    assert (ops.margins(l, rule, 3, b) > 0).all()


@pytest.mark.parametrize("rule", RULES, ids=str)
def test_gate_gradient_against_autograd_and_differences(rule):
    r = rng(2)
    l = r.normal(size=(7, 16))
    idx, dg = ops.choose(l, rule, 3), r.normal(size=(7, 3))
    dl = ops.gates_backward(dg, l, idx, rule)
    lt = torch.from_numpy(l).requires_grad_()
    s = torch.sigmoid(lt) if rule.score == "sigmoid" else torch.softmax(lt, 1)
    g = s.gather(1, torch.from_numpy(idx))
    if rule.renormalise:
        g = g / g.sum(1, keepdim=True)
    assert np.allclose(rule.scale * g.detach().numpy(), ops.gates(l, idx, rule), rtol=1e-13)
    (rule.scale * g * torch.from_numpy(dg)).sum().backward()
    assert np.allclose(lt.grad.numpy(), dl, rtol=1e-11, atol=1e-14)
    d = r.normal(size=l.shape)
    assert difference(lambda v: (ops.gates(v, idx, rule) * dg).sum(), l, d) == pytest.approx((dl * d).sum(), rel=1e-6, abs=1e-9)


def test_ties_go_to_the_lower_id():
    l = np.zeros((1, 8))
    assert ops.choose(l, ops.Rule(), 3).tolist() == [[0, 1, 2]]
    assert ops.choose(l, ops.Rule("sigmoid", 4, 2, 2), 3).tolist() == [[0, 1, 2]]
    l[0, 5] = 1.0
    assert ops.choose(l, ops.Rule("sigmoid", 4, 2, 1), 3).tolist() == [[0, 1, 5]]


def test_masked_rows():
    l = np.full((2, 4), -np.inf)
    l[1, 2] = 0.0
    for rule in (ops.Rule(), ops.Rule("sigmoid")):
        assert ops.choose(l, rule, 2).tolist() == [[0, 1], [0, 2]]
        g = ops.gates(l, ops.choose(l, rule, 2), rule)
        assert g[0].tolist() == [0, 0] and g[1].tolist() == [0, 1]
        assert (ops.gates_backward(np.ones((2, 2)), l, ops.choose(l, rule, 2), rule) == 0).all()


def test_e4m3_against_torch():
    r = rng(3)
    v = np.concatenate([r.normal(size=20000) * 10.0 ** r.integers(-4, 3, 20000), [0.0, 448.0, -448.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    v = v.astype(np.float32).clip(-448, 448)
    assert np.array_equal(ops.e4m3(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def test_blocks():
    r = rng(4)
    w = r.normal(size=(200, 256))
    q, s = ops.quantise_blocks(w)
    assert s.shape == (2, 2) and np.abs(q).max() == 448.0
    assert np.allclose(ops.spread_blocks(q, s), w, atol=np.abs(w).max() / 448 * 2 ** 4)
    w[:128, :128] = 0
    q, s = ops.quantise_blocks(w)
    assert (q[:128, :128] == 0).all() and s[0, 0] == 2.0 ** -100 / 448
    q, s = ops.quantise_rows(w)
    assert s.shape == (200, 2) and np.abs(ops.spread_rows(q, s) - w).max() <= 2.0 ** -4 * np.abs(w).max()
