"""The 64-bit definitions that the gradients are tested against (tests/grad_utils.py): their values against the C
oracle, their gradients against central differences of the oracle.

A central difference along a unit step of h = 1e-5 is off by h^2 / 6 times the third derivative (a few times the value
here: 1e-10) and by 2^-52 |L| / h (2e-11 |L|), so 1e-7 of the sum of magnitudes is well above both.
"""
import numpy as np
import pytest
import torch

import oracle
from tests import grad_utils as G

H, BOUND = 1e-5, 1e-7


def draws(seed):
    r = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=r, dtype=torch.float64)


def cu_of(lens):
    return np.cumsum([0] + list(lens)).astype(np.int32)


def t64(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float64))


def rule_inputs(lens, nqk, nv, dk, dv, seed=0):
    n, t = draws(seed), sum(lens)
    g, beta = -n(t, nv).abs(), torch.sigmoid(n(t, nv))
    return [n(t, nqk, dk), n(t, nqk, dk), n(t, nv, dv), g, beta, n(len(lens), nv, dk, dv)]


@pytest.mark.parametrize("l2", [True, False])
@pytest.mark.parametrize("lens,nqk,nv", [((5,), 1, 1), ((70, 0, 1, 9), 2, 4), ((3, 3), 1, 3)])
def test_rule_is_the_oracles(lens, nqk, nv, l2):
    x = rule_inputs(lens, nqk, nv, 8, 6)
    if not l2:
        x[1] = x[1] / x[1].norm(dim=-1, keepdim=True)
    out, fin = G.rule(*x, lens, qk_l2norm=l2)
    ref_o, ref_s = oracle.recurrent(*[y.numpy() for y in x], cu_of(lens), qk_l2norm=l2)
    assert np.allclose(out.numpy(), ref_o, rtol=0, atol=1e-11 * np.abs(ref_o).max())
    assert np.allclose(fin.numpy(), ref_s, rtol=0, atol=1e-11 * np.abs(ref_s).max())


def differences(loss, x, grads, seed, scale=1.0):
    """Every input along two random directions; where `loss` is linear in nothing the step stays small."""
    n = draws(seed)
    for i, (a, g) in enumerate(zip(x, grads)):
        for _ in range(2):
            d = n(*a.shape)
            d = d / d.norm().clamp(min=1e-30)
            lo, hi = ([y if j != i else y + s * H * d for j, y in enumerate(x)] for s in (-1, 1))
            l0, l1 = loss(lo), loss(hi)
            want = (l1 - l0) / (2 * H)
            assert abs(want - (g * d).sum().item()) <= BOUND * max(1.0, abs(l0) + abs(l1)) * scale, i


@pytest.mark.parametrize("lens,nqk,nv", [((7,), 1, 1), ((66, 0, 1, 5), 1, 2)])
def test_rule_gradients_are_differences_of_the_oracle(lens, nqk, nv):
    x = rule_inputs(lens, nqk, nv, 8, 6, seed=1)
    n = draws(2)
    do, ds = n(*x[2].shape), n(*x[5].shape)

    def loss(y):
        o, s = oracle.recurrent(*[t.numpy() for t in y], cu_of(lens))
        return float((o * do.numpy()).sum() + (s * ds.numpy()).sum())
    differences(loss, x, G.rule_grads(*x, do, ds, lens), 3)


def test_gate_and_its_gradients():
    n = draws(4)
    x = [3 * n(20, 3), 3 * n(20, 3), n(3), n(3)]
    g, b = G.gate(*x)
    rg, rb = oracle.gates(*[y.numpy() for y in x])
    assert np.allclose(g.numpy(), rg, rtol=1e-13, atol=0) and np.allclose(b.numpy(), rb, rtol=1e-13, atol=0)
    dg, db = n(20, 3), n(20, 3)
    leaves = [y.clone().requires_grad_() for y in x]
    grads = torch.autograd.grad(list(G.gate(*leaves)), leaves, [dg, db])

    def loss(y):
        a, c = oracle.gates(*[t.numpy() for t in y])
        return float((a * dg.numpy()).sum() + (c * db.numpy()).sum())
    differences(loss, x, grads, 5)


def test_norm_and_its_gradients():
    n = draws(6)
    x, eps = [n(11, 64), n(11, 64), n(64)], 1e-3
    ref = oracle.gated_rmsnorm(*[y.numpy() for y in x], eps)
    assert np.allclose(G.norm(*x, eps).numpy(), ref, rtol=1e-12, atol=1e-14)
    dy = n(11, 64)
    leaves = [y.clone().requires_grad_() for y in x]
    grads = torch.autograd.grad(G.norm(*leaves, eps), leaves, dy)
    differences(lambda y: float((oracle.gated_rmsnorm(*[t.numpy() for t in y], eps) * dy.numpy()).sum()), x, grads, 7)


@pytest.mark.parametrize("k", [1, 3, 4])
def test_conv_and_its_gradients(k):
    lens, c = (5, 0, 1, 2, 9), 6
    n = draws(8)
    x = [n(sum(lens), c), n(c, k), n(c), n(len(lens), c, k)]

    def ref(y):
        return oracle.causal_conv1d(y[0].numpy(), y[1].numpy(), y[2].numpy(), cu_of(lens), y[3].numpy())
    y, st = G.conv(*x, lens)
    ry, rs = ref(x)
    assert np.allclose(y.numpy(), ry, rtol=1e-12, atol=1e-14) and np.array_equal(st.numpy(), rs)
    dy, ds = n(*y.shape), n(*st.shape)
    leaves = [t.clone().requires_grad_() for t in x]
    grads = torch.autograd.grad(list(G.conv(*leaves, lens)), leaves, [dy, ds])

    def loss(z):
        a, b = ref(z)
        return float((a * dy.numpy()).sum() + (b * ds.numpy()).sum())
    differences(loss, x, grads, 9)


def test_a_planted_mistake_is_found():
    """The bound tells a gradient that lacks one of its terms from the right one: here the L2 norm's."""
    lens = (40,)
    x = rule_inputs(lens, 1, 2, 8, 6, seed=10)
    n = draws(11)
    do, ds = n(*x[2].shape), torch.zeros(1, 2, 8, 6, dtype=torch.float64)
    right = G.rule_grads(*x, do, ds, lens)
    q = x[0]
    along = (right[0] + 1e-3 * q)  # the norm takes the part along q out; put some of it back
    with pytest.raises(AssertionError):
        G.assert_close(along.float(), right[0], torch.float32, "dq")
