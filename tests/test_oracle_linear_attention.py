"""Pins of the fp64 linear-attention and group-norm oracles on the CPU: closed
forms, and every gradient against central differences."""
import numpy as np
import pytest

from oracle import group_norm as gn
from oracle import linear_attention as la


def draw(T, H, Dk, Dv, seed, h0=True):
    r = np.random.default_rng(seed)
    x = dict(q=r.normal(size=(T, H, Dk)), k=r.normal(size=(T, H, Dk)), v=r.normal(size=(T, H, Dv)),
             log_decay=-r.uniform(0, 1, size=H), h0=r.normal(size=(H, Dk, Dv)) if h0 else None)
    return x


@pytest.mark.parametrize("T", [1, 2, 9])
def test_forward_is_the_decayed_sum(T):
    """o_t = sum_s gamma^(t-s) (q_t . k_s) v_s + gamma^(t+1) h0^T q_t."""
    x = draw(T, 2, 3, 4, T)
    o, S = la.forward(**x)
    for h in range(2):
        g = np.exp(x["log_decay"][h])
        for t in range(T):
            want = g ** (t + 1) * x["h0"][h].T @ x["q"][t, h]
            for s in range(t + 1):
                want = want + g ** (t - s) * (x["q"][t, h] @ x["k"][s, h]) * x["v"][s, h]
            np.testing.assert_allclose(o[t, h], want, rtol=1e-12, atol=1e-12)
        want = g ** T * x["h0"][h] + sum(g ** (T - 1 - s) * np.outer(x["k"][s, h], x["v"][s, h]) for s in range(T))
        np.testing.assert_allclose(S[h], want, rtol=1e-12, atol=1e-12)


def test_decay_of_zero_and_one():
    x = draw(5, 2, 3, 4, 1)
    x["log_decay"] = np.array([-np.inf, 0.0])
    o, _ = la.forward(**x)
    np.testing.assert_allclose(o[3, 0], (x["q"][3, 0] @ x["k"][3, 0]) * x["v"][3, 0])
    want = x["h0"][1].T @ x["q"][3, 1] + sum((x["q"][3, 1] @ x["k"][s, 1]) * x["v"][s, 1] for s in range(4))
    np.testing.assert_allclose(o[3, 1], want)


def test_gradients_match_differences():
    """L is linear in each of q, k, v, h0: central differences are exact up to
    the rounding of L (1e-16 |L| / step)."""
    x = draw(6, 2, 3, 4, 2)
    r = np.random.default_rng(3)
    d_o, dh = r.normal(size=(6, 2, 4)), r.normal(size=(2, 3, 4))
    got = dict(zip(("q", "k", "v", "h0"), la.backward(**x, d_o=d_o, dh_final=dh)))

    def loss(y):
        o, S = la.forward(**y)
        return (o * d_o).sum() + (S * dh).sum()

    for name in got:
        step = r.normal(size=x[name].shape)
        up, dn = dict(x), dict(x)
        up[name], dn[name] = x[name] + 0.5 * step, x[name] - 0.5 * step
        np.testing.assert_allclose((got[name] * step).sum(), loss(up) - loss(dn), rtol=1e-11)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("shape,groups", [((2, 1, 12), 3), ((3, 5, 8), 2), ((1, 4, 6), 6)])
def test_norm_gradients_match_differences(shape, groups, act):
    """Fourth-order differences: truncation h^4, rounding 1e-16 / h at h = 1e-3."""
    r = np.random.default_rng(5)
    x, dy = r.normal(size=shape), r.normal(size=shape)
    w, b = 1 + 0.2 * r.normal(size=shape[-1]), r.normal(size=shape[-1])
    _, mean, rstd = gn.forward(x, w, b, groups, 1e-5, act)
    dx, dw, db = gn.backward(dy, x, w, b, mean, rstd, groups, act)
    for name, grad, at in (("x", dx, x), ("w", dw, w), ("b", db, b)):
        d = r.normal(size=at.shape)

        def loss(e):
            v = dict(x=x, w=w, b=b)
            v[name] = at + e * d
            return (gn.forward(v["x"], v["w"], v["b"], groups, 1e-5, act)[0] * dy).sum()

        h = 1e-3
        diff = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
        np.testing.assert_allclose((grad * d).sum(), diff, rtol=1e-7, atol=1e-8)
