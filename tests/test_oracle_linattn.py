"""Pins of the linear-attention oracle: values by hand, the closed form, a
split sequence, finite differences of a scalar loss and the step as a
sequence of one."""

import numpy as np
import pytest

from oracle.linattn_oracle import linattn_bwd, linattn_fwd, linattn_step


def _inputs(B=2, H=4, Hk=2, L=5, dk=3, dv=2, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.normal(size=(B, Hk, L, dk)), k=r.normal(size=(B, Hk, L, dk)), v=r.normal(size=(B, H, L, dv)),
                g=-np.exp(r.normal(size=(B, H, L))), h0=r.normal(size=(B, H, dk, dv)))


def test_two_steps_by_hand():
    q = np.array([[[[1.0], [2.0]]]])
    k = np.array([[[[3.0], [5.0]]]])
    v = np.array([[[[7.0], [11.0]]]])
    g = np.log(np.array([[[0.5, 0.25]]]))
    o, h, _ = linattn_fwd(q, k, v, g, h0=np.array([[[[4.0]]]]), scale=0.5)
    # S_1 = 0.5*4 + 21 = 23, S_2 = 0.25*23 + 55 = 60.75
    assert np.allclose(o.ravel(), [0.5 * 1 * 23, 0.5 * 2 * 60.75])
    assert np.allclose(h.ravel(), [60.75])


def test_closed_form():
    x = _inputs()
    o, _, _ = linattn_fwd(**x, scale=0.7)
    G = np.cumsum(x["g"], -1)
    for b in range(2):
        for h in range(4):
            for t in range(5):
                want = np.exp(G[b, h, t]) * (x["q"][b, h // 2, t] @ x["h0"][b, h])
                for j in range(t + 1):
                    want = want + np.exp(G[b, h, t] - G[b, h, j]) * (x["q"][b, h // 2, t] @ x["k"][b, h // 2, j]) * x["v"][b, h, j]
                assert np.allclose(o[b, h, t], 0.7 * want)


def test_split_sequence_and_step():
    x = _inputs(L=6)
    o, h, _ = linattn_fwd(**x, scale=0.7)
    cut = lambda a, s: {n: (y[:, :, s] if n != "h0" else y) for n, y in a.items()}  # noqa: E731
    o1, h1, _ = linattn_fwd(**cut(x, slice(0, 2)), scale=0.7)
    y = dict(cut(x, slice(2, 6)), h0=h1)
    o2, h2, _ = linattn_fwd(**y, scale=0.7)
    assert np.allclose(np.concatenate([o1, o2], 2), o) and np.allclose(h2, h)
    pool = np.concatenate([x["h0"][::-1], x["h0"][:1] * 0 + 9])
    os, new = linattn_step(x["q"][:, :, 0], x["k"][:, :, 0], x["v"][:, :, 0], x["g"][:, :, 0], pool, [1, 0], 0.7)
    assert np.allclose(os, o[:, :, 0]) and np.all(new[2] == 9)
    os, new2 = linattn_step(x["q"][:, :, 0], x["k"][:, :, 0], x["v"][:, :, 0], x["g"][:, :, 0], pool, [-1, 7], 0.7)
    assert np.all(os[0] == 0) and np.isnan(os[1]).all() and np.array_equal(new2, pool)


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "h0"])
def test_gradient_by_differences(name):
    x = _inputs()
    r = np.random.default_rng(1)
    go, gh = r.normal(size=x["v"].shape), r.normal(size=x["h0"].shape)

    def loss(y):
        o, h, _ = linattn_fwd(**y, scale=0.7)
        return (o * go).sum() + (h * gh).sum()

    got = linattn_bwd(**x, g_o=go, g_hL=gh, scale=0.7)["g_" + name]
    num = np.zeros_like(x[name])
    for i in np.ndindex(*num.shape):
        p, m = (dict(x, **{name: x[name].copy()}) for _ in range(2))
        p[name][i] += 1e-5
        m[name][i] -= 1e-5
        num[i] = (loss(p) - loss(m)) / 2e-5
    assert np.abs(got - num).max() <= 1e-8 * (1 + np.abs(num).max())
