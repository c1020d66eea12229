"""The selective layer's oracle against differences, its own step form and
closed forms; the error bounds that it carries against fp32 arithmetic."""

import numpy as np
import pytest

from oracle import ssm_oracle as O


def rng(seed=0):
    return np.random.default_rng(seed)


def scan_inputs(B=2, L=7, D=8, N=8, G=1, seed=0):
    r = rng(seed)
    n = r.standard_normal
    return dict(x=n((B, L, D)), dt=n((B, L, D)), A=-np.exp(n((D, N)) * 0.5), Bm=n((B, G, L, N)), Cm=n((B, G, L, N)), D=n(D),
                z=n((B, L, D)), dt_bias=n(D) - 1.0, h0=n((B, D, N)))


def differences(f, args, names, cot, g, outs, eps=1e-6):
    """Every gradient in `names` against central differences along random directions."""
    r = rng(5)
    for name, key in zip(names, outs):
        for _ in range(3):
            v = r.standard_normal(args[name].shape)
            hi, lo = dict(args), dict(args)
            hi[name], lo[name] = args[name] + eps * v, args[name] - eps * v
            num = sum((c * (a - b)).sum() for c, a, b in zip(cot, f(**hi), f(**lo))) / (2 * eps)
            assert abs(num - (g[key] * v).sum()) <= 1e-7 * (1 + np.abs(g[key] * v).sum()), name


@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("sp", [True, False])
def test_scan_gradient(G, sp):
    a = scan_inputs(D=16, G=G)
    if not sp:
        a["dt"], a["dt_bias"] = np.abs(a["dt"]), np.abs(a["dt_bias"])
    r = rng(1)
    gy, gh = r.standard_normal(a["x"].shape), r.standard_normal(a["h0"].shape)
    g = O.selscan_bwd(**a, sp=sp, g_y=gy, g_hL=gh)
    names = ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0")
    differences(lambda **k: O.selscan_fwd(**k, sp=sp)[:2], a, names, (gy, gh), g,
                ("g_x", "g_dt", "g_A", "g_B", "g_C", "g_D", "g_z", "g_dt_bias", "g_h0"))


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("L", [1, 2, 9])
@pytest.mark.parametrize("act", [True, False])
def test_conv_gradient(W, L, act):
    r = rng(2)
    n = r.standard_normal
    a = dict(x=n((2, L, 8)), w=n((8, W)), bias=n(8), x0=n((2, W - 1, 8)))
    gy, gx = n((2, L, 8)), n((2, W - 1, 8))
    g = O.conv_bwd(**a, act=act, g_y=gy, g_xL=gx)
    differences(lambda **k: O.conv_fwd(**k, act=act), a, ("x", "w", "bias", "x0"), (gy, gx), g, ("g_x", "g_w", "g_bias", "g_x0"))


@pytest.mark.parametrize("gate", [None, "before", "after"])
@pytest.mark.parametrize("per_head", [True, False])
def test_norm_gradient(gate, per_head):
    r = rng(3)
    n = r.standard_normal
    shape = (3, 8) if per_head else (8,)
    a = dict(x=n((2, 3, 5, 8)), w=n(shape), res_scale=n(shape))
    if gate:
        a["z"] = n((2, 3, 5, 8))
    gy = n((2, 3, 5, 8))
    g = O.norm_bwd(**a, gate=gate, g_y=gy)
    names = tuple(a)
    differences(lambda **k: (O.norm_fwd(**k, gate=gate),), a, names, (gy,), g, tuple("g_" + k for k in names))


def test_steps_and_cuts():
    """A prompt in two parts, and token by token on a pool, gives what it gives in one."""
    a = scan_inputs(B=1)
    y, h, _ = O.selscan_fwd(**a)
    cut = lambda t, s: dict(t, **{n: t[n][:, s] for n in ("x", "dt", "z")}, **{n: t[n][:, :, s] for n in ("Bm", "Cm")})  # noqa: E731
    y1, h1, _ = O.selscan_fwd(**cut(a, slice(0, 3)))
    y2, h2, _ = O.selscan_fwd(**dict(cut(a, slice(3, 7)), h0=h1))
    assert np.allclose(np.concatenate([y1, y2], 1), y) and np.allclose(h2, h)
    pool = np.zeros((3, 8, 8))
    pool[2] = a["h0"][0]
    for t in range(7):
        yt, pool = O.selscan_step(a["x"][:, t], a["dt"][:, t], a["A"], a["Bm"][:, :, t], a["Cm"][:, :, t], pool, a["D"],
                                  a["z"][:, t], a["dt_bias"], state_idx=[2])
        assert np.allclose(yt, y[:, t])
    assert np.allclose(pool[2], h[0]) and not pool[:2].any()
    r = rng(4)
    x, w, x0 = r.standard_normal((1, 5, 8)), r.standard_normal((8, 4)), r.standard_normal((1, 3, 8))
    y, xL = O.conv_fwd(x, w, None, x0)
    pool = x0.copy()
    for t in range(5):
        yt, pool = O.conv_step(x[:, t], w, pool)
        assert np.allclose(yt, y[:, t])
    assert np.array_equal(pool, xL)


def test_closed_form():
    """Constant inputs: a geometric series in every state."""
    L, N = 20, 8
    A = -np.arange(1.0, N + 1)[None].repeat(8, 0)
    one = np.ones
    y, h, _ = O.selscan_fwd(one((1, L, 8)), 0.1 * one((1, L, 8)), A, one((1, 1, L, N)), one((1, 1, L, N)), sp=False)
    a = np.exp(0.1 * A[0])
    assert np.allclose(h[0, 0], 0.1 * (1 - a ** L) / (1 - a))
    assert np.allclose(y[0, -1, 0], h[0, 0].sum())


def test_bounds_hold_in_fp32():
    """The definitions run in numpy fp32 stay within what Bound says, and the bound is no more than some thousand times what it is off by."""
    a = scan_inputs(B=2, L=40, D=16, N=16, seed=6)
    f = {k: v.astype(np.float32) for k, v in a.items()}
    B = {k: (O.Bound(v) if k != "A" else v.astype(np.float64)) for k, v in f.items()}
    y, h, _ = O.selscan_fwd(**B)
    y32, h32, _ = O.selscan_fwd(**f)
    assert y32.dtype == np.float32
    for got, ref in ((y32, y), (h32, h)):
        off = np.abs(got - ref.v)
        assert (off <= ref.e).all()
        assert ref.e.mean() < 3000 * off.mean()
