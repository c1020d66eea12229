"""Plain fp64 numpy oracle of the selective state-space layer: a short causal
convolution, the selective scan and the norm around a block, with their
gradients by the chain rule, step by step from the definitions.  Test
infrastructure only.

Every function takes plain arrays, or ``Bound`` values, which carry along
with each number what fp32 arithmetic may have added to it; the same lines then
give the reference and how far from it a result may lie.

x, dt, z [B,L,D]; Bm, Cm [B,G,L,N]; A [D,N]; w [D,W]; conv states [B,W-1,D];
scan states [B,D,N]; norm rows [B,H,L,d].
"""

import numpy as np

U = 2.0 ** -24   # half a step of fp32, relative


class Bound:
    """v: the value; m: the same sum with every term's magnitude; e: what
    roundings to fp32 may have added, first order, whatever the order of a
    sum: an addition rounds by U of the magnitudes it joins, a product
    by U of itself.  Inputs are exact."""

    __array_ufunc__ = None

    def __init__(self, v, m=None, e=None):
        self.v = np.asarray(v, np.float64)
        self.m = np.abs(self.v) if m is None else m
        self.e = np.zeros_like(self.v) if e is None else e

    @staticmethod
    def of(x):
        return x if isinstance(x, Bound) else Bound(x)

    @property
    def shape(self):
        return self.v.shape

    @property
    def ndim(self):
        return self.v.ndim

    def __add__(self, o):
        o = Bound.of(o)
        m = self.m + o.m
        return Bound(self.v + o.v, m, self.e + o.e + U * m)

    __radd__ = __add__

    def __neg__(self):
        return Bound(-self.v, self.m, self.e)

    def __sub__(self, o):
        return self + (-Bound.of(o))

    def __rsub__(self, o):
        return Bound.of(o) + (-self)

    def __mul__(self, o):
        o = Bound.of(o)
        m = self.m * o.m
        return Bound(self.v * o.v, m, self.m * o.e + self.e * o.m + self.e * o.e + U * m)

    __rmul__ = __mul__

    def __getitem__(self, i):
        return Bound(self.v[i], self.m[i], self.e[i])

    def reshape(self, *s):
        return Bound(self.v.reshape(*s), self.m.reshape(*s), self.e.reshape(*s))

    def sum(self, axis):
        n = int(np.prod([self.v.shape[a] for a in np.atleast_1d(axis)]))
        axis = tuple(np.atleast_1d(axis))
        m = self.m.sum(axis)
        return Bound(self.v.sum(axis), m, self.e.sum(axis) + n * U * m)

    def map(self, f, slope, own):
        """f of it: its error times the slope, and `own` roundings of the result."""
        v = f(self.v)
        return Bound(v, np.abs(v), np.abs(slope(self.v)) * self.e + own * U * np.abs(v))


def _sig(x):
    return np.exp(-np.logaddexp(0.0, -x))


def sigmoid(x):
    # An exponential (two for it and its argument's product), an addition, a reciprocal and a product.  Where it is taken
    # the short way the argument, x log2 e, is off by half a step of itself and by that of log2 e: 1.3 |x| U of e^-x.
    return x.map(_sig, lambda v: _sig(v) * (1 - _sig(v)), 8 + 1.3 * np.abs(x.v)) if isinstance(x, Bound) else _sig(x)


def softplus(x):
    # the exponential, a logarithm, a reciprocal, three products, a sum
    return x.map(lambda v: np.logaddexp(0.0, v), _sig, 12) if isinstance(x, Bound) else np.logaddexp(0.0, x)


def silu(x):
    return x * sigmoid(x)


def silu_slope(x):
    s = sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


def decay(d, A):
    """exp(d A).  The exponent is a product with A log2 e (two roundings), of
    a step or of a sum of up to 64 steps in fp32, of which each step takes its
    share; the exponential itself has two."""
    if not isinstance(d, Bound):
        return np.exp(d * A)
    x = d.v * A
    v = np.exp(x)
    return Bound(v, v, v * (np.abs(A) * d.e + 70 * U * np.abs(x) + 3 * U))


def rsqrt(x):
    return x.map(lambda v: v ** -0.5, lambda v: 0.5 * v ** -1.5, 3) if isinstance(x, Bound) else x ** -0.5


def stack(xs, axis):
    if xs and isinstance(xs[0], Bound):
        return Bound(*(np.stack([getattr(x, n) for x in xs], axis) for n in "vme"))
    return np.stack(xs, axis)


def concat(xs, axis):
    if any(isinstance(x, Bound) for x in xs):
        xs = [Bound.of(x) for x in xs]
        return Bound(*(np.concatenate([getattr(x, n) for x in xs], axis) for n in "vme"))
    return np.concatenate(xs, axis)


# ---- convolution

def _window(x, w, x0):
    W = w.shape[1]
    B, L, D = x.shape
    return concat([np.zeros((B, W - 1, D)) if x0 is None else x0, x], 1), W, L


def conv_pre(x, w, bias=None, x0=None):
    full, W, L = _window(x, w, x0)
    pre = full[:, 0:L] * w[:, 0]
    for j in range(1, W):
        pre = pre + full[:, j:j + L] * w[:, j]
    return pre if bias is None else pre + bias


def conv_fwd(x, w, bias=None, x0=None, act=True):
    """(y, x_L)"""
    full, W, L = _window(x, w, x0)
    pre = conv_pre(x, w, bias, x0)
    return (silu(pre) if act else pre), full[:, L:]


def conv_bwd(x, w, g_y, bias=None, x0=None, g_xL=None, act=True):
    full, W, L = _window(x, w, x0)
    B, _, D = x.shape
    p = g_y * silu_slope(conv_pre(x, w, bias, x0)) if act else g_y
    rows = []
    for i in range(L + W - 1):   # every row of the window's: what reads it
        g = None
        for j in range(W):
            t = i - j
            if 0 <= t < L:
                term = p[:, t] * w[:, j]
                g = term if g is None else g + term
        if i >= L and g_xL is not None:
            g = g_xL[:, i - L] if g is None else g + g_xL[:, i - L]
        rows.append(np.zeros((B, D)) if g is None else g)
    if any(isinstance(r, Bound) for r in rows):
        rows = [Bound.of(r) for r in rows]
    g = stack(rows, 1)
    return {"g_x": g[:, W - 1:], "g_x0": g[:, :W - 1], "g_bias": (p * np.ones_like(full.v[:, :L] if isinstance(full, Bound) else full[:, :L])).sum((0, 1)),
            "g_w": stack([(p * full[:, j:j + L]).sum((0, 1)) for j in range(W)], 1)}


def conv_step(x, w, state, bias=None, state_idx=None, act=True):
    """(y [B,D], pool)"""
    pool, W = np.array(state, np.float64), w.shape[1]
    y, seen = np.zeros(x.shape), set()
    for b in range(x.shape[0]):
        s = b if state_idx is None else int(state_idx[b])
        if s < 0:
            continue
        if s >= pool.shape[0] or s in seen:
            y[b] = np.nan
            continue
        seen.add(s)
        y[b] = conv_fwd(x[b][None, None], w, bias, pool[s][None], act)[0][0, 0]
        pool[s] = np.concatenate([pool[s][1:], x[b][None]])
    return y, pool


# ---- selective scan

def _steps(x, dt, dt_bias, sp):
    raw = dt if dt_bias is None else dt + dt_bias
    return raw, (softplus(raw) if sp else raw)


def _wide(t, D):
    """[B,G,N] for every channel: [B,D,N]."""
    rep = D // t.shape[1]
    if isinstance(t, Bound):
        return Bound(*(np.repeat(getattr(t, n), rep, 1) for n in "vme"))
    return np.repeat(t, rep, 1)


def selscan_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, sp=True, h0=None):
    """(y, h_L, states [h_{-1}, h_0, ..])"""
    B, L, K = x.shape
    _, d = _steps(x, dt, dt_bias, sp)
    h = np.zeros((B, K, A.shape[1])) if h0 is None else h0
    if isinstance(x, Bound):
        h = Bound.of(h)
    states, ys = [h], []
    for t in range(L):
        h = decay(d[:, t][..., None], A) * h + (d[:, t] * x[:, t])[..., None] * _wide(Bm[:, :, t], K)
        states.append(h)
        ys.append((h * _wide(Cm[:, :, t], K)).sum(-1))
    y = stack(ys, 1)
    if D is not None:
        y = y + x * D
    return (y if z is None else y * silu(z)), h, states


def selscan_bwd(x, dt, A, Bm, Cm, g_y, D=None, z=None, dt_bias=None, sp=True, h0=None, g_hL=None):
    B, L, K = x.shape
    G, N = Bm.shape[1], A.shape[1]
    raw, d = _steps(x, dt, dt_bias, sp)
    y, _, S = selscan_fwd(x, dt, A, Bm, Cm, D, None, dt_bias, sp, h0)
    out = {}
    g = g_y
    if z is not None:
        out["g_z"] = g_y * y * silu_slope(z)
        g = g_y * silu(z)
    lam = np.zeros((B, K, N)) if g_hL is None else g_hL
    gB, gC, gu, gd, gA = [None] * L, [None] * L, [None] * L, [None] * L, []
    for t in reversed(range(L)):
        lam = g[:, t][..., None] * _wide(Cm[:, :, t], K) + lam
        gC[t] = (S[t + 1] * g[:, t][..., None]).reshape(B, G, K // G, N).sum(2)
        gB[t] = (lam * (d[:, t] * x[:, t])[..., None]).reshape(B, G, K // G, N).sum(2)
        gu[t] = (lam * _wide(Bm[:, :, t], K)).sum(-1)
        lam = lam * decay(d[:, t][..., None], A)
        p = lam * S[t]
        gd[t] = (p * A).sum(-1)
        gA.append((p * d[:, t][..., None]).sum(0))
    gu, gd = stack(gu, 1), stack(gd, 1)
    gx = d * gu
    if D is not None:
        gx = gx + g * D
    graw = x * gu + gd
    if sp:
        graw = graw * sigmoid(raw)
    out.update(g_x=gx, g_dt=graw, g_dt_bias=graw.sum((0, 1)), g_A=stack(gA, 0).sum(0), g_D=(g * x).sum((0, 1)),
               g_B=stack(gB, 2), g_C=stack(gC, 2), g_h0=lam)
    return out


def selscan_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, sp=True, state_idx=None):
    """(y [B,D], pool)"""
    pool = np.array(state, np.float64)
    y, seen = np.zeros(x.shape), set()
    for b in range(x.shape[0]):
        s = b if state_idx is None else int(state_idx[b])
        if s < 0:
            continue
        if s >= pool.shape[0] or s in seen:
            y[b] = np.nan
            continue
        seen.add(s)
        row = lambda t: None if t is None else t[b][None, None]  # noqa: E731
        yb, h, _ = selscan_fwd(row(x), row(dt), A, Bm[b][None, :, None], Cm[b][None, :, None], D, row(z), dt_bias, sp,
                               pool[s][None])
        y[b], pool[s] = yb[0, 0], h[0]
    return y, pool


# ---- norm

def _heads(t):
    """[H,d] or [d] against rows [B,H,L,d]."""
    return t[:, None] if t.ndim == 2 else t


def norm_fwd(x, w, z=None, gate=None, residual=None, res_scale=None, eps=1e-5):
    u = x * silu(z) if gate == "before" else x
    n = u * rsqrt((u * u).sum(-1) * (1.0 / x.shape[-1]) + eps)[..., None] * _heads(w)
    if gate == "after":
        n = n * silu(z)
    if res_scale is not None:
        n = n * _heads(res_scale)
    return n if residual is None else n + residual


def norm_bwd(x, w, g_y, z=None, gate=None, res_scale=None, eps=1e-5):
    d = x.shape[-1]
    u = x * silu(z) if gate == "before" else x
    r = rsqrt((u * u).sum(-1) * (1.0 / d) + eps)[..., None]
    k = u * r
    n = k * _heads(w)
    out = {}
    fold = lambda t: t.sum((0, 2)) if w.ndim == 2 else t.sum((0, 1, 2))  # noqa: E731
    if gate == "after":
        n = n * silu(z)
    g = g_y
    if res_scale is not None:
        out["g_res_scale"] = fold(g_y * n)
        g = g_y * _heads(res_scale)
    if gate == "after":
        out["g_z"] = g * (k * _heads(w)) * silu_slope(z)
        g = g * silu(z)
    out["g_w"] = fold(g * k)
    gw = g * _heads(w)
    gu = r * (gw - k * ((gw * k).sum(-1) * (1.0 / d))[..., None])
    if gate == "before":
        out["g_z"] = gu * x * silu_slope(z)
        gu = gu * silu(z)
    out["g_x"] = gu
    return out
