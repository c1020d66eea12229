"""The selective state-space layer on the GPU against the fp64 oracle, at the
sizes, layouts and sequences where it can go wrong.

Tolerances, elementwise, from the arithmetic: the oracle runs on ``Bound``
values, which add up what every fp32 rounding on the way may do (see
oracle/ssm_oracle.py: additions round by 2^-24 of all the magnitudes that they
join, whatever their order; what special functions have is stated there).
bf16 outputs add half a step of bf16, 2^-8 of the value.  Results below fp32's
normal numbers may be zero: 1e-30 is free.
"""

import numpy as np
import pytest

from oracle import ssm_oracle as O
from tests._gpu import lib

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DT = pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def bound(t):
    return None if t is None else O.Bound(f64(t))


def close(got, ref, what):
    assert tuple(got.shape) == tuple(ref.shape), f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    g = f64(got)
    if not g.size:
        return
    assert np.isfinite(g).all(), f"{what}: not finite"
    tol = ref.e * 1.01 + 1e-30
    if got.dtype == BF:
        tol = tol + 2.0 ** -8 * (np.abs(ref.v) + tol)
    worst = float((np.abs(g - ref.v) / tol).max())
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def check(got, ref):
    for n in got:
        close(got[n], ref[n], n)


class Gen:
    def __init__(self, seed, dt):
        self.g, self.dt = torch.Generator().manual_seed(seed), dt

    def f(self, *s, size=1.0):
        return (torch.randn(*s, generator=self.g) * size).cuda()

    def t(self, *s, size=1.0):
        return (torch.randn(*s, generator=self.g) * size).to(self.dt).cuda()


def bounds(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()


# ---- convolution

def conv_inputs(B, L, D, W, dt, seed=0, S=None, state=True):
    r = Gen(seed, dt)
    S = B if S is None else S
    x = dict(x=r.t(B, L, D), w=r.f(D, W, size=W ** -0.5), bias=r.f(D, size=0.3))
    if state:
        x["x0"] = r.t(S, W - 1, D)
    return x, r.t(B, L, D), r.t(S, W - 1, D)


def conv_ref(x, act=True):
    return O.conv_fwd(bound(x["x"]), f64(x["w"]), f64(x.get("bias")), f64(x.get("x0")), act)


def conv_gref(x, gy, gx, act=True):
    return O.conv_bwd(bound(x["x"]), f64(x["w"]), bound(gy), f64(x.get("bias")), f64(x.get("x0")), f64(gx), act)


@DT
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,L,D", [(1, 1, 8), (2, 2, 24), (3, 3, 64), (2, 15, 520), (1, 17, 256), (2, 67, 40), (1, 260, 1032)])
def test_conv(B, L, D, W, dt):
    P = lib()
    x, gy, gx = conv_inputs(B, L, D, W, dt)
    y, xL = P.pdssm_conv_fwd(**x)
    ry, rx = conv_ref(x)
    close(y, ry, "y")
    assert np.array_equal(f64(xL), O.Bound.of(rx).v)
    check(P.pdssm_conv_bwd(**x, g_y=gy, g_xL=gx), conv_gref(x, gy, gx))


@DT
@pytest.mark.parametrize("silu", [True, False])
def test_conv_without_what_is_optional(dt, silu):
    P = lib()
    x, gy, _ = conv_inputs(2, 33, 48, 4, dt, state=False)
    del x["bias"]
    y, xL = P.pdssm_conv_fwd(**x, silu=silu)
    ry, rx = conv_ref(x, silu)
    close(y, ry, "y")
    assert np.array_equal(f64(xL), O.Bound.of(rx).v)
    g = P.pdssm_conv_bwd(**x, g_y=gy, silu=silu, want_x0=False)
    assert set(g) == {"g_x", "g_w", "g_bias"}
    check(g, conv_gref(x, gy, None, silu))


LENGTHS = [(1,), (0, 5, 0, 0, 1, 2, 3, 70, 0), (31, 33, 16, 64, 1, 0), (300, 2, 15)]


@DT
@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("W", [2, 4])
def test_conv_packed(dt, lens, W):
    """Every sequence as by itself; rows before the first and behind the last stay as they are."""
    P = lib()
    S, n, before, after = len(lens), sum(lens), 3, 5
    x, gy, gx = conv_inputs(1, n + before + after, 40, W, dt, S=S, seed=1)
    cu = bounds(lens) + before
    mark = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    out = {"y": mark(x["x"])}
    y, xL = P.pdssm_conv_fwd(**x, cu_seqlens=cu, out=out)
    gout = {"g_x": mark(x["x"])}
    g = P.pdssm_conv_bwd(**x, g_y=gy, g_xL=gx, cu_seqlens=cu, out=gout)
    for t in (y, g["g_x"]):
        assert (t[:, :before] == 7).all() and (t[:, before + n:] == 7).all()
    gw = gb = None
    for i, m in enumerate(lens):
        at = slice(before + sum(lens[:i]), before + sum(lens[:i]) + m)
        xi = dict(x, x=x["x"][:, at], x0=x["x0"][i:i + 1])
        if m:
            ry, rx = conv_ref(xi)
            close(y[:, at], ry, f"y of {i}")
            r = conv_gref(xi, gy[:, at], gx[i:i + 1])
            close(g["g_x"][:, at], r["g_x"], f"g_x of {i}")
            close(g["g_x0"][i:i + 1], r["g_x0"], f"g_x0 of {i}")
            gw, gb = (r["g_w"], r["g_bias"]) if gw is None else (gw + r["g_w"], gb + r["g_bias"])
            assert np.array_equal(f64(xL[i:i + 1]), O.Bound.of(rx).v)
        else:
            assert torch.equal(xL[i], x["x0"][i]) and torch.equal(g["g_x0"][i], gx[i])
    close(g["g_w"], gw, "g_w")
    close(g["g_bias"], gb, "g_bias")


@DT
def test_conv_many_short_strips(dt):
    """More parts of g_w than one round of sums takes."""
    P = lib()
    x, gy, gx = conv_inputs(1100, 1, 8, 3, dt)
    check(P.pdssm_conv_bwd(**x, g_y=gy, g_xL=gx), conv_gref(x, gy, gx))
    x, gy, gx = conv_inputs(9, 4111, 8, 2, dt, seed=3)
    check(P.pdssm_conv_bwd(**x, g_y=gy, g_xL=gx), conv_gref(x, gy, gx))


# ---- selective scan

def scan_inputs(B, L, D, N, dt, G=1, seed=0, S=None, state=True, z=True, size=0.5):
    r = Gen(seed, dt)
    S = B if S is None else S
    x = dict(x=r.t(B, L, D), dt=r.t(B, L, D, size=0.7), A=-torch.exp(r.f(D, N, size=size)) * 2.0,
             Bm=r.t(B, L, G, N).transpose(1, 2), Cm=r.t(B, L, G, N).transpose(1, 2), D=r.f(D), dt_bias=r.f(D) - 3.0)
    if z:
        x["z"] = r.t(B, L, D)
    if state:
        x["h0"] = r.f(S, D, N)
    return x, r.t(B, L, D), r.f(S, D, N, size=0.3)


def scan_args(x):
    b = {n: bound(t) for n, t in x.items()}
    b["A"] = f64(x["A"])
    return b


def check_scan(x, y, hL, sp=True):
    ry, rh, _ = O.selscan_fwd(**scan_args(x), sp=sp)
    close(y, ry, "y")
    close(hL, rh, "h_L")


def check_scan_bwd(x, g, gy, gh, sp=True):
    check(g, O.selscan_bwd(**scan_args(x), g_y=bound(gy), g_hL=bound(gh), sp=sp))


SHAPES = [(1, 1, 8, 8, 1), (2, 3, 24, 16, 1), (1, 15, 64, 16, 2), (2, 16, 40, 8, 1), (1, 17, 72, 24, 3), (2, 31, 16, 32, 1),
          (1, 33, 48, 40, 2), (1, 63, 136, 16, 1), (2, 65, 64, 64, 4), (1, 129, 88, 16, 1), (3, 200, 32, 16, 2)]


@DT
@pytest.mark.parametrize("B,L,D,N,G", SHAPES)
def test_scan(B, L, D, N, G, dt):
    P = lib()
    x, gy, gh = scan_inputs(B, L, D, N, dt, G)
    check_scan(x, *P.pdssm_selscan_fwd(**x))
    check_scan_bwd(x, P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh), gy, gh)


@DT
@pytest.mark.parametrize("L,N", [(600, 16), (1500, 16), (1100, 32), (520, 64), (700, 8)])
def test_scan_cut_into_segments(L, N, dt):
    """One long sequence: its segments run side by side."""
    P = lib()
    x, gy, gh = scan_inputs(1, L, 40, N, dt, seed=2)
    check_scan(x, *P.pdssm_selscan_fwd(**x))
    check_scan_bwd(x, P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh), gy, gh)


@DT
@pytest.mark.parametrize("sp", [True, False])
@pytest.mark.parametrize("L", [40, 700])
def test_scan_without_what_is_optional(sp, L, dt):
    P = lib()
    x, gy, _ = scan_inputs(1, L, 48, 16, dt, state=False, z=False)
    del x["D"], x["dt_bias"]
    if not sp:
        x["dt"] = (x["dt"].float().abs() * 0.1).to(dt)
    check_scan(x, *P.pdssm_selscan_fwd(**x, softplus=sp), sp)
    g = P.pdssm_selscan_bwd(**x, g_y=gy, softplus=sp, want_h0=False)
    assert set(g) == {"g_x", "g_dt", "g_A", "g_B", "g_C", "g_D", "g_dt_bias"}
    check_scan_bwd(x, g, gy, None, sp)


@DT
@pytest.mark.parametrize("lens", LENGTHS + [(900, 0, 1, 130), (64,) * 12])
@pytest.mark.parametrize("N,G", [(16, 2), (40, 1)])
def test_scan_packed(dt, lens, N, G):
    P = lib()
    S, n, before, after = len(lens), sum(lens), 2, 70
    x, gy, gh = scan_inputs(1, n + before + after, 48, N, dt, G, S=S, seed=4)
    cu = bounds(lens) + before
    mark = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    y, hL = P.pdssm_selscan_fwd(**x, cu_seqlens=cu, out={"y": mark(x["x"])})
    g = P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, cu_seqlens=cu, out={
        "g_x": mark(gy), "g_dt": mark(gy), "g_z": mark(gy), "g_B": mark(x["Bm"]), "g_C": mark(x["Cm"])})
    for t in (y, g["g_x"], g["g_dt"], g["g_z"], g["g_B"].transpose(1, 2), g["g_C"].transpose(1, 2)):
        assert (t[:, :before] == 7).all() and (t[:, before + n:] == 7).all()
    sums = {}
    for i, m in enumerate(lens):
        at = slice(before + sum(lens[:i]), before + sum(lens[:i]) + m)
        if not m:
            assert torch.equal(hL[i], x["h0"][i]) and torch.equal(g["g_h0"][i], gh[i])
            continue
        xi = dict(x, h0=x["h0"][i:i + 1], **{k: x[k][:, at] for k in ("x", "dt", "z")}, **{k: x[k][:, :, at] for k in ("Bm", "Cm")})
        check_scan(xi, y[:, at], hL[i:i + 1])
        r = O.selscan_bwd(**scan_args(xi), g_y=bound(gy[:, at]), g_hL=bound(gh[i:i + 1]))
        for k in ("g_x", "g_dt", "g_z"):
            close(g[k][:, at], r[k], f"{k} of {i}")
        for k in ("g_B", "g_C"):
            close(g[k][:, :, at], r[k], f"{k} of {i}")
        close(g["g_h0"][i:i + 1], r["g_h0"], f"g_h0 of {i}")
        for k in ("g_A", "g_D", "g_dt_bias"):
            sums[k] = r[k] if k not in sums else sums[k] + r[k]
    for k in sums:
        close(g[k], sums[k], k)


def test_scan_of_whole_sequences_from_many_pieces():
    """Enough channels that no sequence is cut, while the states behind the gradient still come in pieces: batched, and packed."""
    P = lib()
    x, gy, gh = scan_inputs(48, 260, 256, 8, BF, seed=7)
    check_scan_bwd(x, P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh), gy, gh)
    lens = (130, 0, 129, 45)
    x, gy, gh = scan_inputs(1, sum(lens), 4096, 8, BF, S=4, seed=8)
    g = P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, cu_seqlens=bounds(lens))
    for i, m in enumerate(lens):
        at = slice(sum(lens[:i]), sum(lens[:i]) + m)
        if not m:
            assert torch.equal(g["g_h0"][i], gh[i])
            continue
        xi = dict(x, h0=x["h0"][i:i + 1], **{k: x[k][:, at] for k in ("x", "dt", "z")}, **{k: x[k][:, :, at] for k in ("Bm", "Cm")})
        r = O.selscan_bwd(**scan_args(xi), g_y=bound(gy[:, at]), g_hL=bound(gh[i:i + 1]))
        for k in ("g_x", "g_dt", "g_z"):
            close(g[k][:, at], r[k], f"{k} of {i}")
        for k in ("g_B", "g_C"):
            close(g[k][:, :, at], r[k], f"{k} of {i}")
        close(g["g_h0"][i:i + 1], r["g_h0"], f"g_h0 of {i}")


def test_rows_past_32_bits():
    """Tensors of more than 4 GiB: the last sequence of a packed call is what it is by itself."""
    P = lib()
    L, last, D, N = 270000, 70, 8192, 8
    r = torch.Generator("cuda").manual_seed(3)
    t = lambda *s: torch.randn(s, generator=r, device="cuda", dtype=BF)  # noqa: E731
    cu = torch.tensor([0, L - last, L], dtype=torch.int32).cuda()
    x, gy = t(1, L, D), t(1, L, D)
    tail = slice(L - last, L)
    w = torch.randn(D, 4, generator=r, device="cuda")
    y, xL = P.pdssm_conv_fwd(x, w, cu_seqlens=cu)
    y2, xL2 = P.pdssm_conv_fwd(x[:, tail].clone(), w)
    assert torch.equal(y[:, tail], y2) and torch.equal(xL[1:], xL2)
    g = P.pdssm_conv_bwd(x, w, gy, cu_seqlens=cu, out={"g_x": y})
    assert torch.equal(g["g_x"][:, tail], P.pdssm_conv_bwd(x[:, tail].clone(), w, gy[:, tail].clone())["g_x"])
    n = torch.randn(D, generator=r, device="cuda")
    assert torch.equal(P.pdssm_norm_fwd(x, n, out=y)[:, tail], P.pdssm_norm_fwd(x[:, tail].clone(), n))
    assert torch.equal(P.pdssm_norm_bwd(x, n, gy, out={"g_x": y})["g_x"][:, tail], P.pdssm_norm_bwd(x[:, tail].clone(), n, gy[:, tail].clone())["g_x"])
    del y
    A = -torch.exp(torch.randn(D, N, generator=r, device="cuda"))
    Bm, Cm = (t(1, L, 1, N).transpose(1, 2) for _ in range(2))
    part = dict(x=x[:, tail].clone(), dt=x[:, tail].clone(), A=A, Bm=Bm[:, :, tail], Cm=Cm[:, :, tail])
    y, hL = P.pdssm_selscan_fwd(x, x, A, Bm, Cm, cu_seqlens=cu)
    check_scan(part, y[:, tail], hL[1:])
    g = P.pdssm_selscan_bwd(x, x, A, Bm, Cm, gy, cu_seqlens=cu, out={"g_x": y})
    ref = O.selscan_bwd(**scan_args(part), g_y=bound(gy[:, tail]))
    for k in ("g_x", "g_dt"):
        close(g[k][:, tail], ref[k], k)
    for k in ("g_B", "g_C"):
        close(g[k][:, :, tail], ref[k], k)


@DT
def test_offsets_that_are_not_in_order(dt):
    """Offsets out of range or of order are cut to the rows: every call ends, and touches nothing outside its tensors (the
    guard rows around the outputs stay as they are); what comes before the first wrong offset is right."""
    P = lib()
    L, D, N = 700, 48, 16
    for off in ((0, 300, 5000, 700), (0, 300, 100, 700), (-50, 300, 250, 900), (0, 700, 0, 700, 0, 700, 0, 700), (700, 0, 700, 3)):
        S = len(off) - 1
        x, gy, gh = scan_inputs(1, L, D, N, dt, 2, S=S, seed=11)
        cu = torch.tensor(off, dtype=torch.int32).cuda()
        guard = lambda t, rows=8: torch.full((t.shape[0], t.shape[1] + 2 * rows, *t.shape[2:]), 7.0, dtype=t.dtype, device="cuda")  # noqa: E731
        full = {k: guard(gy) for k in ("y", "g_x", "g_dt", "g_z", "c", "cg")}
        mid = {k: t[:, 8:-8] for k, t in full.items()}
        y, hL = P.pdssm_selscan_fwd(**x, cu_seqlens=cu, out={"y": mid["y"]})
        P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, cu_seqlens=cu, out={k: mid[k] for k in ("g_x", "g_dt", "g_z")})
        c, cy, cx = conv_inputs(1, L, D, 4, dt, S=S)
        P.pdssm_conv_fwd(**c, cu_seqlens=cu, out={"y": mid["c"]})
        P.pdssm_conv_bwd(**c, g_y=cy, g_xL=cx, cu_seqlens=cu, out={"g_x": mid["cg"]})
        torch.cuda.synchronize()
        for t in full.values():
            assert (t[:, :8] == 7).all() and (t[:, -8:] == 7).all()
        if off[:2] == (0, 300) and off[2] != 100:
            one = dict(x, h0=x["h0"][:1], **{k: x[k][:, :300] for k in ("x", "dt", "z")}, **{k: x[k][:, :, :300] for k in ("Bm", "Cm")})
            check_scan(one, y[:, :300], hL[:1])


@DT
def test_scan_decays_of_all_sizes(dt):
    """Steps that forget everything, and steps that forget nothing."""
    P = lib()
    for shift, size in ((12.0, 0.1), (-30.0, 0.1), (-3.0, 3.0)):
        x, gy, gh = scan_inputs(2, 70, 32, 16, dt, size=size, seed=5)
        x["dt_bias"] = x["dt_bias"] + shift
        check_scan(x, *P.pdssm_selscan_fwd(**x))
        check_scan_bwd(x, P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh), gy, gh)
    x["A"] = torch.zeros_like(x["A"])   # a sum of everything
    check_scan(x, *P.pdssm_selscan_fwd(**x))
    check_scan_bwd(x, P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh), gy, gh)


@pytest.mark.parametrize("softplus_at", [-100.0, -40.0, -16.7, -16.0, -9.0, -5.0, -1.0, 0.0, 1.0, 15.0, 40.0, 1e4])
def test_step_sizes_keep_their_digits(softplus_at):
    """One token from zero with x = B = C = 1: y is the step itself, to a few steps of fp32."""
    P = lib()
    n = 4096
    raw = (torch.tensor(softplus_at) + torch.linspace(-0.5, 0.5, n) * (softplus_at != 0 or 1)).cuda()
    one = torch.ones(1, n, device="cuda")
    Bm = torch.zeros(1, 1, 8, device="cuda")
    Bm[..., 0] = 1
    y = P.pdssm_selscan_step(one, raw[None].contiguous(), torch.zeros(n, 8, device="cuda"), Bm, Bm, torch.zeros(1, n, 8, device="cuda"))
    want = np.logaddexp(0.0, f64(raw))
    err = np.abs(f64(y)[0] - want) / np.maximum(want, 1e-37)
    assert err.max() <= 12 * 2.0 ** -24 or softplus_at <= -100.0 and np.abs(f64(y)).max() <= 1e-37


# ---- single tokens

IDX = [None, [3, 0, 5, 1], [-1, 2, -7, 0], [4, 4, 9, 4], [6, 7, -1, 6]]


@DT
@pytest.mark.parametrize("idx", IDX)
@pytest.mark.parametrize("D,N,G", [(8, 8, 1), (136, 16, 1), (1032, 24, 3), (64, 64, 4), (48, 40, 2)])
def test_scan_step(dt, idx, D, N, G):
    P = lib()
    x, _, _ = scan_inputs(4, 1, D, N, dt, G, S=7, seed=6)
    row = {k: (t[:, 0] if k in ("x", "dt", "z") else t[:, :, 0] if k in ("Bm", "Cm") else t) for k, t in x.items() if k != "h0"}
    pool = x["h0"].clone()
    i = None if idx is None else torch.tensor(idx, dtype=torch.int32).cuda()
    y = P.pdssm_selscan_step(**row, state=pool, state_idx=i)
    seen = set()
    for b in range(4):
        s = b if idx is None else idx[b]
        if s < 0:
            assert (y[b] == 0).all()
        elif s >= 7 or s in seen:
            assert torch.isnan(y[b]).all()
        else:
            seen.add(s)
            one = {k: (t[b:b + 1] if k in ("x", "dt", "z", "Bm", "Cm") else t) for k, t in x.items()}
            one["h0"] = x["h0"][s:s + 1]
            check_scan(one, y[b:b + 1, None], pool[s:s + 1])
    for s in set(range(7)) - seen:
        assert torch.equal(pool[s], x["h0"][s])


@DT
@pytest.mark.parametrize("idx", IDX)
@pytest.mark.parametrize("D,W", [(8, 2), (1032, 4), (200, 3)])
def test_conv_step(dt, idx, D, W):
    P = lib()
    x, _, _ = conv_inputs(4, 1, D, W, dt, S=7)
    pool = x["x0"].clone()
    i = None if idx is None else torch.tensor(idx, dtype=torch.int32).cuda()
    y = P.pdssm_conv_step(x["x"][:, 0], x["w"], pool, bias=x["bias"], state_idx=i)
    seen = set()
    for b in range(4):
        s = b if idx is None else idx[b]
        if s < 0:
            assert (y[b] == 0).all()
        elif s >= 7 or s in seen:
            assert torch.isnan(y[b]).all()
        else:
            seen.add(s)
            ry, rx = conv_ref(dict(x, x=x["x"][b:b + 1], x0=x["x0"][s:s + 1]))
            close(y[b:b + 1, None], ry, "y")
            assert np.array_equal(f64(pool[s:s + 1]), O.Bound.of(rx).v)
    for s in set(range(7)) - seen:
        assert torch.equal(pool[s], x["x0"][s])


# ---- norm

def norm_inputs(shape, dt, gate, scale, per_head, seed=0, near=True):
    r = Gen(seed, dt)
    B, H, L, d = shape
    rows = (lambda: r.t(B, L, H, d).transpose(1, 2)) if near else (lambda: r.t(B, H, L, d))
    ws = (H, d) if per_head else (d,)
    x = dict(x=rows(), w=1.0 + r.f(*ws, size=0.2))
    if gate:
        x["z"] = rows()
    if scale:
        x["res_scale"] = r.f(*ws, size=0.5)
    return x, rows(), rows()


def norm_args(x):
    return {n: bound(t) for n, t in x.items()}


def check_norm(x, residual, gy, gate, eps=1e-5):
    P = lib()
    y = P.pdssm_norm_fwd(**x, gate=gate, residual=residual, eps=eps)
    eps32 = float(np.float32(eps))
    a = norm_args(x)
    close(y, O.norm_fwd(**a, gate=gate, residual=bound(residual), eps=eps32), "y")
    check(P.pdssm_norm_bwd(**x, g_y=gy, gate=gate, eps=eps), O.norm_bwd(**a, g_y=bound(gy), gate=gate, eps=eps32))


@DT
@pytest.mark.parametrize("d", [8, 16, 24, 32, 64, 72, 120, 256, 264, 512, 520, 768, 1000, 1032, 2048, 2056, 4096, 4104, 8192])
def test_norm_rows(d, dt):
    x, res, gy = norm_inputs((2, 1, 5, d), dt, "after", True, False)
    check_norm(x, res, gy, "after")


@DT
@pytest.mark.parametrize("gate", [None, "before", "after"])
@pytest.mark.parametrize("scale,residual", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("shape,near", [((2, 3, 7, 32), True), ((1, 5, 70, 64), False), ((3, 24, 11, 40), True), ((2, 4, 3, 520), True)])
def test_norm(shape, near, gate, scale, residual, dt):
    for per_head in (True, False):
        x, res, gy = norm_inputs(shape, dt, gate, scale, per_head, near=near, seed=2)
        check_norm(x, res if residual else None, gy, gate)


@DT
def test_norm_many_rows(dt):
    """More rows than a gradient has workgroups, more parts than one round of sums takes."""
    x, res, gy = norm_inputs((2, 1, 9001, 8), dt, "before", True, False)
    check_norm(x, res, gy, "before")
    x, res, gy = norm_inputs((1, 6, 3001, 16), dt, "after", True, False, near=False)
    check_norm(x, res, gy, "after")


@DT
def test_norm_of_zeros_and_large_rows(dt):
    x, res, gy = norm_inputs((1, 1, 4, 64), dt, None, False, False)
    x["x"][:, :, 0] = 0
    x["x"][:, :, 1] *= 1e15
    x["x"][:, :, 2] *= 1e-15
    check_norm(x, res, gy, None, eps=1e-6)


# ---- layouts, streams, graphs

def strided(t, where="slice"):
    """The same values, rows of a wider tensor."""
    wide = torch.empty(*t.shape[:-1], t.shape[-1] * 2 + 16, dtype=t.dtype, device=t.device)
    out = wide[..., 8:8 + t.shape[-1]]
    out.copy_(t)
    return out


@DT
def test_strided_and_broadcast_inputs(dt):
    """Slices of wider rows, a batch that shares one row of inputs, step-major and head-major groups: the same results, bit for bit."""
    P = lib()
    x, gy, gh = scan_inputs(3, 50, 48, 16, dt, 2)
    y, hL = P.pdssm_selscan_fwd(**x)
    g = P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh)
    s = {k: (strided(t) if k in ("x", "dt", "z", "Bm", "Cm") else t) for k, t in x.items()}
    y2, hL2 = P.pdssm_selscan_fwd(**s, out={"y": strided(y)})
    g2 = P.pdssm_selscan_bwd(**s, g_y=strided(gy), g_hL=gh)
    assert torch.equal(y, y2) and torch.equal(hL, hL2) and all(torch.equal(g[k], g2[k]) for k in g)
    s = dict(x, Bm=x["Bm"].contiguous(), Cm=x["Cm"].contiguous())
    assert torch.equal(P.pdssm_selscan_fwd(**s)[0], y)
    one = {k: (t[:1] if k in ("x", "dt", "z", "Bm", "Cm") else t) for k, t in x.items()}
    wide = {k: (t.expand(3, *t.shape[1:]) if k in ("x", "dt", "z", "Bm", "Cm") else t) for k, t in one.items()}
    full = {k: (t.contiguous() if k in ("x", "dt", "z", "Bm", "Cm") else t) for k, t in wide.items()}
    assert torch.equal(P.pdssm_selscan_fwd(**wide)[0], P.pdssm_selscan_fwd(**full)[0])
    gw, gf = (P.pdssm_selscan_bwd(**t, g_y=gy, g_hL=gh) for t in (wide, full))
    assert all(torch.equal(gw[k], gf[k]) for k in gw)
    c, gy, gx = conv_inputs(2, 50, 48, 4, dt)
    y, xL = P.pdssm_conv_fwd(**c)
    y2, xL2 = P.pdssm_conv_fwd(**dict(c, x=strided(c["x"])), out={"y": strided(y)})
    assert torch.equal(y, y2) and torch.equal(xL, xL2)
    g, g2 = P.pdssm_conv_bwd(**c, g_y=gy, g_xL=gx), P.pdssm_conv_bwd(**dict(c, x=strided(c["x"])), g_y=strided(gy), g_xL=gx)
    assert all(torch.equal(g[k], g2[k]) for k in g)
    n, res, gy = norm_inputs((2, 3, 9, 64), dt, "after", True, True)
    y = P.pdssm_norm_fwd(**n, gate="after", residual=res)
    m = dict(n, x=strided(n["x"]), z=strided(n["z"]))
    assert torch.equal(P.pdssm_norm_fwd(**m, gate="after", residual=strided(res), out=strided(y)), y)
    wide = gy[:1].expand_as(gy)   # a gradient that every sequence shares
    g, g2 = P.pdssm_norm_bwd(**n, g_y=wide, gate="after"), P.pdssm_norm_bwd(**m, g_y=wide.contiguous(), gate="after")
    assert all(torch.equal(g[k], g2[k]) for k in ("g_x", "g_z"))
    # sums over rows run in the order in which the heads of x lie: both within the bound, not the same
    ref = O.norm_bwd(**norm_args(n), g_y=bound(wide), gate="after", eps=float(np.float32(1e-5)))
    check(g, ref)
    check(g2, ref)


@DT
def test_layer_of_all_three(dt):
    """Norm, convolution, scan, gated norm with the residual, as a layer calls them: a prompt in one call, in two
    with the states passed on, packed, and token by token agree with one another, and with the oracle's layer."""
    P = lib()
    r = Gen(9, dt)
    B, L, D, N, W, cut = 2, 90, 64, 16, 4, 37
    x, w1, w2, sc = r.t(B, L, D), 1 + r.f(D, size=0.1), 1 + r.f(D, size=0.1), r.f(D, size=0.3)
    wc, bc = r.f(D, W, size=0.5), r.f(D, size=0.1)
    p = dict(A=-torch.exp(r.f(D, N, size=0.5)), D=r.f(D), dt_bias=r.f(D) - 3)
    dtr, z = r.t(B, L, D), r.t(B, L, D)
    Bm, Cm = r.t(B, L, 1, N).transpose(1, 2), r.t(B, L, 1, N).transpose(1, 2)

    def prompt(s, x0=None, h0=None, cu=None, flat=False):
        f = (lambda t: t.reshape(1, -1, D)) if flat else (lambda t: t)
        fb = (lambda t: t.transpose(1, 2).reshape(1, -1, 1, N).transpose(1, 2)) if flat else (lambda t: t)
        u, c0 = P.pdssm_conv_fwd(P.pdssm_norm_fwd(f(x[:, s]), w1), wc, bias=bc, x0=x0, cu_seqlens=cu)
        y, h = P.pdssm_selscan_fwd(u, f(dtr[:, s]), p["A"], fb(Bm[:, :, s]), fb(Cm[:, :, s]), D=p["D"], dt_bias=p["dt_bias"],
                                   h0=h0, cu_seqlens=cu)
        return P.pdssm_norm_fwd(y, w2, z=f(z[:, s]), gate="after", residual=f(x[:, s]), res_scale=sc), c0, h

    whole, c1, h1 = prompt(slice(0, L))
    a, c0, h0 = prompt(slice(0, cut))
    b, c2, h2 = prompt(slice(cut, L), c0, h0)
    packed, c3, h3 = prompt(slice(0, L), cu=torch.tensor([0, L, 2 * L], dtype=torch.int32).cuda(), flat=True)
    tokens = []
    c4, h4 = c0.clone(), h0.clone()
    for t in range(cut, L):
        u = P.pdssm_conv_step(P.pdssm_norm_fwd(x[:, t:t + 1], w1)[:, 0], wc, c4, bias=bc)
        y = P.pdssm_selscan_step(u, dtr[:, t], p["A"], Bm[:, :, t], Cm[:, :, t], h4, D=p["D"], dt_bias=p["dt_bias"])
        tokens.append(P.pdssm_norm_fwd(y[:, None], w2, z=z[:, t:t + 1], gate="after", residual=x[:, t:t + 1], res_scale=sc))
    # the same cells by other roads: fp32 roundings apart, and in bf16 a step of an intermediate may turn over
    tol = 2e-5 if dt == F32 else 0.06
    near = lambda p, q: float((p.double() - q.double()).abs().max()) <= tol * (1 + float(q.double().abs().max()))  # noqa: E731
    assert near(torch.cat([a, b], 1), whole) and near(torch.cat([a] + tokens, 1), whole) and near(packed.reshape(B, L, D), whole)
    assert torch.equal(c1, c2) and torch.equal(c1, c3) and torch.equal(c1, c4)
    assert near(h2, h1) and near(h3, h1) and near(h4, h1)
    if dt == F32:
        n = O.norm_fwd(f64(x)[:, None], f64(w1))[:, 0]
        u, _ = O.conv_fwd(n, f64(wc), f64(bc))
        y, _, _ = O.selscan_fwd(u, f64(dtr), f64(p["A"]), f64(Bm), f64(Cm), f64(p["D"]), None, f64(p["dt_bias"]))
        ref = O.norm_fwd(y[:, None], f64(w2), f64(z)[:, None], "after", f64(x)[:, None], f64(sc))[:, 0]
        assert np.abs(f64(whole) - ref).max() <= 2e-5 * (1 + np.abs(ref).max())


def test_norm_behind_linear_attention():
    """The gated norm of every head's output, in the layout that pdssm_linattn_fwd writes."""
    P = lib()
    r = Gen(10, BF)
    B, H, L, d = 2, 4, 100, 64
    q, k, v, z = (r.t(B, L, H, d).transpose(1, 2) for _ in range(4))
    o, _ = P.pdssm_linattn_fwd(q, k, v, -torch.rand(B, L, H, device="cuda").transpose(1, 2) * 0.1)
    w = 1 + r.f(H, d, size=0.1)
    y = P.pdssm_norm_fwd(o, w, z=z, gate="after")
    assert y.stride() == o.stride()
    close(y, O.norm_fwd(bound(o), f64(w), bound(z), "after", eps=float(np.float32(1e-5))), "y")
    g = P.pdssm_norm_bwd(o, w, z, z=z, gate="after")
    back = P.pdssm_linattn_bwd(q, k, v, -torch.ones(H, device="cuda") * 0.1, g["g_x"])
    assert all(torch.isfinite(t).all() for t in back.values())


def calls(dt, seed=0):
    """Every entry point once, as functions of nothing that write to outputs of their own and return them."""
    P = lib()
    x, gy, gh = scan_inputs(1, 700, 48, 16, dt, 2, seed=seed)
    c, cy, cx = conv_inputs(2, 70, 48, 4, dt, seed=seed)
    n, res, ny = norm_inputs((2, 3, 40, 64), dt, "before", True, True, seed=seed)
    row = {k: (t[:, 0] if k in ("x", "dt", "z") else t[:, :, 0] if k in ("Bm", "Cm") else t) for k, t in x.items() if k != "h0"}
    pool, cpool = x["h0"].clone(), c["x0"].clone()

    def step():
        pool.copy_(x["h0"])
        cpool.copy_(c["x0"])
        return [P.pdssm_selscan_step(**row, state=pool), pool, P.pdssm_conv_step(c["x"][:, 0], c["w"], cpool), cpool]

    return [lambda: list(P.pdssm_selscan_fwd(**x)), lambda: list(P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh).values()),
            lambda: list(P.pdssm_conv_fwd(**c)), lambda: list(P.pdssm_conv_bwd(**c, g_y=cy, g_xL=cx).values()),
            lambda: [P.pdssm_norm_fwd(**n, gate="before", residual=res)],
            lambda: list(P.pdssm_norm_bwd(**n, g_y=ny, gate="before").values()), step]


@DT
def test_same_from_run_to_run_and_on_another_stream(dt):
    side = torch.cuda.Stream()
    for i, f in enumerate(calls(dt)):
        first = [t.clone() for t in f()]
        assert all(torch.equal(a, b) for a, b in zip(first, f())), i
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = f()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again)), i


@DT
def test_captured_and_replayed(dt):
    """Two captured runs of every call, each with a workspace of its pool, replayed in turn with eager calls between."""
    fs, gs = calls(dt), calls(dt, seed=1)
    eager = [[t.clone() for t in f()] for f in fs], [[t.clone() for t in g()] for g in gs]
    torch.cuda.synchronize()
    graphs = []
    for side in (fs, gs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [f() for f in side]
        graphs.append((g, outs))
    for turn in range(3):
        for (g, outs), want in zip(graphs, eager):
            for o in outs:
                for t in o:
                    t.fill_(3.0)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for o, w in zip(outs, want):
                assert all(torch.equal(a, b) for a, b in zip(o, w))
            for f, w in zip(fs, eager[0]):
                assert all(torch.equal(a, b) for a, b in zip(f(), w))


@DT
def test_given_workspace(dt):
    """A workspace with anything in it gives what a new one does; one that is a byte short is refused."""
    P = lib()
    x, gy, gh = scan_inputs(1, 700, 48, 16, dt, 2)
    y, hL = P.pdssm_selscan_fwd(**x)
    ws = torch.full((1 << 24,), 0xff, dtype=torch.uint8, device="cuda")
    y2, hL2 = P.pdssm_selscan_fwd(**x, workspace=ws)
    assert torch.equal(y, y2) and torch.equal(hL, hL2) and P.workspace_error_flag(ws) == 0
    ws.fill_(0xff)
    a, b = P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh), P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, workspace=ws)
    assert all(torch.equal(a[k], b[k]) for k in a) and P.workspace_error_flag(ws) == 0
    c, cy, cx = conv_inputs(2, 70, 48, 4, dt)
    ws.fill_(0xff)
    a, b = P.pdssm_conv_bwd(**c, g_y=cy, g_xL=cx), P.pdssm_conv_bwd(**c, g_y=cy, g_xL=cx, workspace=ws)
    assert all(torch.equal(a[k], b[k]) for k in a) and P.workspace_error_flag(ws) == 0
    n, _, ny = norm_inputs((2, 3, 40, 64), dt, "before", True, True)
    ws.fill_(0xff)
    a, b = P.pdssm_norm_bwd(**n, g_y=ny, gate="before"), P.pdssm_norm_bwd(**n, g_y=ny, gate="before", workspace=ws)
    assert all(torch.equal(a[k], b[k]) for k in a) and P.workspace_error_flag(ws) == 0
    for f in (lambda w: P.pdssm_selscan_fwd(**x, workspace=w), lambda w: P.pdssm_conv_bwd(**c, g_y=cy, workspace=w),
              lambda w: P.pdssm_norm_bwd(**n, g_y=ny, gate="before", workspace=w)):
        with pytest.raises(ValueError, match="needed"):
            f(ws[:64])


@DT
def test_workspaces_of_the_size_asked_for(dt):
    """The bytes that the queries name are enough, and the bytes behind them stay as they are."""
    P = lib()
    bf = dt == BF

    def room(n):
        whole = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        return whole, whole[:n]

    for B, L, pack in ((1, 700, None), (2, 130, None), (1, 700, (5, 0, 600, 95))):
        S = len(pack) if pack else B
        x, gy, gh = scan_inputs(B, L, 48, 16, dt, 2, S=S)
        cu = bounds(pack) if pack else None
        n = P.selscan_workspace_bytes(S, L, 48, 16, 2, bf, pack is not None)
        if n:
            whole, ws = room(n)
            P.pdssm_selscan_fwd(**x, cu_seqlens=cu, workspace=ws)
            assert (whole[n:] == 0x5a).all()
        n = P.selscan_bwd_workspace_bytes(S, L, 48, 16, 2, bf, pack is not None)
        whole, ws = room(n)
        P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, cu_seqlens=cu, workspace=ws)
        assert (whole[n:] == 0x5a).all()
        c, cy, cx = conv_inputs(B, L, 48, 4, dt, S=S)
        n = P.conv_bwd_workspace_bytes(S, L, 48, 4, bf, pack is not None)
        whole, ws = room(n)
        P.pdssm_conv_bwd(**c, g_y=cy, g_xL=cx, cu_seqlens=cu, workspace=ws)
        assert (whole[n:] == 0x5a).all()
    for per_head in (True, False):
        m, _, ny = norm_inputs((2, 3, 400, 64), dt, "before", True, per_head)
        n = P.norm_bwd_workspace_bytes(2, 3, 400, 64, bf, per_head)
        whole, ws = room(n)
        P.pdssm_norm_bwd(**m, g_y=ny, gate="before", workspace=ws)
        assert (whole[n:] == 0x5a).all()


@DT
def test_rows_outside_the_sequences_do_not_matter(dt):
    """Not-a-number and infinity before the first and behind the last sequence change nothing."""
    P = lib()
    lens, before, after = (70, 0, 33, 600), 5, 40
    S, n = len(lens), sum((70, 0, 33, 600))
    x, gy, gh = scan_inputs(1, before + n + after, 48, 16, dt, 2, S=S)
    c, cy, cx = conv_inputs(1, before + n + after, 48, 4, dt, S=S)
    cu = bounds(lens) + before
    got = []
    for fill in (0.0, float("nan"), float("inf")):
        for t in (x["x"], x["dt"], x["z"], gy, c["x"], cy):
            t[:, :before] = fill
            t[:, before + n:] = fill
        for k in ("Bm", "Cm"):
            x[k][:, :, :before] = fill
            x[k][:, :, before + n:] = fill
        y, hL = P.pdssm_selscan_fwd(**x, cu_seqlens=cu)
        g = P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, cu_seqlens=cu)
        v, vL = P.pdssm_conv_fwd(**c, cu_seqlens=cu)
        e = P.pdssm_conv_bwd(**c, g_y=cy, g_xL=cx, cu_seqlens=cu)
        rows = lambda t: t[:, before:before + n]  # noqa: E731
        heads = lambda t: t[:, :, before:before + n]  # noqa: E731
        got.append([rows(y), hL, rows(v), vL, rows(e["g_x"]), e["g_w"], e["g_bias"], e["g_x0"], heads(g["g_B"]), heads(g["g_C"])]
                   + [rows(g[k]) for k in ("g_x", "g_dt", "g_z")] + [g[k] for k in ("g_A", "g_D", "g_dt_bias", "g_h0")])
    for other in got[1:]:
        assert all(torch.equal(p, q) for p, q in zip(got[0], other))


def test_refused_on_the_device():
    """What only the C ABI sees: overlaps, alignment, limits."""
    P = lib()
    x, gy, gh = scan_inputs(1, 20, 16, 8, F32)
    with pytest.raises(P.PdssmError, match="overlaps"):
        P.pdssm_selscan_fwd(**x, out={"y": x["x"]})
    with pytest.raises(P.PdssmError, match="overlap"):
        P.pdssm_selscan_bwd(**x, g_y=gy, out={"g_x": (t := torch.empty_like(gy)), "g_dt": t})
    with pytest.raises(P.PdssmError, match="aligned"):
        P.pdssm_selscan_fwd(**dict(x, x=torch.zeros(1, 20, 17, device="cuda")[..., 1:]))
    with pytest.raises(P.PdssmError, match="multiple of 8"):
        P.pdssm_selscan_fwd(torch.zeros(1, 4, 16, device="cuda"), torch.zeros(1, 4, 16, device="cuda"), -torch.ones(16, 12, device="cuda"),
                            torch.zeros(1, 1, 4, 12, device="cuda"), torch.zeros(1, 1, 4, 12, device="cuda"))
    c, cy, cx = conv_inputs(1, 20, 16, 4, F32)
    with pytest.raises(P.PdssmError, match="W=5"):
        P.pdssm_conv_fwd(c["x"], torch.zeros(16, 5, device="cuda"))
    with pytest.raises(P.PdssmError, match="overlaps"):
        P.pdssm_conv_fwd(**c, out={"y": c["x"]})
    with pytest.raises(P.PdssmError, match="rows of output"):
        P.pdssm_conv_fwd(**c, out={"y": torch.zeros(1, 1, 16, device="cuda").expand(1, 20, 16)})
    n, res, ny = norm_inputs((1, 1, 4, 64), F32, None, False, False)
    with pytest.raises(P.PdssmError, match="eps"):
        P.pdssm_norm_fwd(**n, eps=0.0)
    with pytest.raises(P.PdssmError, match="overlaps"):
        P.pdssm_norm_fwd(**n, residual=res, out=res)
