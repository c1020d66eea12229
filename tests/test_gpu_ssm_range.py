"""The selective layer at the ends of its inputs' range: steps and gates of a
type's lowest value, which switch a token off, and of infinity.

softplus and the sigmoid of anything below about -104 are zero in fp32, so a call
with such a value in some places has to give what the same call gives with
-1e4 there, bit for bit (zeros of either sign are equal): no tolerances.
"""

import pytest

from tests._gpu import lib
from tests.test_gpu_ssm import DT, F32, Gen, bounds, conv_inputs, norm_inputs, scan_inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

OFF = -1e4


def lowest(dt):
    return float(torch.finfo(dt).min)


LOW = pytest.mark.parametrize("low", [lowest, lambda dt: -2.5e38, lambda dt: float("-inf")], ids=["lowest", "-2.5e38", "-inf"])
FINITE = pytest.mark.parametrize("low", [lowest, lambda dt: -2.5e38], ids=["lowest", "-2.5e38"])


def put(t, mask, value):
    return t.masked_fill(mask, value)


def mask_of(t, seed=0):
    """A fifth of the places; whole tokens too, the first and the last among them (of rows with heads: whole heads)."""
    g = torch.Generator().manual_seed(seed)
    m = torch.rand(t.shape, generator=g) < 0.2
    m |= (torch.rand(t.shape[:-1], generator=g) < 0.1)[..., None]
    m[:, 0] = m[:, -1] = True
    return m.cuda()


def same(a, b, names=None):
    for n in names or a:
        assert not torch.isnan(a[n]).any(), n
        assert torch.equal(a[n], b[n]), n


SHAPES = [((2, 70, 48, 16, 2), None), ((1, 700, 40, 64, 1), None), ((1, 700, 48, 24, 2), (5, 0, 600, 33, 62)), ((1, 1, 8, 8, 1), None)]


def scan_all(x, gy, gh, cu=None):
    P = lib()
    y, hL = P.pdssm_selscan_fwd(**x, cu_seqlens=cu)
    return dict(P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, cu_seqlens=cu), y=y, h_L=hL)


@DT
@LOW
@pytest.mark.parametrize("shape,lens", SHAPES)
def test_steps_of_the_lowest_value(shape, lens, low, dt):
    B, L, D, N, G = shape
    x, gy, gh = scan_inputs(B, L, D, N, dt, G, S=len(lens) if lens else B)
    cu = bounds(lens) if lens else None
    m = mask_of(x["dt"])
    a, b = (scan_all(dict(x, dt=put(x["dt"], m, v)), gy, gh, cu) for v in (low(dt), OFF))
    same(a, b)
    assert (a["g_dt"][m] == 0).all()
    # every token off: the state passes through as it is, and its gradient too
    a = scan_all(dict(x, dt=torch.full_like(x["dt"], low(dt))), gy, None, cu)
    assert torch.equal(a["h_L"], x["h0"]) and (a["g_dt"] == 0).all() and (a["g_A"] == 0).all()
    # and by the channels' own bias, with which fp32's lowest value gives infinity
    bias = x["dt_bias"].clone()
    bias[::3] = lowest(F32)
    a = scan_all(dict(x, dt=put(x["dt"], m, low(dt)), dt_bias=bias), gy, gh, cu)
    bias = bias.clone()
    bias[::3] = OFF
    same(a, scan_all(dict(x, dt=put(x["dt"], m, OFF), dt_bias=bias), gy, gh, cu))
    assert torch.equal(a["h_L"][:, ::3], x["h0"][:, ::3])


@DT
@FINITE
@pytest.mark.parametrize("shape,lens", SHAPES)
def test_scan_gates_of_the_lowest_value(shape, lens, low, dt):
    B, L, D, N, G = shape
    x, gy, gh = scan_inputs(B, L, D, N, dt, G, S=len(lens) if lens else B)
    cu = bounds(lens) if lens else None
    m = mask_of(x["z"])
    a, b = (scan_all(dict(x, z=put(x["z"], m, v)), gy, gh, cu) for v in (low(dt), OFF))
    same(a, b)
    assert (a["y"][m] == 0).all() and (a["g_z"][m] == 0).all()


def test_gates_of_large_values():
    """From about 17 up the sigmoid is one in fp32: the gate is z itself, and its slope one."""
    P = lib()
    x, gy, _ = scan_inputs(2, 70, 48, 16, F32, 2, z=False)
    x["x"], x["h0"], gy = x["x"] * 2.0 ** -10, x["h0"] * 2.0 ** -10, gy * 2.0 ** -10
    plain, hL = P.pdssm_selscan_fwd(**x)
    z = torch.full_like(gy, 2.5e38)
    y, h = P.pdssm_selscan_fwd(**x, z=z)
    assert torch.equal(y, plain * z) and torch.equal(h, hL) and torch.isfinite(y).all()
    g = P.pdssm_selscan_bwd(**x, z=z, g_y=gy)
    assert all(torch.isfinite(t).all() for n, t in g.items() if n != "g_A")
    n, _, ny = norm_inputs((2, 3, 7, 64), F32, None, False, True)
    n["w"], ny = n["w"] * 2.0 ** -10, ny * 2.0 ** -10
    plain = P.pdssm_norm_fwd(**n)
    z = torch.full_like(plain, 2.5e38)
    assert torch.equal(P.pdssm_norm_fwd(**n, z=z, gate="after"), plain * z)
    assert all(torch.isfinite(t).all() for t in P.pdssm_norm_bwd(**n, z=z, gate="after", g_y=ny).values())
    v = torch.full((1, 3, 8), 2.5e38, device="cuda")
    w = torch.tensor([[0.0, 1.0]]).expand(8, 2).contiguous().cuda()
    assert torch.equal(P.pdssm_conv_fwd(v, w)[0], v)
    assert (P.pdssm_conv_bwd(v, w, torch.ones_like(v))["g_x"] == 1).all()


@DT
@LOW
@pytest.mark.parametrize("D,N,G", [(8, 8, 1), (136, 16, 1), (96, 24, 3), (64, 64, 4)])
def test_tokens_of_the_lowest_value(D, N, G, low, dt):
    """One token: the state that it finds is left as it is."""
    P = lib()
    x, _, _ = scan_inputs(4, 1, D, N, dt, G, S=6)
    row = {k: (t[:, 0] if k in ("x", "dt", "z") else t[:, :, 0] if k in ("Bm", "Cm") else t) for k, t in x.items() if k != "h0"}
    got = []
    for v in (low(dt), OFF):
        pool = x["h0"].clone()
        y = P.pdssm_selscan_step(**dict(row, dt=torch.full_like(row["dt"], v)), state=pool)
        assert torch.equal(pool, x["h0"])
        got.append(y)
    assert not torch.isnan(got[0]).any() and torch.equal(*got)
    if low(dt) > float("-inf"):
        pool, kept = x["h0"].clone(), x["h0"].clone()
        P.pdssm_selscan_step(**row, state=kept)
        assert (P.pdssm_selscan_step(**dict(row, z=torch.full_like(row["z"], low(dt))), state=pool) == 0).all()
        assert torch.equal(pool, kept)


@DT
@FINITE
@pytest.mark.parametrize("W", [2, 4])
def test_convolution_of_the_lowest_value(W, low, dt):
    """Taps of which only the last is not zero, so that a sum is one row's value."""
    P = lib()
    x, gy, gx = conv_inputs(2, 70, 48, W, dt)
    x["w"] = torch.zeros_like(x["w"])
    x["w"][:, -1] = 1.0
    del x["bias"]
    m = mask_of(x["x"])
    calls = []
    for v in (low(dt), OFF):
        c = dict(x, x=put(x["x"], m, v))
        pool = c["x0"].clone()
        step = P.pdssm_conv_step(c["x"][:, 0], c["w"], pool)
        g = P.pdssm_conv_bwd(**c, g_y=gy, g_xL=gx)
        calls.append(dict(y=P.pdssm_conv_fwd(**c)[0], step=step, g_x=g["g_x"], g_bias=g["g_bias"], g_x0=g["g_x0"]))
    same(*calls)
    assert (calls[0]["y"][m] == 0).all()


@DT
@FINITE
@pytest.mark.parametrize("gate", ["before", "after"])
@pytest.mark.parametrize("d", [8, 64, 520, 2056])
def test_norm_gates_of_the_lowest_value(d, gate, low, dt):
    P = lib()
    x, res, gy = norm_inputs((2, 2, 5, d), dt, gate, True, True)
    m = mask_of(x["z"])
    calls = []
    for v in (low(dt), OFF):
        c = dict(x, z=put(x["z"], m, v))
        calls.append(dict(P.pdssm_norm_bwd(**c, g_y=gy, gate=gate), y=P.pdssm_norm_fwd(**c, gate=gate, residual=res)))
    same(*calls)


@DT
def test_what_is_no_number_stays_one(dt):
    """A step that is not a number spoils its own channel from its token on, and is not taken for zero."""
    P = lib()
    x, _, _ = scan_inputs(2, 70, 48, 16, dt, 2)
    y, hL = P.pdssm_selscan_fwd(**x)
    bad = x["dt"].clone()
    bad[1, 40, 5] = float("nan")
    y2, hL2 = P.pdssm_selscan_fwd(**dict(x, dt=bad))
    assert torch.isnan(y2[1, 40:, 5]).all() and torch.isnan(hL2[1, 5]).all()
    rest = torch.ones_like(y, dtype=torch.bool)
    rest[1, 32:, 5] = False
    assert torch.equal(y2[rest], y[rest])
    ch = torch.ones_like(hL, dtype=torch.bool)
    ch[1, 5] = False
    assert torch.equal(hL2[ch], hL[ch])
    row = {k: (t[:, 0] if k in ("x", "dt", "z") else t[:, :, 0] if k in ("Bm", "Cm") else t) for k, t in x.items() if k != "h0"}
    pool, none = x["h0"].clone(), row["dt"].clone()
    none[0, 3] = float("nan")
    y = P.pdssm_selscan_step(**dict(row, dt=none), state=pool)
    assert torch.isnan(y[0, 3]) and torch.isnan(pool[0, 3]).all()
    assert int(torch.isnan(y).sum()) == 1 and int(torch.isnan(pool).sum()) == 16


@DT
@pytest.mark.parametrize("shape,lens", [((2, 70, 48, 24, 2), None), ((1, 700, 40, 40, 1), None), ((1, 700, 48, 16, 2), (5, 0, 600, 33, 62)),
                                        ((1, 40, 16, 64, 1), None)])
def test_steps_of_the_highest_value(shape, lens, dt):
    """Steps without an input that forget everything, many in a row: their sum passes fp32.  A step of 1e4 forgets
    everything too where A is below -0.02, and nothing where A is zero."""
    P = lib()
    B, L, D, N, G = shape
    x, gy, gh = scan_inputs(B, L, D, N, dt, G, S=len(lens) if lens else B)
    x["A"] = x["A"].clamp(max=-0.02)
    cu = bounds(lens) if lens else None
    m = mask_of(x["dt"])
    x["x"] = put(x["x"], m, 0.0)
    high = float(torch.finfo(dt).max)
    a, b = (scan_all(dict(x, dt=put(x["dt"], m, v)), gy, gh, cu) for v in (high, 1e4))
    for g in (a, b):
        g["g_x"][m] = 0   # (a step's size times what follows from it)
    same(a, b)
    x["A"][:, ::3] = 0.0
    a, b = (P.pdssm_selscan_fwd(**dict(x, dt=put(x["dt"], m, v)), cu_seqlens=cu) for v in (high, 1e4))
    same(dict(zip("yh", a)), dict(zip("yh", b)))
    row = {k: (t[:, 0] if k in ("x", "dt", "z") else t[:, :, 0] if k in ("Bm", "Cm") else t) for k, t in x.items() if k != "h0"}
    row["x"] = torch.zeros_like(row["x"])
    got = []
    for v in (high, 1e4):
        pool = x["h0"].clone()
        y = P.pdssm_selscan_step(**dict(row, dt=torch.full_like(row["dt"], v)), state=pool)
        got.append(dict(y=y, pool=pool))
    same(*got)
    assert torch.equal(pool[..., ::3], x["h0"][..., ::3]) and (pool[:B, :, 1::3] == 0).all()


@DT
def test_decays_of_the_lowest_value(dt):
    """A state that every step forgets is kept by a step of zero."""
    P = lib()
    x, gy, gh = scan_inputs(1, 300, 48, 24, dt, 2)
    m = mask_of(x["dt"])
    x["dt"] = put(x["dt"], m, lowest(dt))
    got = []
    for v in (lowest(F32), -1e8):   # (other steps are above 1e-5: both forget everything)
        x["A"][:, ::3] = v
        y, hL = P.pdssm_selscan_fwd(**x)
        pool = x["h0"].clone()
        row = {k: (t[:, 0] if k in ("x", "dt", "z") else t[:, :, 0] if k in ("Bm", "Cm") else t) for k, t in x.items() if k != "h0"}
        step = P.pdssm_selscan_step(**row, state=pool)
        got.append(dict(y=y, h_L=hL, step=step, pool=pool))
    same(*got)
    assert torch.equal(pool, x["h0"])   # (the first token is switched off)


@DT
def test_sequences_without_rows(dt):
    """Packed sequences none of which has a row: states pass through, rows stay as they are, weights have no gradient."""
    P = lib()
    for L in (1, 700):
        x, gy, gh = scan_inputs(1, L, 48, 16, dt, 2, S=3)
        for at in (0, L):
            cu = torch.full((4,), at, dtype=torch.int32, device="cuda")
            mark = lambda t: torch.full_like(t, 7.0)  # noqa: E731
            y, hL = P.pdssm_selscan_fwd(**x, cu_seqlens=cu, out={"y": mark(gy)})
            g = P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, cu_seqlens=cu, out={
                "g_x": mark(gy), "g_dt": mark(gy), "g_z": mark(gy), "g_B": mark(x["Bm"]), "g_C": mark(x["Cm"])})
            assert torch.equal(hL, x["h0"]) and torch.equal(g["g_h0"], gh)
            assert all((t == 7).all() for t in (y, g["g_x"], g["g_dt"], g["g_z"], g["g_B"], g["g_C"]))
            assert all((g[k] == 0).all() for k in ("g_A", "g_D", "g_dt_bias"))
            c, cy, cx = conv_inputs(1, L, 48, 4, dt, S=3)
            y, xL = P.pdssm_conv_fwd(**c, cu_seqlens=cu, out={"y": mark(cy)})
            g = P.pdssm_conv_bwd(**c, g_y=cy, g_xL=cx, cu_seqlens=cu, out={"g_x": mark(cy)})
            assert torch.equal(xL, c["x0"]) and torch.equal(g["g_x0"], cx)
            assert (y == 7).all() and (g["g_x"] == 7).all() and (g["g_w"] == 0).all() and (g["g_bias"] == 0).all()


@DT
@pytest.mark.parametrize("d", [64, 1032])
def test_rows_whose_squares_pass_fp32(d, dt):
    """They have a norm of zero and no gradient; their neighbours are what they are by themselves."""
    P = lib()
    x, res, gy = norm_inputs((1, 2, 6, d), dt, None, False, True)
    x["x"][:, :, 2] = x["x"][:, :, 2].sign() * 1e20
    y, g = P.pdssm_norm_fwd(**x, residual=res), P.pdssm_norm_bwd(**x, g_y=gy)
    assert torch.equal(y[:, :, 2], res[:, :, 2]) and (g["g_x"][:, :, 2] == 0).all()
    keep = [0, 1, 3, 4, 5]
    part = dict(x, x=x["x"][:, :, keep].contiguous())
    y2, g2 = P.pdssm_norm_fwd(**part, residual=res[:, :, keep].contiguous()), P.pdssm_norm_bwd(**part, g_y=gy[:, :, keep].contiguous())
    assert torch.equal(y[:, :, keep], y2) and torch.equal(g["g_x"][:, :, keep], g2["g_x"])
    assert torch.isfinite(g["g_w"]).all()
