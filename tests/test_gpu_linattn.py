"""Linear attention with a decay for each head on the GPU against the fp64
oracle, at the sizes, layouts and masks where it can go wrong.

Tolerances, elementwise, from the arithmetic.  Every output is a sum of
products; `mag` is the same sum with every term's magnitude (the oracle run on
absolute values).  A term passes through at most
  dk + dv + 64 + L additions, the exponentials (argument held to 2^-24, each
  e^-d wrong by (d + 2) 2^-24, worst against its own size where d is about 1)
  and one multiplication per chunk,
so fp32 work is off by at most (dk + dv + L + 128) 2^-24 mag.  bf16 outputs add
half a step of bf16 (2^-8 of the value) and two pieces of 8 bits for the state
and for the weighted scores (each within 2^-16 of a term: 2^-15 mag).  States
and gradients of bf16 inputs use three pieces, within 2^-23.  The log-decay
gradient is a difference of sums, so its `mag` is the sum of what they hold.
"""

import numpy as np
import pytest

from oracle.linattn_oracle import linattn_bwd, linattn_fwd, linattn_step
from tests._gpu import lib

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(B, H, Hk, L, dk, dv, dt, seed=0, const=False, decay=-3.0, state=True):
    """Tensors [B,H,L,d] on the device (head-major); decays around exp(-exp(decay))."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = dict(q=n(B, Hk, L, dk).to(dt), k=(n(B, Hk, L, dk) * dk ** -0.5).to(dt), v=n(B, H, L, dv).to(dt),
             g_o=n(B, H, L, dv).to(dt))
    x["log_decay"] = -torch.exp(n(H) + decay) if const else -torch.exp(1.5 * n(B, H, L) + decay)
    x["h0"] = n(B, H, dk, dv) if state else None
    x["g_hL"] = n(B, H, dk, dv) if state else None
    return {a: (b.cuda() if b is not None else None) for a, b in x.items()}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def decays(x):
    g = f64(x["log_decay"])
    if g.ndim == 1:
        B, H, L = x["v"].shape[:3]
        g = np.broadcast_to(g[None, :, None], (B, H, L))
    return g


def close(got, ref, bound, what):
    got = f64(got)
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    assert np.isfinite(got).all(), f"{what}: not finite"
    err = np.abs(got - ref)
    worst = float((err / np.maximum(bound, 1e-30)).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def bounds(x, ref, mag, dt_out, pieces=3):
    B, H, L, dv = x["v"].shape
    dk = x["q"].shape[-1]
    b = (dk + dv + L + 128) * 2.0 ** -24 * mag + 1e-30
    if x["v"].dtype == BF:
        b = b + (2.0 ** -15 if pieces == 2 else 2.0 ** -22) * mag
    if dt_out == BF:
        b = b + 2.0 ** -8 * np.abs(ref)
    return b


def absolute(x):
    a = {n: (None if t is None else np.abs(f64(t))) for n, t in x.items() if n != "log_decay"}
    return a, decays(x)


def check_fwd(x, o, hL, scale):
    g = decays(x)
    ro, rh, _ = linattn_fwd(f64(x["q"]), f64(x["k"]), f64(x["v"]), g, f64(x["h0"]), scale)
    a, g = absolute(x)
    mo, mh, _ = linattn_fwd(a["q"], a["k"], a["v"], g, a["h0"], abs(scale))
    close(o, ro, bounds(x, ro, mo, o.dtype, 2), "o")
    close(hL, rh, bounds(x, rh, mh, F32), "h_L")


def check_bwd(x, r, scale):
    g = decays(x)
    ref = linattn_bwd(f64(x["q"]), f64(x["k"]), f64(x["v"]), g, f64(x["g_o"]), f64(x["h0"]), f64(x["g_hL"]), scale)
    a, g = absolute(x)
    mag = linattn_bwd(a["q"], a["k"], a["v"], g, a["g_o"], a["h0"], a["g_hL"], abs(scale))
    for n in ("g_q", "g_k", "g_v"):
        close(r[n], ref[n], bounds(x, ref[n], mag[n], r[n].dtype), n)
    if "g_h0" in r:
        close(r["g_h0"], ref["g_h0"], bounds(x, ref["g_h0"], mag["g_h0"], F32), "g_h0")
    # what the sums of the log-decay gradient hold: every r_i and c_j from t on, and the pairs past the end
    H, Hk = a["v"].shape[1], a["q"].shape[1]
    held = log_decay_mag(a, g, scale)
    want, m = ref["g_g"], held
    if x["log_decay"].dim() == 1:
        want, m = want.sum((0, 2)), m.sum((0, 2))
    close(r["g_log_decay"], want, bounds(x, want, m, F32), "g_log_decay")


def log_decay_mag(a, g, scale):
    H, Hk = a["v"].shape[1], a["q"].shape[1]
    rep = lambda t: np.repeat(t, H // Hk, axis=1)  # noqa: E731
    m = linattn_bwd(rep(a["q"]), rep(a["k"]), a["v"], g, a["g_o"], a["h0"], a["g_hL"], abs(scale))
    r = (rep(a["q"]) * m["g_q"]).sum(-1) + (rep(a["k"]) * m["g_k"]).sum(-1)
    end = 0.0
    if a["g_hL"] is not None:
        hL = linattn_fwd(rep(a["q"]), rep(a["k"]), a["v"], g, a["h0"], abs(scale))[1]
        end = (hL * a["g_hL"]).sum((-1, -2))[..., None]
    return r[..., ::-1].cumsum(-1)[..., ::-1] + end + m["g_g"]


def fwd(x, scale=None, **kw):
    return lib().pdssm_linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], h0=x["h0"], scale=scale, **kw)


def bwd(x, scale=None, **kw):
    return lib().pdssm_linattn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["g_o"], h0=x["h0"], g_hL=x["g_hL"],
                                   scale=scale, **kw)


SHAPES = [
    # B, H, Hk, L, dk, dv, const, state
    (1, 1, 1, 1, 8, 8, False, True),
    (2, 3, 3, 63, 16, 64, True, False),
    (1, 2, 1, 64, 32, 32, False, True),
    (2, 2, 2, 65, 64, 32, False, False),
    (1, 4, 2, 130, 40, 72, False, True),
    (1, 3, 1, 100, 128, 128, True, True),
    (2, 2, 2, 97, 128, 64, False, True),
    (1, 2, 2, 70, 200, 24, False, True),
    (1, 2, 1, 129, 256, 256, False, True),
    (1, 2, 2, 33, 24, 136, True, True),
    (1, 1, 1, 700, 64, 64, False, True),      # few rows: the step axis is cut into segments
    (1, 2, 1, 1100, 96, 160, False, False),
    (1, 1, 1, 513, 16, 256, True, True),
    (1, 2, 1, 300, 256, 192, False, True),
    (1, 1, 1, 530, 192, 256, True, False),
    (2, 1, 1, 600, 128, 128, False, True),    # a gradient's segments are never over 512 steps
]


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
def test_fwd_against_oracle(shape, dt):
    B, H, Hk, L, dk, dv, const, state = shape
    x = make(B, H, Hk, L, dk, dv, dt, seed=L, const=const, state=state)
    print(f"[gpu] linattn fwd {shape} {dt}", flush=True)
    o, hL = fwd(x)
    check_fwd(x, o, hL, dk ** -0.5)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
def test_bwd_against_oracle(shape, dt):
    B, H, Hk, L, dk, dv, const, state = shape
    x = make(B, H, Hk, L, dk, dv, dt, seed=L, const=const, state=state)
    print(f"[gpu] linattn bwd {shape} {dt}", flush=True)
    check_bwd(x, bwd(x), dk ** -0.5)


STEPS = [(1, 1, 1, 8, 8, False), (3, 4, 2, 40, 72, True), (2, 2, 1, 128, 128, False), (33, 8, 8, 16, 64, True),
         (1, 2, 2, 256, 256, False), (5, 3, 3, 200, 24, False), (300, 16, 4, 32, 16, False)]


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", STEPS, ids=lambda s: "x".join(map(str, s[:5])))
def test_step_against_oracle(shape, dt):
    P = lib()
    B, H, Hk, dk, dv, const = shape
    x = make(B, H, Hk, 1, dk, dv, dt, const=const)
    slots = B + 4
    pool = torch.randn(slots, H, dk, dv, generator=torch.Generator().manual_seed(5))
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(6))[:B].to(torch.int32)
    dev, before = pool.cuda(), pool.numpy()
    la = x["log_decay"] if const else x["log_decay"][:, :, 0]
    print(f"[gpu] linattn step {shape} {dt}", flush=True)
    o = P.pdssm_linattn_step(x["q"][:, :, 0], x["k"][:, :, 0], x["v"][:, :, 0], la, dev, state_idx=idx.cuda(), scale=0.3)
    ro, rp = linattn_step(f64(x["q"])[:, :, 0], f64(x["k"])[:, :, 0], f64(x["v"])[:, :, 0], decays(x)[:, :, 0], before, idx, 0.3)
    a, g = absolute(x)
    mo, mp = linattn_step(a["q"][:, :, 0], a["k"][:, :, 0], a["v"][:, :, 0], g[:, :, 0], np.abs(before), idx, 0.3)
    bound = (dk + 16) * 2.0 ** -24 * mo + (2.0 ** -8 * np.abs(ro) if dt == BF else 0.0) + 1e-30
    close(o, ro, bound, "o")
    # a state element: one exponential (2 ulp), one product each side, one addition
    close(dev, rp, 6 * 2.0 ** -24 * mp, "state")
    untouched = sorted(set(range(slots)) - set(idx.tolist()))
    assert np.array_equal(dev.cpu().numpy()[untouched], before[untouched])


def test_step_empty_repeated_and_outside_slots():
    """Empty rows are zero, a slot past the pool or named twice gives NaN and is not touched (twice)."""
    P = lib()
    x = make(6, 2, 2, 1, 32, 32, BF)
    pool = torch.randn(4, 2, 32, 32)
    dev = pool.cuda()
    idx = torch.tensor([2, -1, 2, 4, 0, -7], dtype=torch.int32)
    o = P.pdssm_linattn_step(x["q"][:, :, 0], x["k"][:, :, 0], x["v"][:, :, 0], x["log_decay"][:, :, 0], dev, state_idx=idx.cuda())
    ro, rp = linattn_step(f64(x["q"])[:, :, 0], f64(x["k"])[:, :, 0], f64(x["v"])[:, :, 0], decays(x)[:, :, 0], pool.numpy(), idx, 32 ** -0.5)
    o = f64(o)
    assert np.isnan(o[[2, 3]]).all() and (o[[1, 5]] == 0).all()
    assert np.abs(o[[0, 4]] - ro[[0, 4]]).max() < 0.05
    got = f64(dev)
    assert np.array_equal(got[[1, 3]], pool.double().numpy()[[1, 3]])
    assert np.abs(got - rp).max() < 1e-5


def test_step_repeats_a_prompt():
    """Token by token on the pool gives what the prompt pass gives."""
    P = lib()
    x = make(2, 4, 2, 70, 64, 48, F32)
    o, hL = fwd(x, scale=0.2)
    pool = x["h0"].clone()
    for t in range(70):
        ot = P.pdssm_linattn_step(x["q"][:, :, t], x["k"][:, :, t], x["v"][:, :, t], x["log_decay"][:, :, t], pool, scale=0.2)
        assert (ot - o[:, :, t]).abs().max() <= 2e-5 * (1 + o[:, :, t].abs().max())
    assert (pool - hL).abs().max() <= 2e-5 * (1 + hL.abs().max())


def packed(lens, H, Hk, dk, dv, dt, tail=5, const=False, state=True, lead=0):
    total = sum(lens)
    x = make(1, H, Hk, lead + total + tail, dk, dv, dt, seed=total, const=const, state=False)
    if state:
        g = torch.Generator().manual_seed(9)
        x["h0"] = torch.randn(len(lens), H, dk, dv, generator=g).cuda()
        x["g_hL"] = torch.randn(len(lens), H, dk, dv, generator=g).cuda()
    cu = torch.tensor([lead] + [lead + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32).cuda()
    return x, cu


def part(x, cu, i):
    a, b = int(cu[i]), int(cu[i + 1])
    y = {n: (t if t is None or t.dim() < 3 or n in ("h0", "g_hL") else t[:, :, a:b]) for n, t in x.items()}
    for n in ("h0", "g_hL"):
        y[n] = None if x[n] is None else x[n][i:i + 1]
    return y, a, b


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("lens,H,Hk,dk,dv,const", [
    ([5, 0, 64, 1, 130, 0], 2, 1, 32, 64, False),
    ([700, 3, 290], 1, 1, 64, 128, True),       # segments: more than one in the long sequences
    ([0, 0], 2, 2, 16, 16, False),
    ([1], 3, 1, 128, 8, False),
])
def test_packed(lens, H, Hk, dk, dv, const, dt):
    """Each sequence as if alone; rows around them hold NaN, are not read and stay as they were."""
    x, cu = packed(lens, H, Hk, dk, dv, dt, tail=7, const=const, lead=3)
    lo, hi = int(cu[0]), int(cu[-1])
    for n in ("q", "k", "v", "g_o", "log_decay"):
        if x[n].dim() >= 3:
            x[n][:, :, :lo] = float("nan")
            x[n][:, :, hi:] = float("nan")
    o = torch.full_like(x["v"], 7.0)
    print(f"[gpu] linattn packed {lens} {dt}", flush=True)
    _, hL = fwd(x, scale=0.3, cu_seqlens=cu, out={"o": o})
    out = {n: torch.full_like(x[m], 7.0) for n, m in (("g_q", "q"), ("g_k", "k"), ("g_v", "v"))}
    if not const:
        out["g_log_decay"] = torch.full_like(x["log_decay"], 7.0)
    r = bwd(x, scale=0.3, cu_seqlens=cu, out=out)
    for t in (o, *out.values()):
        assert (t[:, :, :lo] == 7).all() and (t[:, :, hi:] == 7).all()
    total = np.zeros(H)
    held = np.zeros(H)
    for i in range(len(lens)):
        y, a, b = part(x, cu, i)
        if a == b:
            assert torch.equal(hL[i], x["h0"][i]) and torch.equal(r["g_h0"][i], x["g_hL"][i])
            continue
        check_fwd(y, o[:, :, a:b], hL[i:i + 1], 0.3)
        s = {n: r[n][:, :, a:b] for n in ("g_q", "g_k", "g_v")}
        s["g_h0"] = r["g_h0"][i:i + 1]
        if const:
            z = dict(y, log_decay=x["log_decay"])
            ref = linattn_bwd(f64(y["q"]), f64(y["k"]), f64(y["v"]), decays(z), f64(y["g_o"]), f64(y["h0"]), f64(y["g_hL"]), 0.3)
            ab, g = absolute(z)
            total += ref["g_g"].sum((0, 2))
            held += log_decay_mag(ab, g, 0.3).sum((0, 2))
            mag = linattn_bwd(ab["q"], ab["k"], ab["v"], g, ab["g_o"], ab["h0"], ab["g_hL"], 0.3)
            for n in ("g_q", "g_k", "g_v"):
                close(s[n], ref[n], bounds(y, ref[n], mag[n], s[n].dtype), n)
        else:
            s["g_log_decay"] = r["g_log_decay"][:, :, a:b]
            check_bwd(y, s, 0.3)
    if const:
        close(r["g_log_decay"], total, bounds(x, total, held, F32), "g_log_decay")


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_layouts_agree(dt):
    """Step-major tensors, slices of one projection, broadcast inputs: the same bits as contiguous ones."""
    B, H, L, d = 2, 3, 100, 32
    x = make(B, H, H, L, d, d, dt)
    base, hb = fwd(x)
    gb = bwd(x)
    wide = torch.empty(B, L, H, 3 * d + 16, dtype=dt, device="cuda")
    y = dict(x)
    for i, n in enumerate(("q", "k", "v")):
        wide[..., i * d:(i + 1) * d] = x[n].transpose(1, 2)
        y[n] = wide[..., i * d:(i + 1) * d].transpose(1, 2)
    y["g_o"] = x["g_o"].transpose(1, 2).contiguous().transpose(1, 2)
    y["log_decay"] = x["log_decay"].permute(2, 0, 1).contiguous().permute(1, 2, 0)
    o, h = fwd(y)
    g = bwd(y)
    assert o.stride(2) > o.stride(1) and g["g_q"].stride(2) > g["g_q"].stride(1)
    assert torch.equal(o, base) and torch.equal(h, hb)
    for n in gb:
        assert torch.equal(g[n], gb[n]), n
    # gradients into slices of one buffer
    buf = torch.zeros_like(wide)
    sl = {n: buf[..., i * d:(i + 1) * d].transpose(1, 2) for i, n in enumerate(("g_q", "g_k", "g_v"))}
    g2 = bwd(y, out=dict(sl))
    for n in ("g_q", "g_k", "g_v"):
        assert torch.equal(g2[n], gb[n]) and g2[n].data_ptr() == sl[n].data_ptr()
    assert (buf[..., 3 * d:] == 0).all()
    # one query for all heads and one decay for all steps, broadcast by strides
    z = dict(x, q=x["q"][:, :1].expand(B, H, L, d), log_decay=x["log_decay"][:, :, :1].expand(B, H, L))
    c = {n: (t.contiguous() if t is not None else None) for n, t in z.items()}
    assert torch.equal(fwd(z)[0], fwd(c)[0])
    gz, gc = bwd(z), bwd(c)
    for n in gc:
        assert torch.equal(gz[n], gc[n]), n


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("L,dk,dv", [(200, 32, 32), (140, 128, 128), (600, 64, 40), (100, 256, 64)])
def test_decays_at_their_ends(L, dk, dv, dt):
    """No decay, a decay that forgets at once, minus infinity (the state starts anew), strong decays
    before weak ones (differences of large sums), and a chunk at the border between both kinds of weights."""
    x = make(1, 5, 5, L, dk, dv, dt)
    g = x["log_decay"]
    g[:, 0] = 0.0
    g[:, 1] = -200.0
    g[:, 2, ::37] = float("-inf")
    g[:, 3, ::3] = -60.0
    g[:, 4] = -24.0 * np.log(2.0) / 32 * (1 + 0.001 * torch.randn(L, generator=torch.Generator().manual_seed(1)).cuda())
    print(f"[gpu] linattn decays {L} {dk} {dv} {dt}", flush=True)
    o, hL = fwd(x, scale=1.0)
    check_fwd(x, o, hL, 1.0)
    check_bwd(x, bwd(x, scale=1.0), 1.0)
    x["log_decay"] = torch.tensor([0.0, -1e-4, float("-inf"), -90.0, -0.52]).cuda()
    check_fwd(x, *fwd(x, scale=1.0), 1.0)
    check_bwd(x, bwd(x, scale=1.0), 1.0)


def test_sequences_of_one_step_have_no_decay_gradient():
    """Without a state before it a token's decay meets nothing: exactly zero."""
    x, cu = packed([1, 1, 1], 3, 1, 64, 96, BF, tail=0, state=False)
    assert (bwd(x, cu_seqlens=cu)["g_log_decay"] == 0).all()


def test_many_sequences_around_a_long_one():
    """More sequences than a round of the segment table, one of them cut into segments."""
    lens = [int(v) for v in np.random.default_rng(0).integers(0, 5, 150)] + [900] + [2] * 150 + [333]
    x, cu = packed(lens, 1, 1, 32, 32, BF, tail=3)
    o, hL = fwd(x, scale=0.4, cu_seqlens=cu)
    r = bwd(x, scale=0.4, cu_seqlens=cu)
    for i in (0, 1, 77, 149, 150, 151, 299, 300, 301):
        y, a, b = part(x, cu, i)
        if a == b:
            assert torch.equal(hL[i], x["h0"][i])
            continue
        check_fwd(y, o[:, :, a:b], hL[i:i + 1], 0.4)
        s = {n: r[n][:, :, a:b] for n in ("g_q", "g_k", "g_v", "g_log_decay")}
        check_bwd(y, dict(s, g_h0=r["g_h0"][i:i + 1]), 0.4)


@pytest.mark.parametrize("bad", [[0, 40, 30, 700, 1000], [-5, 100, 90, 2000, 1 << 30], [900, 800, 700, 0, 5],
                                 [0, 1000, 0, 1000, 0, 1000, 0, 1000, 0, 1000]])
def test_offsets_out_of_order_touch_nothing_outside(bad):
    """Offsets outside the rows or out of order are cut: rows of the buffers around the tensors stay, and a
    sequence whose own bounds are in order and apart from the others' is right."""
    L = 1000
    x = make(1, 2, 1, L, 32, 32, BF, state=False)
    cu = torch.tensor(bad, dtype=torch.int32).cuda()
    n = len(bad) - 1
    guard = {m: torch.full((1, 2 if m in ("o", "g_v") else 1, L + 2000, 32), 5.0, dtype=BF, device="cuda") for m in ("o", "g_q", "g_k", "g_v")}
    gl = torch.full((1, 2, L + 2000), 5.0, device="cuda")
    view = {m: t[:, :, 1000:1000 + L] for m, t in guard.items()}
    hs = torch.full((n + 2, 2, 32, 32), 5.0, device="cuda")
    print(f"[gpu] linattn offsets {bad}", flush=True)
    fwd(x, cu_seqlens=cu, out={"o": view["o"], "h_L": hs[1:-1]})
    bwd(x, cu_seqlens=cu, out={**{m: view[m] for m in ("g_q", "g_k", "g_v")}, "g_log_decay": gl[:, :, 1000:1000 + L]})
    torch.cuda.synchronize()
    for t in (*guard.values(), gl):
        assert (t[:, :, :1000] == 5).all() and (t[:, :, 1000 + L:] == 5).all()
    assert (hs[0] == 5).all() and (hs[-1] == 5).all()
    if bad[:2] == [0, 40]:
        y = {m: (t[:, :, :40] if t is not None else None) for m, t in x.items()}
        ro = linattn_fwd(f64(y["q"]), f64(y["k"]), f64(y["v"]), decays(y), None, 32 ** -0.5)[0]
        assert np.abs(f64(view["o"][:, :, :30]) - ro[:, :, :30]).max() < 0.05


def test_offsets_past_32_bits():
    """Batch strides over 2^31 elements and a pool of states over 2^32 bytes."""
    P = lib()
    B, H, L, d = 2, 1, 70, 32
    far = (1 << 31) + 64
    buf = torch.empty(far + 4 * L * d, dtype=BF, device="cuda")
    x = make(B, H, H, L, d, d, BF)
    y = dict(x)
    for i, n in enumerate(("q", "k", "v", "g_o")):
        y[n] = buf.as_strided((B, H, L, d), (far, L * d, d, 1), i * L * d)
        y[n].copy_(x[n])
    a, b = fwd(x), fwd(y)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = bwd(x), bwd(y)
    assert all(torch.equal(ga[n], gb[n]) for n in ga)
    del buf, y
    slots = (1 << 32) // (128 * 128 * 4) + 40
    pool = torch.zeros(slots, 1, 128, 128, device="cuda")
    t = make(2, 1, 1, 1, 128, 128, BF)
    idx = torch.tensor([slots - 1, 3], dtype=torch.int32).cuda()
    pool[idx.long()] = t["h0"]
    o = P.pdssm_linattn_step(t["q"][:, :, 0], t["k"][:, :, 0], t["v"][:, :, 0], t["log_decay"][:, :, 0], pool, state_idx=idx)
    small = t["h0"].clone()
    o2 = P.pdssm_linattn_step(t["q"][:, :, 0], t["k"][:, :, 0], t["v"][:, :, 0], t["log_decay"][:, :, 0], small)
    assert torch.equal(o, o2) and torch.equal(pool[idx.long()], small)
    assert int((pool != 0).any(-1).any(-1).sum()) == 2


def test_gradient_by_differences():
    """The gradient of a scalar loss along random directions against central differences of the GPU's own
    forward pass.  A step of 2^-5 leaves (2^-5)^2 / 6 of the third derivative; the loss is a polynomial of degree
    three in q, k, v and h0 together (four with two factors of k and v, smooth in the decays), so its error
    is under 2^-10 of the sums' size, and the fp32 losses add 2^-24 / 2^-5 of theirs."""
    x = make(1, 4, 2, 90, 32, 24, F32, decay=-2.0)
    r = bwd(x, scale=0.7)
    gen = torch.Generator().manual_seed(3)

    def loss(y):
        o, hL = fwd(y, scale=0.7)
        return float((o.double() * x["g_o"].double()).sum() + (hL.double() * x["g_hL"].double()).sum())

    for n in ("q", "k", "v", "log_decay", "h0"):
        d = torch.randn(x[n].shape, generator=gen).cuda()
        if n == "log_decay":
            d = d * x[n]          # in proportion: no decay becomes positive
        e = 2.0 ** -5
        num = (loss(dict(x, **{n: x[n] + e * d})) - loss(dict(x, **{n: x[n] - e * d}))) / (2 * e)
        got = float((r["g_" + n].double() * d.double()).sum())
        size = float((r["g_" + n].double() * d.double()).abs().sum())
        assert abs(num - got) <= 2.0 ** -10 * size, (n, num, got, size)


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own, running together."""
    a, b = make(1, 2, 1, 900, 64, 64, BF, seed=1), make(1, 2, 1, 900, 64, 64, BF, seed=2)
    want = [(fwd(x), bwd(x)) for x in (a, b)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(s[i]):
                got[i].append((fwd(x), bwd(x)))
    torch.cuda.synchronize()
    for i in range(2):
        for f, g in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(f, want[i][0])) and all(torch.equal(g[n], want[i][1][n]) for n in g)


def test_scale_zero_and_negative():
    x = make(1, 2, 2, 80, 32, 32, F32)
    for s in (0.0, -1.5):
        check_fwd(x, *fwd(x, scale=s), s)
        check_bwd(x, bwd(x, scale=s), s)


def test_runs_agree_bit_for_bit():
    x = make(1, 2, 1, 900, 64, 64, BF)
    a, b = fwd(x), fwd(x)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a, b = bwd(x), bwd(x)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_stream_workspace_and_header():
    """On a side stream, with caller workspaces left full of garbage, and the header's error word zero."""
    P = lib()
    x = make(1, 2, 2, 900, 64, 64, BF)
    o, hL = fwd(x)
    g = bwd(x)
    d = P.linattn_dims(1, 2, 900, 64, 64, bf16=True, scale=64 ** -0.5)
    ws = torch.full((P.linattn_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    wb = torch.full((P.linattn_bwd_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, h2 = fwd(x, workspace=ws)
        g2 = bwd(x, workspace=wb)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(hL, h2) and all(torch.equal(g[n], g2[n]) for n in g)
    assert P.workspace_error_flag(ws) == 0 and P.workspace_error_flag(wb) == 0


def test_two_graphs_replayed():
    """A prompt and its gradient captured with a workspace each, replayed on new inputs between eager calls."""
    P = lib()
    x = make(1, 2, 1, 700, 64, 64, BF, seed=1)
    y = make(1, 2, 1, 700, 64, 64, BF, seed=2)
    idx = torch.tensor([1, 0, -1], dtype=torch.int32).cuda()
    step = make(3, 2, 1, 1, 64, 64, BF, seed=3)
    pool0 = torch.randn(4, 2, 64, 64).cuda()
    pool = pool0.clone()

    def run_step(p):
        return P.pdssm_linattn_step(step["q"][:, :, 0], step["k"][:, :, 0], step["v"][:, :, 0], step["log_decay"][:, :, 0], p,
                                    state_idx=idx)

    fwd(x), bwd(x), run_step(pool.clone())
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        o, hL = fwd(x)
        so = run_step(pool)
    with torch.cuda.graph(gb):
        g = bwd(x)
    want_pool = pool0.clone()
    pool.copy_(pool0)
    for turn, src in enumerate((y, make(1, 2, 1, 700, 64, 64, BF, seed=4), y)):
        for n in x:
            x[n].copy_(src[n])
        ga.replay()
        gb.replay()
        torch.cuda.synchronize()
        eo, eh = fwd(src)
        eg = bwd(src)
        es = run_step(want_pool)
        torch.cuda.synchronize()
        assert torch.equal(o, eo) and torch.equal(hL, eh), turn
        assert all(torch.equal(g[n], eg[n]) for n in g), turn
        assert torch.equal(so, es) and torch.equal(pool, want_pool), turn


def test_captured_packed_call_follows_its_offsets():
    """The segment table is made on the device: a replay sees the offsets that are there then."""
    x, cu = packed([500, 300, 0, 203], 2, 1, 64, 32, BF, tail=0)
    fwd(x, cu_seqlens=cu), bwd(x, cu_seqlens=cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, hL = fwd(x, cu_seqlens=cu)
        g = bwd(x, cu_seqlens=cu)
    for lens in ([500, 300, 0, 203], [1, 0, 1001, 1], [0, 1003, 0, 0], [250, 251, 251, 251]):
        cu.copy_(torch.tensor([0] + lens).cumsum(0))
        graph.replay()
        torch.cuda.synchronize()
        eo, eh = fwd(x, cu_seqlens=cu)
        eg = bwd(x, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert torch.equal(o, eo) and torch.equal(hL, eh), lens
        assert all(torch.equal(g[n], eg[n]) for n in g), lens
        for i in range(4):
            y, a, b = part(x, cu, i)
            if a != b:
                check_fwd(y, eo[:, :, a:b], eh[i:i + 1], 64 ** -0.5)


def test_step_of_many_rows():
    """More rows than a round of the search for an earlier row of the slot, in any order, some of them empty or again."""
    P = lib()
    n, slots = 3001, 3500
    x = make(n, 1, 1, 1, 8, 8, BF)
    gen = torch.Generator().manual_seed(5)
    idx = torch.randperm(slots, generator=gen)[:n].to(torch.int32)
    idx[::97] = -1
    idx[2999] = idx[1500]
    idx[1700] = idx[5]
    pool = torch.randn(slots, 1, 8, 8, generator=gen).cuda()
    new = pool.clone()
    row = lambda t: t[:, :, 0]  # noqa: E731
    o = P.pdssm_linattn_step(row(x["q"]), row(x["k"]), row(x["v"]), row(x["log_decay"]), new, state_idx=idx.cuda())
    ok = idx >= 0
    ok[2999] = ok[1700] = False
    at = idx[ok].long().cuda()
    use = ok.cuda()
    own = pool[at].clone()
    want = P.pdssm_linattn_step(*(row(x[m])[use].contiguous() for m in ("q", "k", "v", "log_decay")), own)
    assert torch.equal(o[use], want) and torch.equal(new[at], own)
    assert (o[(idx < 0).cuda()] == 0).all() and torch.isnan(o[[1700, 2999]].float()).all()
    rest = torch.ones(slots, dtype=torch.bool)
    rest[at.cpu()] = False
    assert torch.equal(new[rest.cuda()], pool[rest.cuda()])


def test_prompt_then_tokens_then_gradient():
    """As they are used together: packed prompts fill a pool, tokens follow, and the gradient of the whole
    prompt equals the one of its two halves joined at the state."""
    P = lib()
    lens = [70, 9, 300]
    x, cu = packed(lens, 4, 2, 64, 32, F32, tail=0, const=False, state=False)
    o, hL = fwd(x, scale=0.5, cu_seqlens=cu)
    pool = torch.randn(5, 4, 64, 32).cuda()
    idx = torch.tensor([3, 0, 2], dtype=torch.int32).cuda()
    pool[idx.long()] = hL
    t = make(3, 4, 2, 1, 64, 32, F32, seed=8)
    ot = P.pdssm_linattn_step(t["q"][:, :, 0], t["k"][:, :, 0], t["v"][:, :, 0], t["log_decay"][:, :, 0], pool, state_idx=idx, scale=0.5)
    for i, n in enumerate(lens):
        y, a, b = part(x, cu, i)
        full = {m: torch.cat([y[m], t[m][i:i + 1]], 2) for m in ("q", "k", "v", "log_decay")}
        full.update(h0=None)
        fo, fh = fwd(full, scale=0.5)
        assert (fo[0, :, -1] - ot[i]).abs().max() <= 3e-5 * (1 + ot[i].abs().max())
        assert (fh[0] - pool[idx[i]]).abs().max() <= 3e-5 * (1 + fh.abs().max())
    y, a, b = part(x, cu, 2)
    y["h0"] = y["g_hL"] = None
    whole = bwd(y, scale=0.5)
    cut = lambda s: {n: (v if v is None else v[:, :, s]) for n, v in y.items()}  # noqa: E731
    first, second = cut(slice(0, 130)), cut(slice(130, 300))
    _, mid = fwd(first, scale=0.5)
    second["h0"] = mid
    g2 = bwd(second, scale=0.5)
    first["g_hL"] = g2["g_h0"]
    g1 = bwd(first, scale=0.5)
    for n in ("g_q", "g_k", "g_v", "g_log_decay"):
        joined = torch.cat([g1[n], g2[n]], 2)
        assert (joined - whole[n]).abs().max() <= 3e-5 * (1 + whole[n].abs().max()), n


def test_refusals_on_the_device():
    P = lib()
    x = make(2, 2, 2, 70, 32, 32, BF)
    with pytest.raises(P.PdssmError, match="overlaps"):
        fwd(x, out={"o": x["v"]})
    with pytest.raises(P.PdssmError, match="rows of output"):
        fwd(x, out={"o": torch.empty(2, 1, 70, 32, dtype=BF, device="cuda").expand(2, 2, 70, 32)})
    with pytest.raises(P.PdssmError, match="16-byte"):
        off = torch.empty(2 * 2 * 70 * 32 + 4, dtype=BF, device="cuda")[4:].view(2, 2, 70, 32)
        fwd(dict(x, q=off))
    with pytest.raises(P.PdssmError, match="16 bytes"):
        fwd(dict(x, k=torch.empty(2, 2, 70, 36, dtype=BF, device="cuda")[..., :32]))
    with pytest.raises(ValueError, match="workspace holds"):
        fwd(x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        fwd(dict(x, q=torch.empty(2, 2, 32, 70, dtype=BF, device="cuda").transpose(2, 3)))
    with pytest.raises(ValueError, match="device tensor"):
        P.pdssm_linattn_step(x["q"][:, :, 0], x["k"][:, :, 0], x["v"][:, :, 0], x["log_decay"][:, :, 0].cpu(), x["h0"].clone())
