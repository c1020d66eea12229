"""Linear attention on the GPU at the ends of its arguments' ranges: grids of
more than 2^32 threads, decays that leave nothing, long memories."""

import pytest

from tests._gpu import lib

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def normals(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return lambda *s, dt=F32, size=1.0: torch.randn(s, generator=g, device="cuda").mul_(size).to(dt)


def test_step_of_more_rows_than_a_launch_has_along_an_axis():
    """2^24 + 3 workgroups of 256 threads: the same bits as two calls on the halves of the rows."""
    P = lib()
    B, n = (1 << 24) + 3, normals(1)
    q, k, v = n(B, 1, 8, dt=BF), n(B, 1, 8, dt=BF), n(B, 1, 8, dt=BF)
    la = n(1).abs_().neg_()
    pool = n(B, 1, 8, 8)
    want = pool.clone()
    print(f"[gpu] linattn step of {B} rows", flush=True)
    o = P.pdssm_linattn_step(q, k, v, la, pool)
    for s in (slice(0, B // 2), slice(B // 2, B)):
        part = P.pdssm_linattn_step(q[s], k[s], v[s], la, want[s])
        assert torch.equal(o[s], part)
    assert torch.equal(pool, want)


@pytest.mark.parametrize("const", [False, True], ids=["tokens", "heads"])
def test_gradient_of_more_sequences_than_a_launch_has_along_an_axis(const):
    """2^23 sequences and heads and some more, 512 threads each for the log-decay gradient: as two calls on halves."""
    P = lib()
    B, H, n = 262149, 32, normals(2)
    x = dict(q=n(B, H, 1, 8, dt=BF), k=n(B, H, 1, 8, dt=BF), v=n(B, H, 1, 8, dt=BF), g_o=n(B, H, 1, 8, dt=BF),
             h0=n(B, H, 8, 8), log_decay=n(H).abs_().neg_() if const else n(B, H, 1).abs_().neg_())
    print(f"[gpu] linattn gradient of {B} x {H} tokens", flush=True)
    r = P.pdssm_linattn_bwd(**x, scale=0.5)
    total, held = torch.zeros(2, H, dtype=torch.float64, device="cuda")
    for s in (slice(0, B // 2), slice(B // 2, B)):
        part = P.pdssm_linattn_bwd(**{m: t if const and m == "log_decay" else t[s] for m, t in x.items()}, scale=0.5)
        for m in ("g_q", "g_k", "g_v", "g_h0"):
            assert torch.equal(r[m][s], part[m]), m
        if const:
            total += part["g_log_decay"].double()
            held += part["g_log_decay"].double().abs()
        else:
            assert torch.equal(r["g_log_decay"][s], part["g_log_decay"])
    if const:
        # the same terms in 64 bits (2^23 additions lose under 2^-29 of a typical sum), each of the three sums rounded once
        whole = r["g_log_decay"].double()
        assert ((whole - total).abs() <= 2.0 ** -23 * (whole.abs() + held)).all()


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("L,dk,dv", [(200, 32, 32), (1100, 128, 128)])
def test_decays_of_zero_have_no_gradient(L, dk, dv, dt):
    """exp(log_decay) is zero: so is its gradient, and not the rounding of the sums that it is a difference of; the
    steps around it keep theirs."""
    P = lib()
    H, n = 3, normals(3)
    x = dict(q=n(1, H, L, dk, dt=dt), k=n(1, H, L, dk, dt=dt), v=n(1, H, L, dv, dt=dt), g_o=n(1, H, L, dv, dt=dt),
             h0=n(1, H, dk, dv), g_hL=n(1, H, dk, dv), log_decay=n(1, H, L).sub_(3.0).exp_().neg_())
    at = torch.zeros(1, H, L, dtype=torch.bool, device="cuda")
    at[:, 0, ::37] = at[:, 1, 5::64] = at[:, 2, L - 1] = at[:, 2, 0] = True
    x["log_decay"][at] = torch.tensor([float("-inf"), -104.5, torch.finfo(F32).min, -1e4] * L, device="cuda")[:int(at.sum())]
    g = P.pdssm_linattn_bwd(**x)["g_log_decay"]
    assert (g[at] == 0).all() and (g[~at] != 0).float().mean() > 0.99
    x["log_decay"] = torch.tensor([float("-inf"), -0.01, -1e30], device="cuda")
    g = P.pdssm_linattn_bwd(**x)["g_log_decay"]
    assert g[0] == 0 and g[2] == 0 and g[1] != 0


def test_first_tokens_without_a_state_have_no_decay_gradient():
    """The state before the first token of every sequence is zero, batched and packed, in one segment and in several."""
    P = lib()
    H, L, n = 2, 1300, normals(4)
    x = dict(q=n(1, H, L, 64, dt=BF), k=n(1, H, L, 64, dt=BF), v=n(1, H, L, 32, dt=BF), g_o=n(1, H, L, 32, dt=BF),
             log_decay=n(1, H, L).sub_(3.0).exp_().neg_())
    g = P.pdssm_linattn_bwd(**x, g_hL=n(1, H, 64, 32))["g_log_decay"]
    assert (g[:, :, 0] == 0).all() and (g[:, :, 1:] != 0).float().mean() > 0.99
    cu = torch.tensor([0, 7, 7, 700, 1300], dtype=torch.int32, device="cuda")
    first = [0, 7, 700]
    r = P.pdssm_linattn_bwd(**x, g_hL=n(4, H, 64, 32), cu_seqlens=cu)["g_log_decay"]
    assert (r[:, :, first] == 0).all()
    r = P.pdssm_linattn_bwd(**x, h0=n(4, H, 64, 32), cu_seqlens=cu)["g_log_decay"]
    assert (r[:, :, first] != 0).any()


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("decay", [-3.0, -0.5, 1.0, 2.3])
@pytest.mark.parametrize("L,dk,dv", [(150, 64, 32), (1100, 32, 128)])
def test_log_decay_gradient_is_as_good_as_its_sums(L, dk, dv, decay, dt):
    """The bound of the sums that g_log_decay is a difference of: r_i = q_i . dq_i and c_j = k_j . dk_j without the
    token's own pair, over the rest of a segment (at most 512 steps), and what meets behind its end.  Each is an fp32
    sum of products of magnitude `mag`, through at most n = dk + dv + 512 + 128 roundings of up to 2^-24 of it, of
    either sign: their sum is within 4 sqrt(n) 2^-24 mag (seven times its root mean square), and those of the terms
    add in squares.  Where the decays are strong (e^-10) the own pair is 10^4 times the rest, so a gradient
    that held its rounding would be out of the bound."""
    import numpy as np

    from oracle.linattn_oracle import linattn_bwd
    from tests.test_gpu_linattn import bwd, decays, f64, make
    H, scale = 3, 0.3
    x = make(1, H, H, L, dk, dv, dt, seed=L + dk)
    x["log_decay"] = -torch.exp(0.3 * x["log_decay"].neg().log() + decay + 0.9)
    g = decays(x)
    a = {n: np.abs(f64(t)) for n, t in x.items()}
    ref = linattn_bwd(f64(x["q"]), f64(x["k"]), f64(x["v"]), g, f64(x["g_o"]), f64(x["h0"]), f64(x["g_hL"]), scale)["g_g"]
    m = linattn_bwd(a["q"], a["k"], a["v"], g, a["g_o"], a["h0"], a["g_hL"], scale)
    own = scale * (a["q"] * a["k"]).sum(-1) * (a["v"] * a["g_o"]).sum(-1)
    # (the magnitudes of q's and of k's terms)
    held = (a["q"] * m["g_q"]).sum(-1) - own + (a["k"] * m["g_k"]).sum(-1) - own
    rest = np.stack([(held[..., t:t + 512] ** 2).sum(-1) for t in range(L)], -1)
    # <S, dS> at a segment's end lies in the rest, or is the state's at the sequence's
    ends = [(s * d).sum((-1, -2)) for s, d in zip(*state_pairs(a, g, scale))]
    end = np.stack([np.max(ends[t:t + 512], axis=0) for t in range(L)], -1)
    bound = 4 * (dk + dv + 640) ** 0.5 * 2.0 ** -24 * np.sqrt(rest + end ** 2) + 2.0 ** -24 * np.abs(ref)
    got = f64(bwd(x, scale=scale)["g_log_decay"])
    worst = float((np.abs(got - ref) / bound).max())
    print(f"[gpu] linattn log-decay gradient {L} {dk} {dv} {decay} {dt}: {worst:.2g} of the bound", flush=True)
    assert worst <= 1.0, worst


def state_pairs(a, g, scale):
    """States behind every step and their adjoints just behind them, of the inputs' magnitudes."""
    import numpy as np

    from oracle.linattn_oracle import linattn_fwd
    S = linattn_fwd(a["q"], a["k"], a["v"], g, a["h0"], scale)[2][1:]
    D, out = a["g_hL"], []
    for t in reversed(range(g.shape[-1])):
        out.append(D)     # dLoss / d(the state behind step t), of the steps behind t
        D = np.exp(g[:, :, t, None, None]) * (D + scale * a["q"][:, :, t, :, None] * a["g_o"][:, :, t, None, :])
    return S, out[::-1]


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (BF, 256), (F32, 128)])
def test_long_memories_round_to_both_sides(dt, d):
    """8192 same-signed steps without decay, in one segment: the additions to the state are all the error there is.
    At most 24 roundings for 32 tokens, so n = 6144, each uniform within 2^-24 of the state at that time, which
    grows in proportion: the root mean square of their sum is sqrt(n / 9) 2^-24 of the state (a third for the
    uniform error, a third for the growth).  Six times of it is allowed, and a d-th of that for the mean over
    d^2 elements.  Half a step lost to one side at each would be n / 4 2^-24."""
    P = lib()
    B, H, L, n = 32, 16 if d < 256 else 8, 8192, normals(5)
    k, v = (n(B, H, L, d).abs_().mul_(d ** -0.25).to(dt) for _ in range(2))
    print(f"[gpu] linattn long memory {d} {dt}", flush=True)
    _, hL = P.pdssm_linattn_fwd(k, k, v, torch.zeros(H, device="cuda"))
    rms = 6144 ** 0.5 / 3 * 2.0 ** -24
    for b, h in ((0, 0), (B - 1, H - 1)):
        want = k[b, h].double().t().contiguous() @ v[b, h].double()
        err = (hL[b, h].double() - want) / want
        assert err.abs().max() <= 6 * rms, float(err.abs().max())
        assert err.mean().abs() <= 6 * rms / d, float(err.mean())


@pytest.mark.parametrize("rate", [2.0 ** -9, 2.0 ** -13])
@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (BF, 256), (F32, 128)])
def test_long_memories_with_a_decay(dt, d, rate):
    """A constant decay over far more steps than it remembers: the error is that of the memory, not of the length.
    A chunk of 32 tokens multiplies the state with a decay that is off by up to 2^-23 (its rounding and the
    exponential's), the same in every chunk: 1 / (32 rate) of them.  The additions, 24 roundings a chunk, of
    either sign, are allowed six times sqrt(24 / (64 rate)) 2^-24 (their squares decay twice as fast)."""
    P = lib()
    B, H, L, n = 8, 16, 16384, normals(6)
    k, v = (n(B, H, L, d).abs_().mul_(d ** -0.25).to(dt) for _ in range(2))
    la = torch.full((H,), rate, dtype=torch.float64, device="cuda").neg_().log1p_().float()
    print(f"[gpu] linattn long memory {d} {dt} {rate}", flush=True)
    _, hL = P.pdssm_linattn_fwd(k, k, v, la)
    r = P.pdssm_linattn_bwd(k, k, v, la, v, scale=1.0)["g_h0"]
    bound = 2.0 ** -23 / (32 * rate) + 6 * (24 / (64 * rate)) ** 0.5 * 2.0 ** -24 + 2.0 ** -22
    steps = torch.arange(L, dtype=torch.float64, device="cuda")
    for b, h in ((0, 0), (B - 1, H - 1)):
        behind, before = (((L - 1 - steps) * la[h].double()).exp(), ((steps + 1) * la[h].double()).exp())
        for got, w in ((hL[b, h], behind), (r[b, h], before)):
            want = (k[b, h].double() * w[:, None]).t().contiguous() @ v[b, h].double()
            err = ((got.double() - want) / want).abs().max()
            assert err <= bound, (float(err), bound)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 24), (24, 128), (256, 40), (200, 256)])
def test_segments_of_every_width(dk, dv, dt):
    """Wide and narrow rows over more than one segment, forwards and backwards."""
    from tests.test_gpu_linattn import bwd, check_bwd, check_fwd, fwd, make
    x = make(1, 2, 1, 777, dk, dv, dt, seed=dk)
    print(f"[gpu] linattn segments {dk} {dv} {dt}", flush=True)
    check_fwd(x, *fwd(x, scale=0.2), 0.2)
    check_bwd(x, bwd(x, scale=0.2), 0.2)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_log_decay_gradient_meets_the_state_at_the_start(dt):
    """The first token's is the product of h0 with its gradient, not what 500 steps' sums leave of it: p products in
    fp32, four and four added in fp32 (three roundings of 2^-24 each, of either sign, so within 6 sqrt(3) 2^-24 of
    the root of their squares' sum), rounded once."""
    P = lib()
    B, H, L, d, n = 4, 16, 500, 64, normals(7)
    x = dict(q=n(B, H, L, d, dt=dt), k=n(B, H, L, d, dt=dt), v=n(B, H, L, d, dt=dt), g_o=n(B, H, L, d, dt=dt),
             h0=n(B, H, d, d), g_hL=n(B, H, d, d), log_decay=n(B, H, L).sub_(6.0).exp_().neg_())
    r = P.pdssm_linattn_bwd(**x, scale=1.0)
    p = x["h0"].double() * r["g_h0"].double()
    want = p.sum((-1, -2))
    bound = 6 * 3 ** 0.5 * 2.0 ** -24 * (p ** 2).sum((-1, -2)).sqrt() + 2.0 ** -24 * want.abs()
    worst = float(((r["g_log_decay"][:, :, 0].double() - want).abs() / bound).max())
    print(f"[gpu] linattn first token's decay gradient {dt}: {worst:.2g} of the bound", flush=True)
    assert worst <= 1.0
