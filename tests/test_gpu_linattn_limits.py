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
