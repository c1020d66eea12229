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
