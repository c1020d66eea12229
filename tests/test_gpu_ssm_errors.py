"""How exact the selective layer's fp32 results are as a whole, and its sums
over more segments than one launch takes.

The elementwise bounds of the other tests add up every rounding's worst case,
hundreds of times what roundings do together.  Here the measure is the same formula,
step by step in numpy's fp32, on the same inputs, with functions that round once.
Roundings that do not know of each other add up in squares, so half as much again as
its error is more than twice its roundings (9/4).  A step from state to state has, in
squares of half a step of fp32, x^2 + 4 there (of the exponent x its product, then the
exponential, the decay's product, the drive and the addition) and 2 x^2 + 7 here at
most (A log2 e too, and v_exp_f32's two half steps): 9/5 where it counts, |x| up to
one.  Outputs of 1000 values and more, where the error of a whole is no matter of luck.
"""

import numpy as np
import pytest

from oracle import ssm_oracle as O
from tests._gpu import lib
from tests.test_gpu_ssm import BF, DT, F32, bounds, check, check_scan_bwd, close, conv_inputs, conv_ref, f64, norm_inputs, scan_args, scan_inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = O.U


def f32(t):
    return None if t is None else t.detach().cpu().numpy()


def once(f):
    """f in 64 bits, rounded to the type of its argument."""
    return lambda x: f(x.astype(np.float64)).astype(x.dtype)


@pytest.fixture
def functions_that_round_once(monkeypatch):
    monkeypatch.setattr(O, "decay", lambda d, A: once(np.exp)(d * A))
    monkeypatch.setattr(O, "_sig", once(O._sig))
    monkeypatch.setattr(O, "softplus", once(lambda x: np.logaddexp(0.0, x)))
    monkeypatch.setattr(O, "sigmoid", once(O._sig))


def as_exact(got, plain, ref):
    for n, t in got.items():
        if t.numel() < 1000:
            continue
        assert plain[n].dtype == np.float32, n
        size = np.linalg.norm(ref[n])
        here, there = (np.linalg.norm(x.astype(np.float64) - ref[n]) / size for x in (f64(t), plain[n]))
        assert here <= 1.5 * there, f"{n}: off by {here:.3g}, step by step in fp32 by {there:.3g}"


@pytest.mark.parametrize("B,L,D,N,G", [(1, 77, 768, 16, 1), (2, 200, 192, 16, 2), (1, 411, 128, 24, 4), (1, 700, 64, 64, 1), (3, 65, 256, 32, 1),
                                       (1, 1500, 40, 16, 1)])
def test_scan(B, L, D, N, G, functions_that_round_once):
    P = lib()
    x, gy, gh = scan_inputs(B, L, D, N, F32, G, seed=21)
    y, hL = P.pdssm_selscan_fwd(**x)
    got = dict(P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh), y=y, h_L=hL)
    sides = []
    for f in (f32, f64):
        a = {k: f(t) for k, t in x.items()}
        ry, rh, _ = O.selscan_fwd(**a)
        sides.append(dict(O.selscan_bwd(**a, g_y=f(gy), g_hL=f(gh)), y=ry, h_L=rh))
    as_exact(got, *sides)


def test_convolution(functions_that_round_once):
    P = lib()
    x, gy, gx = conv_inputs(2, 300, 256, 4, F32, seed=22)
    got = dict(P.pdssm_conv_bwd(**x, g_y=gy, g_xL=gx), y=P.pdssm_conv_fwd(**x)[0])
    sides = []
    for f in (f32, f64):
        a = {k: f(t) for k, t in x.items()}
        sides.append(dict(O.conv_bwd(**a, g_y=f(gy), g_xL=f(gx)), y=O.conv_fwd(**a)[0]))
    as_exact(got, *sides)


@pytest.mark.parametrize("gate", [None, "before", "after"])
@pytest.mark.parametrize("H,d", [(24, 64), (1, 2056)])
def test_norm(H, d, gate, functions_that_round_once):
    P = lib()
    x, res, gy = norm_inputs((2, H, 40, d), F32, gate, True, True, seed=23)
    got = dict(P.pdssm_norm_bwd(**x, g_y=gy, gate=gate), y=P.pdssm_norm_fwd(**x, gate=gate, residual=res))
    sides = []
    for f in (f32, f64):
        a, eps = {k: f(t) for k, t in x.items()}, float(np.float32(1e-5))
        sides.append(dict(O.norm_bwd(**a, g_y=f(gy), gate=gate, eps=eps), y=O.norm_fwd(**a, gate=gate, residual=f(res), eps=eps)))
    as_exact(got, *sides)


@DT
def test_sums_over_more_sequences_than_one_launch_takes(dt):
    """The gradients of A, D and dt_bias are sums over the sequences: over 256 of them in two rounds."""
    P = lib()
    x, gy, gh = scan_inputs(300, 3, 8, 8, dt, seed=24)
    check_scan_bwd(x, P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh), gy, gh)
    x, gy, gh = scan_inputs(259, 5, 40, 24, dt, seed=25)
    n = P.selscan_bwd_workspace_bytes(259, 5, 40, 24, 1, dt == BF)
    whole = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    check_scan_bwd(x, P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, workspace=whole[:n]), gy, gh)
    assert (whole[n:] == 0x5a).all()


@DT
def test_sums_over_more_packed_sequences_than_one_launch_takes(dt):
    P = lib()
    r = np.random.default_rng(5)
    lens = [int(n) for n in r.integers(0, 4, 330)] + [0, 70, 0]
    S, L = len(lens), sum(lens)
    assert 0 in lens[:330]
    x, gy, gh = scan_inputs(1, L, 16, 16, dt, S=S, seed=26)
    n = P.selscan_bwd_workspace_bytes(S, L, 16, 16, 1, dt == BF, True)
    whole = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    g = P.pdssm_selscan_bwd(**x, g_y=gy, g_hL=gh, cu_seqlens=bounds(lens), workspace=whole[:n])
    assert (whole[n:] == 0x5a).all()
    sums = {}
    for i, m in enumerate(lens):
        at = slice(sum(lens[:i]), sum(lens[:i]) + m)
        if not m:
            assert torch.equal(g["g_h0"][i], gh[i])
            continue
        xi = dict(x, h0=x["h0"][i:i + 1], **{k: x[k][:, at] for k in ("x", "dt", "z")}, **{k: x[k][:, :, at] for k in ("Bm", "Cm")})
        ref = O.selscan_bwd(**scan_args(xi), g_y=O.Bound(f64(gy[:, at])), g_hL=O.Bound(f64(gh[i:i + 1])))
        for k in ("g_x", "g_dt", "g_z"):
            close(g[k][:, at], ref[k], f"{k} of {i}")
        close(g["g_h0"][i:i + 1], ref["g_h0"], f"g_h0 of {i}")
        for k in ("g_A", "g_D", "g_dt_bias"):
            sums[k] = ref[k] if k not in sums else sums[k] + ref[k]
    check({k: g[k] for k in sums}, sums)


@DT
def test_sums_over_more_runs_than_one_launch_takes(dt):
    """One long sequence of few channels, cut into more than 256 runs: the sums against those of 16 calls on its parts,
    with the states and their gradients passed on.  A rounding is U of the sum that it is made in, and sums of terms of
    either sign are about the root of their number; a term meets a run's quarter (32 roundings), 12 at the runs' ends and
    about as many in the terms themselves: 100 of both sides, of sums up to the root of L or what the parts have."""
    P = lib()
    L = 65536
    x, gy, _ = scan_inputs(1, L, 8, 8, dt, seed=27, state=False)
    x["A"] = x["A"] - 1.0
    names = ("g_A", "g_D", "g_dt_bias")
    whole = P.pdssm_selscan_bwd(**x, g_y=gy)
    cut = lambda s: dict({k: (t[:, s] if k in ("x", "dt", "z") else t[:, :, s] if k in ("Bm", "Cm") else t) for k, t in x.items()})  # noqa: E731
    n = 4096
    parts = [cut(slice(i, i + n)) for i in range(0, L, n)]
    h, states = None, []
    for p in parts:
        states.append(h)
        _, h = P.pdssm_selscan_fwd(**p, h0=h)
    total, size, back = {}, {}, None
    for i in reversed(range(len(parts))):
        g = P.pdssm_selscan_bwd(**parts[i], g_y=gy[:, i * n:(i + 1) * n], h0=states[i], g_hL=back)
        back = g["g_h0"]
        for k in names:
            total[k] = total.get(k, 0) + f64(g[k])
            size[k] = size.get(k, 0) + np.abs(f64(g[k]))
    for k in names:
        assert np.isfinite(f64(whole[k])).all()
        assert np.abs(f64(whole[k]) - total[k]).max() <= 100 * U * max(size[k].max(), np.sqrt(L)), k
