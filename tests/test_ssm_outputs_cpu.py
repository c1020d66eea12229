"""Outputs that a call of the selective layer does not make, no GPU: named in
out= they would be left as they are, so they are refused."""

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def P():
    from tests._libutil import ensure_built
    ensure_built()
    import structured_sparse_state_pdssm_amd as P
    return P


def z(*s):
    return torch.zeros(s)


B, L, D, N, W = 2, 10, 32, 16, 4


def test_outputs_that_are_not_made(P):
    conv = dict(x=z(B, L, D), w=z(D, W), g_y=z(B, L, D))
    scan = dict(x=z(B, L, D), dt=z(B, L, D), A=z(D, N), Bm=z(B, 1, L, N), Cm=z(B, 1, L, N), g_y=z(B, L, D))
    norm = dict(x=z(B, 3, L, D), w=z(3, D), g_y=z(B, 3, L, D))
    state, row, rows = z(B, W - 1, D), z(B, L, D), z(B, 3, L, D)
    for fn, args, more, name, out in (
            (P.pdssm_conv_bwd, conv, dict(want_x0=False), "g_x0", state),
            (P.pdssm_selscan_bwd, scan, dict(want_h0=False), "g_h0", z(B, D, N)),
            (P.pdssm_selscan_bwd, scan, {}, "g_z", row),
            (P.pdssm_norm_bwd, norm, {}, "g_z", rows),
            (P.pdssm_norm_bwd, norm, dict(z=rows, gate="after"), "g_res_scale", z(3, D))):
        with pytest.raises(ValueError, match=f"out has no '{name}'"):
            fn(**args, **more, out={name: out})


def test_outputs_that_are_made(P):
    """The same names where the call makes them: it comes to the device check."""
    conv = dict(x=z(B, L, D), w=z(D, W), g_y=z(B, L, D))
    scan = dict(x=z(B, L, D), dt=z(B, L, D), A=z(D, N), Bm=z(B, 1, L, N), Cm=z(B, 1, L, N), g_y=z(B, L, D), z=z(B, L, D))
    norm = dict(x=z(B, 3, L, D), w=z(3, D), g_y=z(B, 3, L, D), z=z(B, 3, L, D), gate="before", res_scale=z(3, D))
    for fn, args, out in ((P.pdssm_conv_bwd, conv, {"g_x0": z(B, W - 1, D)}),
                          (P.pdssm_selscan_bwd, scan, {"g_z": z(B, L, D), "g_h0": z(B, D, N)}),
                          (P.pdssm_norm_bwd, norm, {"g_z": z(B, 3, L, D), "g_res_scale": z(3, D)})):
        with pytest.raises(ValueError, match="device tensor"):
            fn(**args, out=out)
