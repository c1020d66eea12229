"""Arguments of the linear-attention calls that the binding refuses on the host, no GPU."""

from types import MappingProxyType

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def P():
    from tests._libutil import ensure_built
    ensure_built()
    import structured_sparse_state_pdssm_amd as P
    return P


B, H, L, dk, dv = 2, 2, 10, 32, 16


def args(**kw):
    z = torch.zeros
    return dict(dict(q=z(B, H, L, dk), k=z(B, H, L, dk), v=z(B, H, L, dv), log_decay=z(B, H, L)), **kw)


def test_unknown_outputs(P):
    """A misspelt name in out= would leave the tensor as it was."""
    g_o = torch.zeros(B, H, L, dv)
    with pytest.raises(ValueError, match="'hL'.*h_L"):
        P.pdssm_linattn_fwd(**args(), out={"hL": torch.zeros(B, H, dk, dv)})
    with pytest.raises(ValueError, match="'g_decay'.*g_log_decay"):
        P.pdssm_linattn_bwd(**args(g_o=g_o), out={"g_q": torch.zeros(B, H, L, dk), "g_decay": torch.zeros(B, H, L)})
    with pytest.raises(TypeError, match="out must be a dict"):
        P.pdssm_linattn_fwd(**args(), out=torch.zeros(B, H, L, dv))
    for out in ({}, None, {"o": torch.zeros(B, H, L, dv)}, {"o": None}, MappingProxyType({"o": None})):
        with pytest.raises(ValueError, match="device tensor"):
            P.pdssm_linattn_fwd(**args(), out=out)
    with pytest.raises(ValueError, match="device tensor"):   # left alone, as asked for
        P.pdssm_linattn_bwd(**args(g_o=g_o), want_h0=False, out={"g_h0": None})


def test_required_tensors(P):
    """None where a tensor is required is named, whatever the argument."""
    for n in ("q", "k", "v", "log_decay"):
        with pytest.raises(TypeError, match=f"{n} must be a torch.Tensor"):
            P.pdssm_linattn_fwd(**args(**{n: None}))
    with pytest.raises(TypeError, match="g_o must be a torch.Tensor"):
        P.pdssm_linattn_bwd(**args(), g_o=None)


def test_sizes_and_scales_past_32_bits():
    """What pdssm_linattn_dims cannot hold is a ValueError that shows it."""
    from tests._libutil import ensure_built
    ensure_built()
    from structured_sparse_state_pdssm_amd import _linattn as A
    assert len(A._pack_dims(1, 2, 1, (1 << 31) - 1, 8, 8, 1, True, False, 0.5)) == 40
    # (a number past fp32 packs as infinity, which the C ABI refuses)
    for f in ((1, 2, 1, 1 << 31, 8, 8, 1, 0, 0, 0.5), (1, 2, 1, 9, 8, 8, 1, 0, 0, "x"), (1, 2, 1, 9, 8, 8, 1, 0, 0, [1.0])):
        with pytest.raises(ValueError, match="32 bits"):
            A._pack_dims(*f)
