"""The selective scan's steps one by one: softplus and its slope to a few steps of
fp32, whatever their size."""

import numpy as np
import pytest

from oracle import ssm_oracle as O
from tests._gpu import lib
from tests.test_gpu_ssm import BF, DT, F32, f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = O.U


@DT
@pytest.mark.parametrize("at", [-80.0, -40.0, -16.7, -9.0, -5.0, -1.0, 0.0, 1.0, 15.0, 40.0, 1e4])
@pytest.mark.parametrize("L", [1, 40, 700])
def test_steps_keep_their_digits(L, at, dt):
    """x = B = C = 1, and states that every step forgets: y is the step itself, and the gradient of dt its slope.
    softplus has 12 half steps of fp32 and the sigmoid 8, as the oracle counts them; bf16 rounds the outputs."""
    P = lib()
    D = 64
    raw = (torch.tensor(at) + torch.linspace(-0.5, 0.5, L * D)).reshape(1, L, D).to(dt).cuda()
    one = torch.ones(1, L, D, dtype=dt, device="cuda")
    Bm = torch.zeros(1, 1, L, 8, dtype=dt, device="cuda")
    Bm[..., 0] = 1
    A = torch.full((D, 8), torch.finfo(F32).min, device="cuda")
    y, _ = P.pdssm_selscan_fwd(one, raw, A, Bm, Bm)
    g = P.pdssm_selscan_bwd(one, raw, A, Bm, Bm, one)
    half = 2.0 ** -8 if dt == BF else 0.0
    v = f64(raw)
    for got, want, n in ((y, np.logaddexp(0.0, v), 12), (g["g_dt"], np.exp(-np.logaddexp(0.0, -v)), 8)):
        assert (np.abs(f64(got) - want) <= want * (n * U + half) * 1.01).all()
