"""The selective layer's calls on the host, no GPU: what the binding refuses
before the library is reached, and what the C ABI refuses under the host
sanitizers, before any launch."""

import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "structured_sparse_state_pdssm_amd", "csrc")
SAN = os.path.join(ROOT, "tests", "sanitize")
HIP_INC = "/opt/rocm/include"
f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def P():
    from tests._libutil import ensure_built
    ensure_built()
    import structured_sparse_state_pdssm_amd as P
    return P


def z(*s, dt=f32):
    return torch.zeros(s, dtype=dt)


B, L, D, N, G, W = 2, 10, 32, 16, 2, 4


def conv(**kw):
    return dict(dict(x=z(B, L, D), w=z(D, W)), **kw)


def scan(**kw):
    return dict(dict(x=z(B, L, D), dt=z(B, L, D), A=z(D, N), Bm=z(B, G, L, N), Cm=z(B, G, L, N)), **kw)


def norm(**kw):
    return dict(dict(x=z(B, 3, L, D), w=z(3, D)), **kw)


def test_correct_calls_stop_at_the_device_check(P):
    calls = [
        (P.pdssm_conv_fwd, conv(bias=z(D), x0=z(B, W - 1, D))),
        (P.pdssm_conv_fwd, conv(x=z(1, L, D), cu_seqlens=z(4, dt=i32), x0=z(3, W - 1, D))),
        (P.pdssm_conv_bwd, conv(g_y=z(B, L, D), g_xL=z(B, W - 1, D))),
        (P.pdssm_conv_step, dict(x=z(B, D), w=z(D, W), state=z(5, W - 1, D), state_idx=z(B, dt=i32))),
        (P.pdssm_selscan_fwd, scan(D=z(D), z=z(B, L, D), dt_bias=z(D), h0=z(B, D, N))),
        (P.pdssm_selscan_bwd, scan(g_y=z(B, L, D), g_hL=z(B, D, N))),
        (P.pdssm_selscan_step, dict(x=z(B, D), dt=z(B, D), A=z(D, N), Bm=z(B, G, N), Cm=z(B, G, N), state=z(5, D, N))),
        (P.pdssm_norm_fwd, norm(z=z(B, 3, L, D), gate="after", residual=z(B, 3, L, D), res_scale=z(3, D))),
        (P.pdssm_norm_fwd, norm(w=z(D))),
        (P.pdssm_norm_fwd, dict(x=z(B, L, D), w=z(D))),
        (P.pdssm_norm_bwd, norm(g_y=z(B, 3, L, D), z=z(B, 3, L, D), gate="before")),
    ]
    for fn, a in calls:
        with pytest.raises(ValueError, match="device tensor"):
            fn(**a)


@pytest.mark.parametrize("name,bad,err", [
    ("x", z(B, L), ValueError), ("x", z(B, L, D, dt=torch.float16), TypeError), ("x", None, TypeError),
    ("w", z(D + 8, W), ValueError), ("w", z(D, W, dt=bf16), TypeError), ("w", z(D), ValueError),
    ("bias", z(D + 1), ValueError), ("x0", z(B, W, D), ValueError), ("x0", z(B, W - 1, D, dt=bf16), TypeError),
    ("cu_seqlens", z(3, dt=i32), ValueError), ("cu_seqlens", z(1, dt=i32), ValueError),
])
def test_conv_refusals(P, name, bad, err):
    with pytest.raises(err, match=name if name != "cu_seqlens" else "cu_seqlens"):
        P.pdssm_conv_fwd(**conv(**{name: bad}))
    with pytest.raises(err, match=name if name != "cu_seqlens" else "cu_seqlens"):
        P.pdssm_conv_bwd(**conv(**{name: bad}), g_y=z(B, L, D))


@pytest.mark.parametrize("name,bad,err", [
    ("x", z(B, L), ValueError), ("dt", z(B, L + 1, D), ValueError), ("dt", None, TypeError), ("dt", z(B, L, D, dt=bf16), TypeError),
    ("A", z(D + 8, N), ValueError), ("A", None, TypeError), ("Bm", z(B, G, L, N + 8), ValueError), ("Bm", z(B, L, N), ValueError),
    ("Cm", z(B, G + 1, L, N), ValueError), ("Cm", None, TypeError), ("D", z(D + 1), ValueError), ("z", z(B, L, D + 8), ValueError),
    ("dt_bias", z(1), ValueError), ("h0", z(B, N, D), ValueError), ("h0", z(B, D, N, dt=bf16), TypeError),
    ("cu_seqlens", z(3, dt=i32), ValueError),
])
def test_scan_refusals(P, name, bad, err):
    match = name if name != "cu_seqlens" else "batch axis"
    with pytest.raises(err, match=match):
        P.pdssm_selscan_fwd(**scan(**{name: bad}))
    with pytest.raises(err, match=match):
        P.pdssm_selscan_bwd(**scan(**{name: bad}), g_y=z(B, L, D))


@pytest.mark.parametrize("kw,err,match", [
    (dict(x=z(L, D)), ValueError, "x must be"), (dict(w=z(4, D)), ValueError, "w must have shape"), (dict(w=None), TypeError, "w must"),
    (dict(gate="after"), ValueError, "come together"), (dict(z=z(B, 3, L, D)), ValueError, "come together"),
    (dict(z=z(B, 3, L, D), gate="middle"), ValueError, "gate must be"), (dict(res_scale=z(D)), ValueError, "res_scale must have shape"),
    (dict(z=z(B, 3, L + 1, D), gate="after"), ValueError, "z must have shape"), (dict(eps="x"), ValueError, "32 bits"),
])
def test_norm_refusals(P, kw, err, match):
    from structured_sparse_state_pdssm_amd import _ssm
    if "eps" in kw:
        with pytest.raises(err, match=match):
            _ssm._pack(_ssm._struct_norm, 1, 1, 1, 8, 0, 0, 0, kw["eps"])
        return
    with pytest.raises(err, match=match):
        P.pdssm_norm_fwd(**norm(**kw))
    with pytest.raises(err, match=match):
        P.pdssm_norm_bwd(**norm(**kw), g_y=z(B, 3, L, D))


def test_unknown_outputs(P):
    """A misspelt name in out= would leave the tensor as it was."""
    with pytest.raises(ValueError, match="'h_l'.*h_L"):
        P.pdssm_selscan_fwd(**scan(), out={"h_l": z(B, D, N)})
    with pytest.raises(ValueError, match="'g_b'"):
        P.pdssm_selscan_bwd(**scan(), g_y=z(B, L, D), out={"g_b": z(B, G, L, N)})
    with pytest.raises(ValueError, match="'xL'.*x_L"):
        P.pdssm_conv_fwd(**conv(), out={"xL": z(B, W - 1, D)})
    with pytest.raises(TypeError, match="out must be a dict"):
        P.pdssm_norm_bwd(**norm(), g_y=z(B, 3, L, D), out=z(B, 3, L, D))


def test_step_refusals(P):
    a = dict(x=z(B, D), dt=z(B, D), A=z(D, N), Bm=z(B, G, N), Cm=z(B, G, N), state=z(5, D, N))
    for kw, err in ((dict(state=z(5, N, D)), ValueError), (dict(state=z(5, D, N, dt=bf16)), TypeError), (dict(dt=None), TypeError),
                    (dict(state_idx=z(B)), TypeError), (dict(state_idx=z(B + 1, dt=i32)), ValueError), (dict(Bm=z(B, N)), ValueError)):
        with pytest.raises(err):
            P.pdssm_selscan_step(**dict(a, **kw))
    a = dict(x=z(B, D, dt=bf16), w=z(D, W), state=z(5, W - 1, D, dt=bf16))
    for kw, err in ((dict(state=z(5, W - 1, D)), TypeError), (dict(state=z(5, W, D, dt=bf16)), ValueError), (dict(x=z(B, 1, D)), ValueError)):
        with pytest.raises(err):
            P.pdssm_conv_step(**dict(a, **kw))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INC), reason="needs g++ and the HIP headers")
def test_abi_under_sanitizers(tmp_path):
    """Validation, workspace sizes and grids of ordinary and extreme dims: built with g++ against launchers that only
    check what they are given."""
    exe = str(tmp_path / "ssm_validation")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
           f"-I{HIP_INC}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(CSRC, "pdscan_ssm_api.cpp"),
           os.path.join(SAN, "ssm_validation.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok: 0 failures" in r.stdout, r.stdout + r.stderr
