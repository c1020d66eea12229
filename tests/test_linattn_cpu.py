"""The linear-attention calls on the host, no GPU: the binding checks every
tensor before the library is reached, the C ABI refuses bad arguments before
any HIP call, and the same validation runs under the host sanitizers."""

import ctypes
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "structured_sparse_state_pdssm_amd", "csrc")
f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def P():
    from tests._libutil import ensure_built
    ensure_built()
    import structured_sparse_state_pdssm_amd as P
    return P


B, H, Hk, L, dk, dv = 2, 4, 2, 10, 32, 64


def z(*s, dt=f32):
    return torch.zeros(s, dtype=dt)


def args(**kw):
    a = dict(q=z(B, Hk, L, dk), k=z(B, Hk, L, dk), v=z(B, H, L, dv), log_decay=z(B, H, L))
    a.update(kw)
    return a


def test_correct_host_calls_stop_at_the_device_check(P):
    for fn, a in ((P.pdssm_linattn_fwd, args()), (P.pdssm_linattn_fwd, args(log_decay=z(H), h0=z(B, H, dk, dv))),
                  (P.pdssm_linattn_bwd, args(g_o=z(B, H, L, dv))),
                  (P.pdssm_linattn_step, dict(q=z(B, Hk, dk), k=z(B, Hk, dk), v=z(B, H, dv), log_decay=z(B, H),
                                              state=z(9, H, dk, dv), state_idx=z(B, dt=i32)))):
        with pytest.raises(ValueError, match="device tensor"):
            fn(**a)


@pytest.mark.parametrize("name,bad,err", [
    ("q", z(B, Hk, L), "q must be"), ("k", z(B, Hk, L, dk + 8), "k must have shape"),
    ("k", z(B, Hk + 1, L, dk), "k must have shape"), ("v", z(B, H, L + 1, dv), "v must have shape"),
    ("log_decay", z(B, H, L + 1), "log_decay must have shape"), ("log_decay", z(H + 1), "log_decay must have shape"),
    ("h0", z(B, H, dv, dk), "h0 must have shape"), ("h0", z(1, H, dk, dv), "h0 must have shape"),
    ("cu_seqlens", z(3, dt=i32), "batch axis"), ("cu_seqlens", z(1, dt=i32), "cu_seqlens must be"),
])
def test_wrong_shapes(P, name, bad, err):
    with pytest.raises(ValueError, match=err):
        P.pdssm_linattn_fwd(**args(**{name: bad}))
    with pytest.raises(ValueError, match=err):
        P.pdssm_linattn_bwd(**args(**{name: bad}), g_o=z(B, H, L, dv))


@pytest.mark.parametrize("name,bad", [("q", z(B, Hk, L, dk, dt=bf16)), ("k", z(B, Hk, L, dk, dt=torch.float16)),
                                      ("v", z(B, H, L, dv, dt=torch.float16)), ("log_decay", z(B, H, L, dt=bf16)),
                                      ("h0", z(B, H, dk, dv, dt=bf16)), ("q", None)])
def test_wrong_types(P, name, bad):
    with pytest.raises(TypeError, match=name if name != "v" else "v must be|must be"):
        P.pdssm_linattn_fwd(**args(**{name: bad}))


def test_outputs_and_packing(P):
    with pytest.raises(ValueError, match="o must have shape"):
        P.pdssm_linattn_fwd(**args(), out={"o": z(B, H, L, dv - 8)})
    with pytest.raises(ValueError, match="h_L must have shape"):
        P.pdssm_linattn_fwd(**args(), out={"h_L": z(B, H, dv, dk)})
    for n, t in (("g_q", z(B, H, L, dk)), ("g_v", z(B, H, L, dk)), ("g_log_decay", z(H)), ("g_h0", z(H, dk, dv))):
        with pytest.raises(ValueError, match=f"{n} must have shape"):
            P.pdssm_linattn_bwd(**args(), g_o=z(B, H, L, dv), out={n: t})
    with pytest.raises(TypeError, match="cu_seqlens must be"):
        P.pdssm_linattn_fwd(q=z(1, Hk, L, dk), k=z(1, Hk, L, dk), v=z(1, H, L, dv), log_decay=z(H),
                            cu_seqlens=z(4, dt=torch.int64))
    with pytest.raises(ValueError, match="h0 must have shape"):   # one state a sequence
        P.pdssm_linattn_fwd(q=z(1, Hk, L, dk), k=z(1, Hk, L, dk), v=z(1, H, L, dv), log_decay=z(H),
                            cu_seqlens=z(4, dt=i32), h0=z(1, H, dk, dv))


def test_step_shapes(P):
    good = dict(q=z(B, Hk, dk), k=z(B, Hk, dk), v=z(B, H, dv), log_decay=z(B, H), state=z(9, H, dk, dv))
    for n, t, err in (("state", z(9, H, dv, dk), "state must have shape"), ("state", z(H, dk, dv), "state must be"),
                      ("state_idx", z(B + 1, dt=i32), "state_idx must have shape"), ("k", z(B, Hk, dk + 8), "k must have"),
                      ("q", z(B, Hk, 1, dk), "q must be"), ("log_decay", z(B, H, 1), "log_decay must have")):
        with pytest.raises(ValueError, match=err):
            P.pdssm_linattn_step(**{**good, n: t})
    with pytest.raises(TypeError, match="state_idx"):
        P.pdssm_linattn_step(**good, state_idx=z(B, dt=torch.int64))


def _fwd(P, d, **kw):
    """The C call on fake addresses that are never dereferenced: every case here must be refused."""
    V = P._lib.PdssmView
    at = lambda i: 0x7f0000000000 + (i << 36)  # noqa: E731
    st = (10 * 4 * 64, 64, 4 * 64)
    p = dict(q=V(at(0), *st), k=V(at(1), *st), v=V(at(2), *st), g=V(at(3), *st), cu=None, h0=at(4), o=V(at(5), *st),
             hL=at(6), ws=at(7), n=1 << 40)
    p.update(kw)
    return P.lib.pdssm_linattn_fwd(d, p["q"], p["k"], p["v"], p["g"], p["cu"], p["h0"], p["o"], p["hL"], p["ws"], p["n"], None)


def test_abi_refusals(P):
    from structured_sparse_state_pdssm_amd import _lib
    P._lib = _lib
    V = _lib.PdssmView
    d = P.linattn_dims(2, 4, 10, 32, 64, Hk=4)
    at = lambda i: 0x7f0000000000 + (i << 36)  # noqa: E731
    st = (10 * 4 * 64, 64, 4 * 64)
    for kw in (dict(q=V(None, *st)), dict(q=None), dict(o=V(None, *st)), dict(hL=None), dict(ws=None), dict(g=None),
               dict(q=V(at(0) + 8, *st)), dict(g=V(at(3) + 2, *st)), dict(k=V(at(1), 2562, 64, 256)),
               dict(v=V(at(2), -64, 64, 256)), dict(cu=at(9)), dict(h0=at(4) + 4), dict(o=V(at(2), *st)),
               dict(o=V(at(5), 0, 64, 256)), dict(o=V(at(5), 2560, 32, 256)), dict(hL=at(4)), dict(ws=at(5))):
        assert _fwd(P, d, **kw) == P.PDSSM_EINVAL, kw
        assert P.lib.pdssm_last_error() != b""
    assert _fwd(P, d, n=255) == -3
    for f, v, code in (("B", 0, -1), ("H", 0, -1), ("Hk", 3, -1), ("L", 0, -1), ("dk", 0, -1), ("dk", 12, -2), ("dv", 264, -2),
                       ("in_dtype", 2, -1), ("packed", 2, -1), ("decay_per_head", 3, -1), ("scale", float("nan"), -1),
                       ("packed", 1, -1)):
        e = P.linattn_dims(2, 4, 10, 32, 64, Hk=4)
        setattr(e, f, v)
        assert _fwd(P, e) == code, (f, v)


def test_limits_of_strides(P):
    """Step strides, and the partial gradients' of shared heads, that a lane's 32-bit offsets would not hold."""
    from structured_sparse_state_pdssm_amd import _lib
    P._lib = _lib
    V = _lib.PdssmView
    at = lambda i: 0x7f0000000000 + (i << 36)  # noqa: E731
    d = P.linattn_dims(1, 4, 10, 32, 64, Hk=4)
    far = 1 << 23
    for n, i in (("q", 0), ("k", 1), ("v", 2), ("o", 5)):
        assert _fwd(P, d, n=255, **{n: V(at(i), 0, 64, far)}) == -3       # every check passed but the workspace's size
        assert _fwd(P, d, n=255, **{n: V(at(i), 0, 64, far + 4)}) == -2 and n.encode() in P.lib.pdssm_last_error()
    assert _fwd(P, d, n=255, g=V(at(3), 0, 1, far + 4)) == -3              # the decays' is not bounded
    one = P.linattn_dims(1, 4, 1, 32, 64, Hk=4)
    assert _fwd(P, one, n=255, q=V(at(0), 0, 64, far + 4)) == -3           # one step: not looked at
    wide = V(at(0), 0, 256, 256)
    rest = [V(at(i), 0, 256, 256) for i in range(1, 9)]

    def bwd(H, Hk):
        e = P.linattn_dims(1, H, 1, 256, 8, Hk=Hk, bf16=True)
        return P.lib.pdssm_linattn_bwd(e, wide, rest[0], rest[1], V(at(9), 0, 1, 0), None, None, rest[2], None, rest[3],
                                       rest[4], rest[5], V(at(10), 0, 1, 0), None, at(11), 255, None)

    assert bwd(1 << 15, 1) == -3 and bwd((1 << 15) + 2, 2) == -2 and b"shared heads" in P.lib.pdssm_last_error()


def test_step_abi_refusals(P):
    from structured_sparse_state_pdssm_amd import _lib
    V = _lib.PdssmView
    at = lambda i: 0x7f0000000000 + (i << 36)  # noqa: E731

    def call(d, slots=5, idx=at(6), state=at(5), o=V(at(4), 256, 64, 0)):
        return P.lib.pdssm_linattn_step(d, V(at(0), 256, 64, 0), V(at(1), 256, 64, 0), V(at(2), 256, 64, 0), V(at(3), 4, 1, 0),
                                        idx, slots, state, o, None)

    d = P.linattn_dims(2, 4, 1, 32, 64, Hk=4)
    assert call(d, slots=0) == -1 and call(d, slots=1, idx=None) == -1 and call(d, state=None) == -1
    assert call(d, state=at(5) + 8) == -1 and call(d, o=V(at(5), 256, 64, 0)) == -1 and call(d, idx=at(6) + 2) == -1
    assert call(P.linattn_dims(2, 4, 2, 32, 64)) == -1 and call(P.linattn_dims(2, 4, 1, 32, 64, packed=True)) == -1


def test_interleaved_outputs_are_told_apart(P):
    """Slices of one row-interleaved buffer share no byte; one row more does.  Checked by what the refusal names."""
    from structured_sparse_state_pdssm_amd import _lib
    V = _lib.PdssmView
    base = 0x7f0000000000
    d = P.linattn_dims(2, 4, 10, 32, 64, Hk=4)
    row = 4 * (32 + 32 + 64)             # q | k | v of all heads, fp32
    at = lambda off: base + 4 * off  # noqa: E731
    q, k, v = (V(at(o), 10 * row, w, row) for o, w in ((0, 32), (128, 32), (256, 64)))
    far = base + (1 << 40)
    ok = dict(q=q, k=k, v=v, g=V(far, 40, 10, 1), cu=None, h0=None, hL=far + (1 << 30), ws=far + (2 << 30), n=255)
    fits = V(far + (3 << 30), 10 * row, 64, row)
    P._lib = _lib
    assert _fwd(P, d, o=fits, **ok) == -3                      # passes every check but the workspace's size
    big = dict(ok, n=1 << 30)
    assert _fwd(P, d, o=V(at(200), 10 * row, 64, row), **big) == -1 and b"overlaps input" in P.lib.pdssm_last_error()


def test_workspace_sizes(P):
    # many rows: the header alone; few rows and a long axis: one state and its decay a segment
    assert P.linattn_workspace_bytes(P.linattn_dims(64, 16, 2048, 128, 128)) == 256
    n = P.linattn_workspace_bytes(P.linattn_dims(1, 1, 4096, 64, 64))
    assert n > 256 + 64 * 64 * 4 and (n - 256) % 256 == 0
    # many sequences in few rows: a state for every whole chunk of 64 rows and one more a sequence, at most
    m = P.linattn_workspace_bytes(P.linattn_dims(50, 1, 4096, 64, 64, packed=True))
    assert m <= 256 + (4096 // 64 + 50) * (64 * 64 * 4 + 4 + 16) + 51 * 4 + 4 * 256


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the HIP headers")
def test_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "la_san")
    san = os.path.join(ROOT, "tests", "sanitize")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
           os.path.join(CSRC, "pdscan_linattn_api.cpp"), os.path.join(san, "linattn_validation.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok: 0 failures" in r.stdout, r.stdout + r.stderr
