"""The selective state-space layer (the pdssm_conv_*, pdssm_selscan_* and
pdssm_norm_* calls of include/pdscan.h): a short causal convolution, the
selective scan and the norm around a block, with their gradients, and single
tokens of the first two.

    conv     y_t = act(bias + sum_j w[:, j] x_{t-W+1+j})
    selscan  d_t = softplus(dt_t + dt_bias),  h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,
             y_t = (C_t . h_t + D x_t) silu(z_t)
    norm     y = residual + res_scale * (w * u / sqrt(mean(u^2) + eps)) [* silu(z)],
             u = x, or x * silu(z)

Shapes: x, dt, z, y [B,L,D]; B and C [B,G,L,N], a group of D / G channels
each; A [D,N]; w [D,W]; scan states [B,D,N] (float32), convolution states
[B,W-1,D] (inputs as they are, the oldest first); a norm's rows [B,H,L,d] or
[B,L,d].  Inputs are float32 or bfloat16, one type a call; weights are
float32.  Inputs may have any strides that are multiples of 16 bytes, with
the last axis contiguous: slices of one projection's rows pass as they are.

Packed sequences: as in ``_linattn``.  Rows outside every sequence are not
written.
"""

import struct

import torch

from ._linattn import (
    _FLOATS,
    _ROWS,
    _WHOLE,
    _bytes,
    _call,
    _check,
    _f32,
    _fn,
    _given,
    _i32,
    _like,
    _pack_view,
    _ptr,
    _verify,
    _view,
    _view1,
    _workspace,
)

_GATES = {None: 0, "before": 1, "after": 2}

_struct_conv = struct.Struct("7i").pack
_struct_scan = struct.Struct("8i").pack
_struct_norm = struct.Struct("7if").pack

_conv_fwd = _fn("pdssm_conv_fwd", "sspppp" + "spp")
_conv_bwd = _fn("pdssm_conv_bwd", "sspppp" + "sps" + "pppp" + "np")
_conv_bytes = _fn("pdssm_conv_bwd_workspace_bytes", "sp")
_conv_step = _fn("pdssm_conv_step", "ssppp" + "ips" + "p")
_scan_fwd = _fn("pdssm_selscan_fwd", "ssspss" + "pspp" + "psp" + "pnp")
_scan_bwd = _fn("pdssm_selscan_bwd", "ssspss" + "pspp" + "psp" + "ssp" + "ssp" + "spp" + "pnp")
_scan_bytes = _fn("pdssm_selscan_workspace_bytes", "sp")
_scan_bwd_bytes = _fn("pdssm_selscan_bwd_workspace_bytes", "sp")
_scan_step = _fn("pdssm_selscan_step", "ssspss" + "pspp" + "ipsp")
_norm_fwd = _fn("pdssm_norm_fwd", "sspsspsp")
_norm_bwd = _fn("pdssm_norm_bwd", "sspspsspsp" + "pnp")
_norm_bytes = _fn("pdssm_norm_bwd_workspace_bytes", "sp")


def _pack(pack, *fields):
    try:
        return pack(*fields)
    except struct.error:
        raise ValueError(f"a size or number in {fields} is none of 32 bits") from None


def _rows_view(t):
    """[B,L,D] as pointer and strides."""
    s = t.stride()
    return _pack_view(t.data_ptr(), s[0], 0, s[1])


def _row_view(t):
    """[B,D], single tokens."""
    return _pack_view(t.data_ptr(), t.stride(0), 0, 0)


def _opt(view, t):
    return None if t is None else view(t)


def _tensors(*named):
    for t, n, rank, shape in named:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
        if t.dim() != rank:
            raise ValueError(f"{n} must be {shape}")


def _dtype(t, name):
    if t.dtype not in _FLOATS:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {t.dtype})")
    return t.dtype


def _sequences(rows, cu_seqlens):
    """Sequences of a call whose batch axis has `rows` rows."""
    if cu_seqlens is None:
        return rows
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be a tensor [S+1]")
    if rows != 1:
        raise ValueError(f"with cu_seqlens the batch axis has one element (got {rows})")
    return cu_seqlens.shape[0] - 1


def _new(t, shape, dtype, like):
    """The caller's output, or a contiguous one (made the quickest way: a small call's time is the host's)."""
    if t is not None:
        return t
    if like.dtype is dtype:
        return torch.empty_like(like) if like.shape == shape and like.is_contiguous() else like.new_empty(shape)
    return like.new_empty(shape, dtype=dtype)


# ---- bytes of workspace, for calls that bring their own (packed: B sequences in L rows)

def conv_bwd_workspace_bytes(B, L, D, W, bf16=False, packed=False):
    return _bytes(_conv_bytes, _pack(_struct_conv, B, L, D, W, bool(bf16), bool(packed), 1))


def selscan_workspace_bytes(B, L, D, N, G=1, bf16=False, packed=False):
    """May be 0: no workspace is needed then."""
    return _bytes(_scan_bytes, _pack(_struct_scan, B, L, D, N, G, bool(bf16), bool(packed), 1))


def selscan_bwd_workspace_bytes(B, L, D, N, G=1, bf16=False, packed=False):
    return _bytes(_scan_bwd_bytes, _pack(_struct_scan, B, L, D, N, G, bool(bf16), bool(packed), 1))


def norm_bwd_workspace_bytes(B, H, L, d, bf16=False, per_head=False):
    return _bytes(_norm_bytes, _pack(_struct_norm, B, H, L, d, bool(bf16), 0, bool(per_head), 1.0))


# ---- convolution

def _conv_args(x, w, bias, x0, silu, cu_seqlens):
    _tensors((x, "x", 3, "[B,L,D]"), (w, "w", 2, "[D,W]"))
    dt = _dtype(x, "x")
    rows, L, D = x.shape
    W = w.shape[1]
    B = _sequences(rows, cu_seqlens)
    sshape = (B, W - 1, D)
    specs = [(x, "x", (rows, L, D), dt, _ROWS), (w, "w", (D, W), _f32, _WHOLE), (bias, "bias", (D,), _f32, _WHOLE),
             (x0, "x0", sshape, dt, _WHOLE), (cu_seqlens, "cu_seqlens", (B + 1,), _i32, _WHOLE)]
    return (B, L, D, W, _FLOATS[dt], cu_seqlens is not None, bool(silu)), sshape, specs


def pdssm_conv_fwd(x, w, bias=None, x0=None, silu=True, cu_seqlens=None, out=None):
    """Prompts.  Returns (y [B,L,D], x_L [B,W-1,D]): x_L is the x0 of what
    follows.  ``out`` may hold "y" and "x_L" to write to."""
    d, sshape, specs = _conv_args(x, w, bias, x0, silu, cu_seqlens)
    given = _given(out, ("y", "x_L"))
    y, xL = given.get("y"), given.get("x_L")
    index, dt = x.get_device(), x.dtype
    _verify(specs + [(y, "y", x.shape, dt, _ROWS), (xL, "x_L", sshape, dt, _WHOLE)], index)
    dims = _pack(_struct_conv, *d)
    y, xL = _new(y, x.shape, dt, x), _new(xL, sshape, dt, x)
    _check(_call(index, lambda stream: _conv_fwd(
        dims, _rows_view(x), w.data_ptr(), _ptr(bias), _ptr(cu_seqlens), _ptr(x0), _rows_view(y), xL.data_ptr(), stream)))
    return y, xL


def pdssm_conv_bwd(x, w, g_y, bias=None, x0=None, g_xL=None, silu=True, cu_seqlens=None, want_x0=True, workspace=None,
                   out=None):
    """Gradient of pdssm_conv_fwd, given the gradients of y and (optional)
    x_L.  Returns dict(g_x, g_w, g_bias[, g_x0]), typed as their inputs; g_bias
    and g_x0 also where bias and x0 are left out (zero).  ``out`` may hold any
    of those returned to write to, and nothing else."""
    d, sshape, specs = _conv_args(x, w, bias, x0, silu, cu_seqlens)
    _tensors((g_y, "g_y", 3, "[B,L,D]"))
    names = ["g_x", "g_w", "g_bias"] + ["g_x0"] * bool(want_x0)
    given = _given(out, names)
    res = {n: given.get(n) for n in names}
    index, dt, dev = x.get_device(), x.dtype, x.device
    D = x.shape[2]
    outs = [(res["g_x"], "g_x", x.shape, dt, _ROWS), (res["g_w"], "g_w", w.shape, _f32, _WHOLE),
            (res["g_bias"], "g_bias", (D,), _f32, _WHOLE), (res.get("g_x0"), "g_x0", sshape, dt, _WHOLE)]
    _verify(specs + [(g_y, "g_y", x.shape, dt, _ROWS), (g_xL, "g_xL", sshape, dt, _WHOLE)] + outs, index)
    dims = _pack(_struct_conv, *d)
    for _, n, shape, dtype, _ in outs:
        if n in res:
            res[n] = _new(res[n], shape, dtype, x)
    ws = _workspace(_bytes(_conv_bytes, dims), dev, workspace)
    _check(_call(index, lambda stream: _conv_bwd(
        dims, _rows_view(x), w.data_ptr(), _ptr(bias), _ptr(cu_seqlens), _ptr(x0), _rows_view(g_y), _ptr(g_xL),
        _rows_view(res["g_x"]), res["g_w"].data_ptr(), res["g_bias"].data_ptr(), _ptr(res.get("g_x0")), ws.data_ptr(),
        ws.numel(), stream)))
    return res


def pdssm_conv_step(x, w, state, bias=None, state_idx=None, silu=True, out=None):
    """One token of every row: x [B,D].  ``state`` [n_slots,W-1,D] is updated
    in place; row b uses slot ``state_idx[b]`` (int32; b when not given).  A
    negative slot is an empty row (y zero, no state touched); one past the
    pool, or named by an earlier row too, gives NaN in y and touches nothing.
    Returns y [B,D] (``out``: a tensor to write it to)."""
    _tensors((x, "x", 2, "[B,D]"), (w, "w", 2, "[D,W]"), (state, "state", 3, "[n_slots,W-1,D]"))
    dt = _dtype(x, "x")
    B, D = x.shape
    W, slots, index = w.shape[1], state.shape[0], x.get_device()
    _verify([(x, "x", (B, D), dt, _ROWS), (w, "w", (D, W), _f32, _WHOLE), (state, "state", (slots, W - 1, D), dt, _WHOLE),
             (bias, "bias", (D,), _f32, _WHOLE), (state_idx, "state_idx", (B,), _i32, _WHOLE),
             (out, "out", (B, D), dt, _ROWS)], index)
    out = _new(out, x.shape, dt, x)
    dims = _pack(_struct_conv, B, 1, D, W, _FLOATS[dt], 0, bool(silu))
    _check(_call(index, lambda stream: _conv_step(
        dims, _row_view(x), w.data_ptr(), _ptr(bias), _ptr(state_idx), slots, state.data_ptr(), _row_view(out), stream)))
    return out


# ---- selective scan

def _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, h0, cu_seqlens):
    _tensors((x, "x", 3, "[B,L,D]"), (A, "A", 2, "[D,N]"), (Bm, "Bm", 4, "[B,G,L,N]"))
    ty = _dtype(x, "x")
    rows, L, K = x.shape
    G, N = Bm.shape[1], A.shape[1]
    B = _sequences(rows, cu_seqlens)
    bshape, sshape = (rows, G, L, N), (B, K, N)
    for t, n in ((dt, "dt"), (Cm, "Cm")):
        if t is None:
            raise TypeError(f"{n} must be a torch.Tensor")
    specs = [(x, "x", (rows, L, K), ty, _ROWS), (dt, "dt", (rows, L, K), ty, _ROWS), (A, "A", (K, N), _f32, _WHOLE),
             (Bm, "Bm", bshape, ty, _ROWS), (Cm, "Cm", bshape, ty, _ROWS), (D, "D", (K,), _f32, _WHOLE),
             (z, "z", (rows, L, K), ty, _ROWS), (dt_bias, "dt_bias", (K,), _f32, _WHOLE),
             (h0, "h0", sshape, _f32, _WHOLE), (cu_seqlens, "cu_seqlens", (B + 1,), _i32, _WHOLE)]
    return (B, L, K, N, G, _FLOATS[ty], cu_seqlens is not None, bool(softplus)), sshape, specs


def pdssm_selscan_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, h0=None, cu_seqlens=None,
                      workspace=None, out=None):
    """Prompts.  Returns (y [B,L,D], h_L [B,D,N]).  ``out`` may hold "y" and
    "h_L" to write to.  A token whose dt is the type's lowest value (or minus
    infinity) is a step of zero (softplus): the state passes it as it is."""
    d, sshape, specs = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, h0, cu_seqlens)
    given = _given(out, ("y", "h_L"))
    y, hL = given.get("y"), given.get("h_L")
    index, ty, dev = x.get_device(), x.dtype, x.device
    _verify(specs + [(y, "y", x.shape, ty, _ROWS), (hL, "h_L", sshape, _f32, _WHOLE)], index)
    dims = _pack(_struct_scan, *d)
    y, hL = _new(y, x.shape, ty, x), _new(hL, sshape, _f32, x if h0 is None else h0)
    nbytes = _bytes(_scan_bytes, dims)   # none where the sequences are not cut
    ws, room = None, 0
    if nbytes or workspace is not None:
        ws = _workspace(nbytes, dev, workspace)
        room = ws.numel()
    _check(_call(index, lambda stream: _scan_fwd(
        dims, _rows_view(x), _rows_view(dt), A.data_ptr(), _view(Bm), _view(Cm), _ptr(D), _opt(_rows_view, z),
        _ptr(dt_bias), _ptr(cu_seqlens), _ptr(h0), _rows_view(y), hL.data_ptr(), _ptr(ws), room, stream)))
    return y, hL


def pdssm_selscan_bwd(x, dt, A, Bm, Cm, g_y, D=None, z=None, dt_bias=None, softplus=True, h0=None, g_hL=None,
                      cu_seqlens=None, want_h0=True, workspace=None, out=None):
    """Gradient of pdssm_selscan_fwd, given the gradients of y and (optional)
    h_L.  Returns dict(g_x, g_dt, g_A, g_B, g_C, g_D, g_dt_bias[, g_z][, g_h0]),
    shaped and typed as their inputs; g_D, g_dt_bias and g_h0 also where
    those are left out (zero).  ``out`` may hold any of those returned to
    write to, and nothing else."""
    d, sshape, specs = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, h0, cu_seqlens)
    _tensors((g_y, "g_y", 3, "[B,L,D]"))
    index, ty, dev = x.get_device(), x.dtype, x.device
    K = x.shape[2]
    names = ["g_x", "g_dt", "g_A", "g_B", "g_C", "g_D", "g_dt_bias"] + ["g_z"] * (z is not None) + ["g_h0"] * bool(want_h0)
    given = _given(out, names)
    res = {n: given.get(n) for n in names}
    outs = [(res["g_x"], "g_x", x.shape, ty, _ROWS), (res["g_dt"], "g_dt", x.shape, ty, _ROWS),
            (res["g_A"], "g_A", A.shape, _f32, _WHOLE), (res["g_B"], "g_B", Bm.shape, ty, _ROWS),
            (res["g_C"], "g_C", Bm.shape, ty, _ROWS), (res["g_D"], "g_D", (K,), _f32, _WHOLE),
            (res["g_dt_bias"], "g_dt_bias", (K,), _f32, _WHOLE), (res.get("g_z"), "g_z", x.shape, ty, _ROWS),
            (res.get("g_h0"), "g_h0", sshape, _f32, _WHOLE)]
    _verify(specs + [(g_y, "g_y", x.shape, ty, _ROWS), (g_hL, "g_hL", sshape, _f32, _WHOLE)] + outs, index)
    dims = _pack(_struct_scan, *d)
    for t, n, shape, dtype, _ in outs:
        if n in res and t is None:
            res[n] = _like(Bm if n == "g_B" else Cm, shape, dev) if n in ("g_B", "g_C") else _new(None, shape, dtype, x)
    ws = _workspace(_bytes(_scan_bwd_bytes, dims), dev, workspace)
    _check(_call(index, lambda stream: _scan_bwd(
        dims, _rows_view(x), _rows_view(dt), A.data_ptr(), _view(Bm), _view(Cm), _ptr(D), _opt(_rows_view, z),
        _ptr(dt_bias), _ptr(cu_seqlens), _ptr(h0), _rows_view(g_y), _ptr(g_hL), _rows_view(res["g_x"]),
        _rows_view(res["g_dt"]), res["g_A"].data_ptr(), _view(res["g_B"]), _view(res["g_C"]), res["g_D"].data_ptr(),
        _opt(_rows_view, res.get("g_z")), res["g_dt_bias"].data_ptr(), _ptr(res.get("g_h0")), ws.data_ptr(), ws.numel(),
        stream)))
    return res


def pdssm_selscan_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, softplus=True, state_idx=None, out=None):
    """One token of every row: x, dt, z [B,D], Bm and Cm [B,G,N].  ``state``
    [n_slots,D,N] is updated in place; ``state_idx`` as in pdssm_conv_step.
    Returns y [B,D] (``out``: a tensor to write it to)."""
    _tensors((x, "x", 2, "[B,D]"), (A, "A", 2, "[D,N]"), (Bm, "Bm", 3, "[B,G,N]"), (state, "state", 3, "[n_slots,D,N]"))
    ty = _dtype(x, "x")
    B, K = x.shape
    G, N, slots, index = Bm.shape[1], A.shape[1], state.shape[0], x.get_device()
    for t, n in ((dt, "dt"), (Cm, "Cm")):
        if t is None:
            raise TypeError(f"{n} must be a torch.Tensor")
    _verify([(x, "x", (B, K), ty, _ROWS), (dt, "dt", (B, K), ty, _ROWS), (A, "A", (K, N), _f32, _WHOLE),
             (Bm, "Bm", (B, G, N), ty, _ROWS), (Cm, "Cm", (B, G, N), ty, _ROWS),
             (state, "state", (slots, K, N), _f32, _WHOLE), (D, "D", (K,), _f32, _WHOLE), (z, "z", (B, K), ty, _ROWS),
             (dt_bias, "dt_bias", (K,), _f32, _WHOLE), (state_idx, "state_idx", (B,), _i32, _WHOLE),
             (out, "out", (B, K), ty, _ROWS)], index)
    out = _new(out, x.shape, ty, x)
    dims = _pack(_struct_scan, B, 1, K, N, G, _FLOATS[ty], 0, bool(softplus))
    _check(_call(index, lambda stream: _scan_step(
        dims, _row_view(x), _row_view(dt), A.data_ptr(), _view1(Bm), _view1(Cm), _ptr(D), _opt(_row_view, z),
        _ptr(dt_bias), _ptr(state_idx), slots, state.data_ptr(), _row_view(out), stream)))
    return out


# ---- norm

def _norm_args(x, w, z, gate, res_scale, eps):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() not in (3, 4):
        raise ValueError("x must be [B,H,L,d] or [B,L,d]")
    dt = _dtype(x, "x")
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor")
    if gate not in _GATES:
        raise ValueError(f"gate must be None, 'before' or 'after' (got {gate!r})")
    if (z is None) != (gate is None):
        raise ValueError("z and gate come together")
    B, L, d = x.shape[0], x.shape[-2], x.shape[-1]
    H = x.shape[1] if x.dim() == 4 else 1
    wshape = (H, d) if w.dim() == 2 else (d,)
    specs = [(x, "x", x.shape, dt, _ROWS), (w, "w", wshape, _f32, _WHOLE), (z, "z", x.shape, dt, _ROWS),
             (res_scale, "res_scale", wshape, _f32, _WHOLE)]
    return (B, H, L, d, _FLOATS[dt], _GATES[gate], w.dim() == 2, eps), wshape, specs


def _norm_view(t):
    return _view(t) if t.dim() == 4 else _rows_view(t)


def _norm_like(t):
    return _like(t, t.shape, t.device) if t.dim() == 4 and not t.is_contiguous() else _new(None, t.shape, t.dtype, t)


def pdssm_norm_fwd(x, w, z=None, gate=None, residual=None, res_scale=None, eps=1e-5, out=None):
    """Norm over the last axis of x [B,H,L,d] or [B,L,d].  ``w`` [H,d] (one row a
    head) or [d]; ``gate``: "before" (the norm is of x silu(z)) or "after" (it is
    multiplied by silu(z)); ``residual`` as x, added to ``res_scale`` (shaped as
    w; one when not given) times the norm.  Returns y as x (``out``: a tensor
    to write it to)."""
    d, _, specs = _norm_args(x, w, z, gate, res_scale, eps)
    index, dt = x.get_device(), x.dtype
    _verify(specs + [(residual, "residual", x.shape, dt, _ROWS), (out, "out", x.shape, dt, _ROWS)], index)
    dims = _pack(_struct_norm, *d)
    out = _norm_like(x) if out is None else out
    _check(_call(index, lambda stream: _norm_fwd(
        dims, _norm_view(x), w.data_ptr(), _opt(_norm_view, z), _opt(_norm_view, residual), _ptr(res_scale),
        _norm_view(out), stream)))
    return out


def pdssm_norm_bwd(x, w, g_y, z=None, gate=None, res_scale=None, eps=1e-5, workspace=None, out=None):
    """Gradient of pdssm_norm_fwd; the residual's is g_y itself.  Returns
    dict(g_x, g_w[, g_z][, g_res_scale]), shaped and typed as their inputs.
    ``out`` may hold any of those returned to write to, and nothing else."""
    d, wshape, specs = _norm_args(x, w, z, gate, res_scale, eps)
    if not isinstance(g_y, torch.Tensor):
        raise TypeError("g_y must be a torch.Tensor")
    index, dt, dev = x.get_device(), x.dtype, x.device
    names = ["g_x", "g_w"] + ["g_z"] * (z is not None) + ["g_res_scale"] * (res_scale is not None)
    given = _given(out, names)
    res = {n: given.get(n) for n in names}
    _verify(specs + [(g_y, "g_y", x.shape, dt, _ROWS), (res["g_x"], "g_x", x.shape, dt, _ROWS),
                     (res["g_w"], "g_w", wshape, _f32, _WHOLE), (res.get("g_z"), "g_z", x.shape, dt, _ROWS),
                     (res.get("g_res_scale"), "g_res_scale", wshape, _f32, _WHOLE)], index)
    dims = _pack(_struct_norm, *d)
    for n in names:
        if res[n] is None:
            res[n] = _norm_like(x if n == "g_x" else z) if n in ("g_x", "g_z") else _new(None, wshape, _f32, w)
    ws = _workspace(_bytes(_norm_bytes, dims), dev, workspace)
    _check(_call(index, lambda stream: _norm_bwd(
        dims, _norm_view(x), w.data_ptr(), _opt(_norm_view, z), _ptr(res_scale), _norm_view(g_y), _norm_view(res["g_x"]),
        res["g_w"].data_ptr(), _opt(_norm_view, res.get("g_z")), _ptr(res.get("g_res_scale")), ws.data_ptr(), ws.numel(),
        stream)))
    return res
