"""Linear attention with a decay for each head (the pdssm_linattn_* calls of
include/pdscan.h): prompts, their gradient and single tokens.

    S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t

Shapes: q, k [B,Hk,L,dk]; v, o, g_o [B,H,L,dv]; log_decay [B,H,L], or [H] for
one constant per head; states [B,H,dk,dv].  Value head h reads query / key
head h // (H // Hk).  q, k, v (float32 or bfloat16, one type) and log_decay
(float32) may have any strides; those of q, k and v leave the last axis
contiguous.  [B,L,H,d] tensors pass as ``x.transpose(1, 2)``; outputs made
here follow the axis order of the tensor they belong to (o and g_v of v, g_q
of q, g_k of k).

Packed sequences: B is 1 in the tensors, L counts all rows and
``cu_seqlens`` (int32, on the device, [S+1]) bounds the S sequences; states
are [S,H,dk,dv].  Rows outside every sequence are not written: where the
outputs are made here they hold whatever the memory held.
"""

import ctypes
import struct
from collections.abc import Mapping

import torch

from ._lib import PDSSM_BF16, PDSSM_F32, PDSSM_OK, PdssmError, PdssmLinattnDims, lib

_FLOATS = {torch.float32: PDSSM_F32, torch.bfloat16: PDSSM_BF16}
_f32, _i32 = torch.float32, torch.int32
_WHOLE, _ROWS, _ANY = range(3)   # layouts: contiguous, contiguous last axis, any strides

# A call is a few microseconds of host work, which is all of a small step's
# time: arguments go as packed bytes (pdssm_linattn_dims, pdssm_view) through
# functions of their own, and the checks run as one expression whose failure
# is explained by the slower ones.
_struct_dims = struct.Struct("9if").pack
_pack_view = struct.Struct("Pqqq").pack


def _fn(name, types):
    f = lib[name]
    f.argtypes = [{"s": ctypes.c_char_p, "p": ctypes.c_void_p, "n": ctypes.c_size_t, "i": ctypes.c_int32}[c]
                  for c in types]
    f.restype = ctypes.c_int
    return f


_fwd = _fn("pdssm_linattn_fwd", "sssssppsppnp")
_bwd = _fn("pdssm_linattn_bwd", "sssssppspsssspp" + "np")
_fwd_bytes = _fn("pdssm_linattn_workspace_bytes", "sp")
_bwd_bytes = _fn("pdssm_linattn_bwd_workspace_bytes", "sp")
_step = _fn("pdssm_linattn_step", "ssssspipsp")


def _check(rc):
    if rc != PDSSM_OK:
        raise PdssmError(rc, lib.pdssm_last_error().decode())


def _explain(specs):
    """Raise what is wrong with the arguments: type, dtype and shape of every
    one first, then where it lies (the C ABI cannot see allocation sizes).
    specs: (tensor or None, name, shape, dtype, layout)."""
    for t, name, shape, dtype, _ in specs:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    dev = specs[0][0].device
    for t, name, shape, _, layout in specs:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor (got {t.device})")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, {specs[0][1]} on {dev}")
        if layout is _WHOLE:
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        elif layout is _ROWS and t.stride(-1) != 1:
            raise ValueError(f"the last axis of {name} must be contiguous")


def _verify(specs, dev):
    if dev < 0:
        return _explain(specs)
    for t, _, shape, dtype, layout in specs:
        if t is not None and not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                                  and t.get_device() == dev
                                  and (layout is _ANY or (t.stride(-1) == 1 if layout is _ROWS else t.is_contiguous()))):
            return _explain(specs)


def _pack_dims(*fields):
    try:
        return _struct_dims(*fields)
    except struct.error:
        raise ValueError(f"scale {fields[-1]!r} or a size in {fields[:6]} (B, H, Hk, L, dk, dv) is no number of 32 bits") from None


def _view(t):
    """A tensor [B,heads,L,..] as pointer and strides."""
    s = t.stride()
    return _pack_view(t.data_ptr(), s[0], s[1], s[2])


def _view1(t):
    """A tensor [B,heads,..] of single tokens."""
    s = t.stride()
    return _pack_view(t.data_ptr(), s[0], s[1], 0)


def _decay_view(t, per_head):
    return _pack_view(t.data_ptr(), 0, 1, 0) if per_head else _view(t)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _like(t, shape, dev):
    """A new tensor [B,H,L,d] in the axis order of t (step-major or head-major)."""
    B, H, L, d = shape
    if t.stride(2) > t.stride(1):
        return torch.empty((B, L, H, d), dtype=t.dtype, device=dev).transpose(1, 2)
    return torch.empty((B, H, L, d), dtype=t.dtype, device=dev)


def _shapes(q, k, v, log_decay, rank, names):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_decay, "log_decay")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
    if q.dim() != rank:
        raise ValueError(f"q must be {names[0]}")
    if v.dim() != rank:
        raise ValueError(f"v must be {names[1]}")
    if v.dtype not in _FLOATS:
        raise TypeError(f"v must be float32 or bfloat16 (got {v.dtype})")


def _dims(q, k, v, log_decay, scale, cu_seqlens):
    """(fields of pdssm_linattn_dims, rows of the batch axis)."""
    _shapes(q, k, v, log_decay, 4, ("[B,Hk,L,dk]", "[B,H,L,dv]"))
    rows, Hk, L, dk = q.shape
    H, dv = v.shape[1], v.shape[3]
    B = rows
    packed = cu_seqlens is not None
    if packed:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens must be a tensor [S+1]")
        if rows != 1:
            raise ValueError(f"with cu_seqlens the batch axis has one element (got {rows})")
        B = cu_seqlens.shape[0] - 1
    if scale is None:
        scale = dk ** -0.5
    return (B, H, Hk, L, dk, dv, _FLOATS[v.dtype], packed, log_decay.dim() == 1, scale), rows


def _call(index, fn):
    """fn(stream) with the tensors' device as the current one."""
    if torch._C._cuda_getDevice() == index:
        return fn(torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(index):
        return fn(torch._C._cuda_getCurrentRawStream(index))


def _bytes(fn, packed):
    n = ctypes.c_size_t(0)
    _check(fn(packed, ctypes.addressof(n)))
    return n.value


def linattn_workspace_bytes(dims):
    n = ctypes.c_size_t(0)
    _check(lib.pdssm_linattn_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)))
    return n.value


def linattn_bwd_workspace_bytes(dims):
    n = ctypes.c_size_t(0)
    _check(lib.pdssm_linattn_bwd_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)))
    return n.value


def linattn_dims(B, H, L, dk, dv, Hk=None, bf16=False, packed=False, decay_per_head=False, scale=1.0):
    """Dims of a call, for the workspace queries (packed: B sequences in L rows)."""
    return PdssmLinattnDims(B, H, H if Hk is None else Hk, L, dk, dv, PDSSM_BF16 if bf16 else PDSSM_F32, packed,
                            decay_per_head, scale)


def _workspace(nbytes, dev, workspace):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a torch.uint8 tensor")
    _verify([(workspace, "workspace", workspace.shape, torch.uint8, _WHOLE)], dev.index)
    if workspace.numel() < nbytes:
        raise ValueError(f"workspace holds {workspace.numel()} bytes, {nbytes} needed")
    return workspace


def _given(out, names):
    """The caller's outputs, by name: a misspelt one would be left as it is."""
    if out is None:
        return {}
    if not isinstance(out, Mapping):
        raise TypeError(f"out must be a dict (got {type(out).__name__})")
    for n in out:
        if n not in names:
            raise ValueError(f"out has no {n!r}: {', '.join(names)}")
    return out


def pdssm_linattn_fwd(q, k, v, log_decay, h0=None, scale=None, cu_seqlens=None, workspace=None, out=None):
    """Prompts.  Returns (o [B,H,L,dv], h_L [B,H,dk,dv]).  ``scale`` is
    dk ** -0.5 when not given; ``out`` may hold "o" and "h_L" to write to."""
    d, rows = _dims(q, k, v, log_decay, scale, cu_seqlens)
    B, H, Hk, L, dk, dv, _, _, per_head, _ = d
    dt, index = v.dtype, q.get_device()
    kshape, vshape, sshape = (rows, Hk, L, dk), (rows, H, L, dv), (B, H, dk, dv)
    given = _given(out, ("o", "h_L"))
    o, hL = given.get("o"), given.get("h_L")
    _verify([(q, "q", kshape, dt, _ROWS), (k, "k", kshape, dt, _ROWS), (v, "v", vshape, dt, _ROWS),
             (log_decay, "log_decay", (H,) if per_head else (rows, H, L), _f32, _WHOLE if per_head else _ANY),
             (h0, "h0", sshape, _f32, _WHOLE), (cu_seqlens, "cu_seqlens", (B + 1,), _i32, _WHOLE),
             (o, "o", vshape, dt, _ROWS), (hL, "h_L", sshape, _f32, _WHOLE)], index)
    dev = q.device
    dims = _pack_dims(*d)
    if o is None:
        o = _like(v, vshape, dev)
    if hL is None:
        hL = torch.empty(sshape, dtype=_f32, device=dev)
    ws = _workspace(_bytes(_fwd_bytes, dims), dev, workspace)
    _check(_call(index, lambda stream: _fwd(
        dims, _view(q), _view(k), _view(v), _decay_view(log_decay, per_head), _ptr(cu_seqlens), _ptr(h0), _view(o),
        hL.data_ptr(), ws.data_ptr(), ws.numel(), stream)))
    return o, hL


def pdssm_linattn_bwd(q, k, v, log_decay, g_o, h0=None, g_hL=None, scale=None, cu_seqlens=None, want_h0=True,
                      workspace=None, out=None):
    """Gradient of pdssm_linattn_fwd, given the gradients of o and (optional)
    h_L.  Returns dict(g_q, g_k, g_v, g_log_decay[, g_h0]), shaped and typed
    as their inputs; g_h0 is dLoss/dh0 also where h0 is left out (zero).
    ``out`` may hold any of them to write to (g_h0 only with want_h0)."""
    d, rows = _dims(q, k, v, log_decay, scale, cu_seqlens)
    if not isinstance(g_o, torch.Tensor):
        raise TypeError("g_o must be a torch.Tensor")
    B, H, Hk, L, dk, dv, _, _, per_head, _ = d
    dt, index = v.dtype, q.get_device()
    kshape, vshape, sshape = (rows, Hk, L, dk), (rows, H, L, dv), (B, H, dk, dv)
    gshape = (H,) if per_head else (rows, H, L)
    glayout = _WHOLE if per_head else _ANY
    given = _given(out, ("g_q", "g_k", "g_v", "g_log_decay", "g_h0"))
    res = {n: given.get(n) for n in ("g_q", "g_k", "g_v", "g_log_decay")}
    if want_h0:
        res["g_h0"] = given.get("g_h0")
    _verify([(q, "q", kshape, dt, _ROWS), (k, "k", kshape, dt, _ROWS), (v, "v", vshape, dt, _ROWS),
             (log_decay, "log_decay", gshape, _f32, glayout), (g_o, "g_o", vshape, dt, _ROWS),
             (h0, "h0", sshape, _f32, _WHOLE), (g_hL, "g_hL", sshape, _f32, _WHOLE),
             (cu_seqlens, "cu_seqlens", (B + 1,), _i32, _WHOLE), (res["g_q"], "g_q", kshape, dt, _ROWS),
             (res["g_k"], "g_k", kshape, dt, _ROWS), (res["g_v"], "g_v", vshape, dt, _ROWS),
             (res["g_log_decay"], "g_log_decay", gshape, _f32, glayout),
             (res.get("g_h0"), "g_h0", sshape, _f32, _WHOLE)], index)
    dev = q.device
    dims = _pack_dims(*d)
    for n, t, shape in (("g_q", q, kshape), ("g_k", k, kshape), ("g_v", v, vshape)):
        if res[n] is None:
            res[n] = _like(t, shape, dev)
    if res["g_log_decay"] is None:
        res["g_log_decay"] = (torch.empty((rows, L, H), dtype=_f32, device=dev).transpose(1, 2)
                              if not per_head and log_decay.stride(2) > log_decay.stride(1)
                              else torch.empty(gshape, dtype=_f32, device=dev))
    if want_h0 and res["g_h0"] is None:
        res["g_h0"] = torch.empty(sshape, dtype=_f32, device=dev)
    ws = _workspace(_bytes(_bwd_bytes, dims), dev, workspace)
    _check(_call(index, lambda stream: _bwd(
        dims, _view(q), _view(k), _view(v), _decay_view(log_decay, per_head), _ptr(cu_seqlens), _ptr(h0), _view(g_o),
        _ptr(g_hL), _view(res["g_q"]), _view(res["g_k"]), _view(res["g_v"]),
        _decay_view(res["g_log_decay"], per_head), _ptr(res.get("g_h0")), ws.data_ptr(), ws.numel(), stream)))
    return res


def pdssm_linattn_step(q, k, v, log_decay, state, state_idx=None, scale=None, out=None):
    """One token of every row: q, k [B,Hk,dk], v [B,H,dv], log_decay [B,H] or
    [H].  ``state`` [n_slots,H,dk,dv] is updated in place; row b uses slot
    ``state_idx[b]`` (int32; b when not given).  A negative slot is an empty
    row (o zero, no state touched); one past the pool, or named by an earlier
    row too, gives NaN in o and touches nothing.  Returns o [B,H,dv]
    (``out``: a tensor to write it to)."""
    _shapes(q, k, v, log_decay, 3, ("[B,Hk,dk]", "[B,H,dv]"))
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a tensor [n_slots,H,dk,dv]")
    kshape, vshape = q.shape, v.shape
    B, Hk, dk = kshape
    H, dv = vshape[1], vshape[2]
    slots = state.shape[0]
    per_head = log_decay.dim() == 1
    dt, index = v.dtype, q.get_device()
    _verify([(q, "q", (B, Hk, dk), dt, _ROWS), (k, "k", kshape, dt, _ROWS), (v, "v", (B, H, dv), dt, _ROWS),
             (log_decay, "log_decay", (H,) if per_head else (B, H), _f32, _WHOLE if per_head else _ANY),
             (state, "state", (slots, H, dk, dv), _f32, _WHOLE), (state_idx, "state_idx", (B,), _i32, _WHOLE),
             (out, "out", vshape, dt, _ROWS)], index)
    if out is None:
        out = torch.empty(vshape, dtype=dt, device=q.device)
    dims = _pack_dims(B, H, Hk, 1, dk, dv, _FLOATS[dt], 0, per_head, dk ** -0.5 if scale is None else scale)
    _check(_call(index, lambda stream: _step(
        dims, _view1(q), _view1(k), _view1(v),
        _pack_view(log_decay.data_ptr(), 0, 1, 0) if per_head else _view1(log_decay), _ptr(state_idx), slots,
        state.data_ptr(), _view1(out), stream)))
    return out
