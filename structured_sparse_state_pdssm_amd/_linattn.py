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

import torch

from ._lib import PDSSM_BF16, PDSSM_F32, PDSSM_OK, PdssmError, PdssmLinattnDims, PdssmView, lib

_FLOATS = {torch.float32: PDSSM_F32, torch.bfloat16: PDSSM_BF16}


def _check(rc):
    if rc != PDSSM_OK:
        raise PdssmError(rc, lib.pdssm_last_error().decode())


def _tensors(specs):
    """Type, dtype and shape of every argument first, then where it lies: the
    C ABI cannot see allocation sizes.  specs: (tensor or None, name, shape,
    dtype, layout), layout "whole" (contiguous), "rows" (contiguous last axis)
    or "any".  Returns the device."""
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
        if layout == "whole":
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        elif layout == "rows" and shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"the last axis of {name} must be contiguous")
    return dev


def _view(t, heads=1, step=2):
    """A tensor [B,heads,L,..] (or [B,heads,..] with step=None) as strides."""
    s = t.stride()
    return PdssmView(t.data_ptr(), s[0], s[heads], s[step] if step is not None else 0)


def _decay_view(t, per_head, step=2):
    return PdssmView(t.data_ptr(), 0, 1, 0) if per_head else _view(t, 1, step)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _like(t, shape, dev):
    """A new tensor [B,H,L,d] in the axis order of t (step-major or head-major)."""
    B, H, L, d = shape
    if t.stride(2) > t.stride(1):
        return torch.empty((B, L, H, d), dtype=t.dtype, device=dev).transpose(1, 2)
    return torch.empty((B, H, L, d), dtype=t.dtype, device=dev)


def _dims(q, k, v, log_decay, scale, cu_seqlens, names=("[B,Hk,L,dk]", "[B,H,L,dv]"), rank=4):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_decay, "log_decay")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
    if q.dim() != rank:
        raise ValueError(f"q must be {names[0]}")
    if v.dim() != rank:
        raise ValueError(f"v must be {names[1]}")
    if v.dtype not in _FLOATS:
        raise TypeError(f"v must be float32 or bfloat16 (got {v.dtype})")
    B, Hk = q.shape[:2]
    H, dv = v.shape[1], v.shape[-1]
    dk = q.shape[-1]
    L = q.shape[2] if rank == 4 else 1
    packed = cu_seqlens is not None
    if packed:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens must be a tensor [S+1]")
        if B != 1:
            raise ValueError(f"with cu_seqlens the batch axis has one element (got {B})")
        B = cu_seqlens.shape[0] - 1
    per_head = log_decay.dim() == 1
    if scale is None:
        scale = dk ** -0.5
    return PdssmLinattnDims(B, H, Hk, L, dk, dv, _FLOATS[v.dtype], packed, per_head, scale)


class _on:
    """The tensors' device as the current one for the length of a call."""

    def __init__(self, dev):
        self.to = dev.index if dev.index is not None else torch.cuda.current_device()

    def __enter__(self):
        self.back = torch.cuda.current_device()
        if self.back != self.to:
            torch.cuda.set_device(self.to)
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def __exit__(self, *_):
        if self.back != self.to:
            torch.cuda.set_device(self.back)


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
    _tensors([(workspace, "workspace", workspace.shape if isinstance(workspace, torch.Tensor) else None, torch.uint8,
               "whole")])
    if workspace.device != dev:
        raise ValueError(f"workspace is on {workspace.device}, q on {dev}")
    if workspace.numel() < nbytes:
        raise ValueError(f"workspace holds {workspace.numel()} bytes, {nbytes} needed")
    return workspace


def pdssm_linattn_fwd(q, k, v, log_decay, h0=None, scale=None, cu_seqlens=None, workspace=None, out=None):
    """Prompts.  Returns (o [B,H,L,dv], h_L [B,H,dk,dv]).  ``scale`` is
    dk ** -0.5 when not given; ``out`` may hold "o" and "h_L" to write to."""
    d = _dims(q, k, v, log_decay, scale, cu_seqlens)
    rows = v.shape[0]
    H, L, dk, dv, dt = d.H, d.L, d.dk, d.dv, v.dtype
    kshape, vshape, sshape = (rows, d.Hk, L, dk), (rows, H, L, dv), (d.B, H, dk, dv)
    dev = q.device
    res = out or {}
    o, hL = res.get("o"), res.get("h_L")
    f32 = torch.float32
    _tensors([(q, "q", kshape, dt, "rows"), (k, "k", kshape, dt, "rows"), (v, "v", vshape, dt, "rows"),
              (log_decay, "log_decay", (H,) if d.decay_per_head else (rows, H, L), f32, "whole" if d.decay_per_head else "any"),
              (h0, "h0", sshape, f32, "whole"), (cu_seqlens, "cu_seqlens", (d.B + 1,), torch.int32, "whole"),
              (o, "o", vshape, dt, "rows"), (hL, "h_L", sshape, f32, "whole")])
    with _on(dev) as stream:
        if o is None:
            o = _like(v, vshape, dev)
        if hL is None:
            hL = torch.empty(sshape, dtype=f32, device=dev)
        ws = _workspace(linattn_workspace_bytes(d), dev, workspace)
        _check(lib.pdssm_linattn_fwd(d, _view(q), _view(k), _view(v), _decay_view(log_decay, d.decay_per_head),
                                     _ptr(cu_seqlens), _ptr(h0), _view(o), _ptr(hL), _ptr(ws), ws.numel(), stream))
    return o, hL


def pdssm_linattn_bwd(q, k, v, log_decay, g_o, h0=None, g_hL=None, scale=None, cu_seqlens=None, want_h0=True,
                      workspace=None, out=None):
    """Gradient of pdssm_linattn_fwd, given the gradients of o and (optional)
    h_L.  Returns dict(g_q, g_k, g_v, g_log_decay[, g_h0]), shaped and typed
    as their inputs; g_h0 is dLoss/dh0 also where h0 is left out (zero)."""
    d = _dims(q, k, v, log_decay, scale, cu_seqlens)
    rows = v.shape[0]
    H, L, dk, dv, dt = d.H, d.L, d.dk, d.dv, v.dtype
    kshape, vshape, sshape = (rows, d.Hk, L, dk), (rows, H, L, dv), (d.B, H, dk, dv)
    gshape = (H,) if d.decay_per_head else (rows, H, L)
    per_head = bool(d.decay_per_head)
    dev = q.device
    f32 = torch.float32
    given = out or {}
    res = {n: given.get(n) for n in ("g_q", "g_k", "g_v", "g_log_decay")}
    if want_h0:
        res["g_h0"] = given.get("g_h0")
    _tensors([(q, "q", kshape, dt, "rows"), (k, "k", kshape, dt, "rows"), (v, "v", vshape, dt, "rows"),
              (log_decay, "log_decay", gshape, f32, "whole" if per_head else "any"), (g_o, "g_o", vshape, dt, "rows"),
              (h0, "h0", sshape, f32, "whole"), (g_hL, "g_hL", sshape, f32, "whole"),
              (cu_seqlens, "cu_seqlens", (d.B + 1,), torch.int32, "whole"), (res["g_q"], "g_q", kshape, dt, "rows"),
              (res["g_k"], "g_k", kshape, dt, "rows"), (res["g_v"], "g_v", vshape, dt, "rows"),
              (res["g_log_decay"], "g_log_decay", gshape, f32, "whole" if per_head else "any"), (res.get("g_h0"), "g_h0", sshape, f32, "whole")])
    with _on(dev) as stream:
        for n, t, shape in (("g_q", q, kshape), ("g_k", k, kshape), ("g_v", v, vshape)):
            if res[n] is None:
                res[n] = _like(t, shape, dev)
        if res["g_log_decay"] is None:
            g = log_decay
            res["g_log_decay"] = (torch.empty((rows, L, H), dtype=f32, device=dev).transpose(1, 2)
                                  if not per_head and g.stride(2) > g.stride(1)
                                  else torch.empty(gshape, dtype=f32, device=dev))
        if want_h0 and res["g_h0"] is None:
            res["g_h0"] = torch.empty(sshape, dtype=f32, device=dev)
        ws = _workspace(linattn_bwd_workspace_bytes(d), dev, workspace)
        _check(lib.pdssm_linattn_bwd(d, _view(q), _view(k), _view(v), _decay_view(log_decay, per_head),
                                     _ptr(cu_seqlens), _ptr(h0), _view(g_o), _ptr(g_hL), _view(res["g_q"]),
                                     _view(res["g_k"]), _view(res["g_v"]), _decay_view(res["g_log_decay"], per_head),
                                     _ptr(res.get("g_h0")), _ptr(ws), ws.numel(), stream))
    return res


def pdssm_linattn_step(q, k, v, log_decay, state, state_idx=None, scale=None, out=None):
    """One token of every row: q, k [B,Hk,dk], v [B,H,dv], log_decay [B,H] or
    [H].  ``state`` [n_slots,H,dk,dv] is updated in place; row b uses slot
    ``state_idx[b]`` (int32; b when not given).  A negative slot is an empty
    row (o zero, no state touched); one past the pool, or named by an earlier
    row too, gives NaN in o and touches nothing.  Returns o [B,H,dv]
    (``out``: a tensor to write it to)."""
    d = _dims(q, k, v, log_decay, scale, None, ("[B,Hk,dk]", "[B,H,dv]"), 3)
    B, H, dk, dv, dt = d.B, d.H, d.dk, d.dv, v.dtype
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a tensor [n_slots,H,dk,dv]")
    slots = state.shape[0]
    per_head = bool(d.decay_per_head)
    f32 = torch.float32
    dev = _tensors([(q, "q", (B, d.Hk, dk), dt, "rows"), (k, "k", (B, d.Hk, dk), dt, "rows"), (v, "v", (B, H, dv), dt, "rows"),
                    (log_decay, "log_decay", (H,) if per_head else (B, H), f32, "whole" if per_head else "any"),
                    (state, "state", (slots, H, dk, dv), f32, "whole"),
                    (state_idx, "state_idx", (B,), torch.int32, "whole"), (out, "out", (B, H, dv), dt, "rows")])
    with _on(dev) as stream:
        if out is None:
            out = torch.empty((B, H, dv), dtype=dt, device=dev)
        _check(lib.pdssm_linattn_step(d, _view(q, 1, None), _view(k, 1, None), _view(v, 1, None),
                                      _decay_view(log_decay, per_head, None), _ptr(state_idx), slots, _ptr(state),
                                      _view(out, 1, None), stream))
    return out
