"""Plain fp64 numpy oracle of linear attention with a decay for each head.

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t

Step by step from the definition, one sequence batch at a time; test
infrastructure only.  q, k [B,Hk,L,dk]; v [B,H,L,dv]; g [B,H,L]; states
[B,H,dk,dv].
"""

import numpy as np


def _heads(x, H):
    return np.repeat(np.asarray(x, np.float64), H // x.shape[1], axis=1)


def linattn_fwd(q, k, v, g, h0=None, scale=1.0):
    """(o [B,H,L,dv], h_L, S [L+1,B,H,dk,dv] with S[0] = h0)."""
    v = np.asarray(v, np.float64)
    B, H, L, dv = v.shape
    q, k = _heads(q, H), _heads(k, H)
    a = np.exp(np.asarray(g, np.float64))
    S = np.zeros((L + 1, B, H, q.shape[-1], dv))
    if h0 is not None:
        S[0] = h0
    o = np.zeros_like(v)
    for t in range(L):
        S[t + 1] = a[:, :, t, None, None] * S[t] + k[:, :, t, :, None] * v[:, :, t, None, :]
        o[:, :, t] = scale * np.einsum("bhi,bhij->bhj", q[:, :, t], S[t + 1])
    return o, S[L].copy(), S


def linattn_bwd(q, k, v, g, g_o, h0=None, g_hL=None, scale=1.0):
    """dict(g_q, g_k, g_v, g_g [B,H,L], g_h0) by the chain rule, one step at a time."""
    v = np.asarray(v, np.float64)
    B, H, L, dv = v.shape
    Hk, dk = q.shape[1], q.shape[-1]
    S = linattn_fwd(q, k, v, g, h0, scale)[2]
    q, k, do = _heads(q, H), _heads(k, H), np.asarray(g_o, np.float64)
    a = np.exp(np.asarray(g, np.float64))
    D = np.zeros((B, H, dk, dv)) if g_hL is None else np.array(g_hL, np.float64)
    gq, gk, gv, gg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((B, H, L))
    for t in reversed(range(L)):
        D = D + scale * q[:, :, t, :, None] * do[:, :, t, None, :]          # dLoss / dS_t
        gq[:, :, t] = scale * np.einsum("bhij,bhj->bhi", S[t + 1], do[:, :, t])
        gk[:, :, t] = np.einsum("bhij,bhj->bhi", D, v[:, :, t])
        gv[:, :, t] = np.einsum("bhij,bhi->bhj", D, k[:, :, t])
        gg[:, :, t] = a[:, :, t] * (S[t] * D).sum((-1, -2))
        D = a[:, :, t, None, None] * D
    fold = lambda x: x.reshape(B, Hk, H // Hk, L, dk).sum(2)  # noqa: E731
    return {"g_q": fold(gq), "g_k": fold(gk), "g_v": gv, "g_g": gg, "g_h0": D}


def linattn_step(q, k, v, g, state, state_idx=None, scale=1.0):
    """(o [B,H,dv], new state pool): q, k [B,Hk,dk]; v [B,H,dv]; g [B,H]."""
    v = np.asarray(v, np.float64)
    B, H, dv = v.shape
    q, k = _heads(q, H), _heads(k, H)
    pool = np.array(state, np.float64)
    o = np.zeros((B, H, dv))
    seen = set()
    for b in range(B):
        s = b if state_idx is None else int(state_idx[b])
        if s < 0:
            continue
        if s >= pool.shape[0] or s in seen:
            o[b] = np.nan
            continue
        seen.add(s)
        pool[s] = np.exp(np.asarray(g, np.float64)[b])[:, None, None] * pool[s] + k[b, :, :, None] * v[b, :, None, :]
        o[b] = scale * np.einsum("hi,hij->hj", q[b], pool[s])
    return o, pool
