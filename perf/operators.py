"""The linear-attention operators (a decay for each head) as they are measured.

S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T and o_t = scale S_t^T q_t, over prompts (``fwd``), their
gradient (``bwd``) and single tokens on a pool of states (``step``).  Query and key heads are shared by
groups of value heads where Hk < H.  Sizes are those of the repository's base and lm_layer workloads
(state rows as the key width, channels per head as the value width), and generic ones.
"""

import math

import torch

own = False


def listed():
    return [
        # one more turn of a chat: a short odd prompt on top of a kept state; latency counts
        dict(name="fwd_turn", op="fwd", B=1, H=8, Hk=8, L=77, dk=64, dv=64, dtype="bf16", pack=0, const=False, state=True),
        # the base workload's batch in fp32, one constant decay per head
        dict(name="fwd_base", op="fwd", B=4, H=8, Hk=8, L=4096, dk=16, dv=64, dtype="f32", pack=0, const=True, state=False),
        # a training batch of the lm_layer shape: 24 heads, 64 state rows, 768 / 24 channels
        dict(name="fwd_lm", op="fwd", B=16, H=24, Hk=24, L=2048, dk=64, dv=32, dtype="bf16", pack=0, const=False, state=False),
        # serving prompts of different lengths in one call, q and k shared by three value heads
        dict(name="fwd_packed", op="fwd", B=1, H=24, Hk=8, L=12001, dk=128, dv=64, dtype="bf16", pack=23, const=False, state=True),
        # one long document: few rows, a long axis
        dict(name="fwd_long", op="fwd", B=1, H=16, Hk=16, L=65536, dk=128, dv=128, dtype="bf16", pack=0, const=False, state=False),
        # the gradient of a small fp32 fine-tuning step with constant decays
        dict(name="bwd_small", op="bwd", B=2, H=4, Hk=4, L=1000, dk=64, dv=64, dtype="f32", pack=0, const=True, state=True),
        # the gradient of the lm_layer training batch
        dict(name="bwd_lm", op="bwd", B=16, H=24, Hk=24, L=2048, dk=64, dv=32, dtype="bf16", pack=0, const=False, state=False),
        # the gradient over packed documents with shared query and key heads
        dict(name="bwd_packed", op="bwd", B=1, H=16, Hk=4, L=8190, dk=128, dv=128, dtype="bf16", pack=9, const=False, state=True),
        # one user's next token: latency counts
        dict(name="step_one", op="step", B=1, H=16, Hk=16, L=1, dk=128, dv=128, dtype="bf16", pack=0, const=False, state=False),
        # an odd batch of the base shape in fp32, constant decays
        dict(name="step_base", op="step", B=33, H=8, Hk=8, L=1, dk=16, dv=64, dtype="f32", pack=0, const=True, state=False),
        # a decoding batch of the lm_layer shape
        dict(name="step_lm", op="step", B=64, H=24, Hk=24, L=1, dk=64, dv=32, dtype="bf16", pack=0, const=False, state=False),
        # a full server: 250 users and 6 empty rows on a pool of 300 slots
        dict(name="step_pool", op="step", B=256, H=16, Hk=4, L=1, dk=128, dv=128, dtype="bf16", pack=300, const=False, state=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "bwd", "step"))
    group = rng.choice((1, 1, 2, 3, 4))
    Hk = _log(rng, 1, 16)
    while Hk * group > 32:
        Hk //= 2
    H = Hk * group
    dk = rng.choice((16, 24, 32, 64, 64, 80, 96, 128, 128, 192, 256))
    dv = rng.choice((16, 32, 40, 64, 64, 96, 128, 128, 160, 256))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    const = rng.random() < 0.3
    state = rng.random() < 0.5
    if op == "step":
        most = max(1, min(512, (256 * 16 * 128 * 128) // (H * dk * dv)))
        B = _log(rng, 1, most)
        return dict(op=op, B=B, H=H, Hk=Hk, L=1, dk=dk, dv=dv, dtype=dtype,
                    pack=B + rng.randint(1, 40) if state else 0, const=const, state=state)
    # no dearer than the longest listed prompt (in fp32 and backwards a quarter of it)
    most = (65536 * 16 * 256) // (H * (dk + dv)) // (1 if op == "fwd" and dtype == "bf16" else 4)
    L = _log(rng, 1, min(65536, most))
    if rng.random() < 0.4:
        return dict(op=op, B=1, H=H, Hk=Hk, L=L, dk=dk, dv=dv, dtype=dtype, pack=rng.randint(1, 40), const=const, state=state)
    B = _log(rng, 1, max(1, min(32, most // L)))
    return dict(op=op, B=B, H=H, Hk=Hk, L=L, dk=dk, dv=dv, dtype=dtype, pack=0, const=const, state=state)


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    rows, H, Hk, dk, dv = c["B"] * c["L"], c["H"], c["Hk"], c["dk"], c["dv"]
    decay = H * 4 if c["const"] else rows * H * 4
    state = H * dk * dv * 4
    qk, vv = rows * Hk * dk * es, rows * H * dv * es
    if c["op"] == "step":
        return {"bytes": 2 * qk + 2 * vv + decay + 2 * c["B"] * state, "flops": 5 * c["B"] * H * dk * dv}
    seqs = c["pack"] or c["B"]
    ends = seqs * state * (2 if c["state"] else 1)
    if c["op"] == "fwd":
        return {"bytes": 2 * qk + 2 * vv + decay + ends, "flops": 5 * rows * H * dk * dv}
    # S and dS again, three products, and the decays' gradient
    return {"bytes": 4 * qk + 3 * vv + 2 * decay + ends + seqs * state * c["state"], "flops": 14 * rows * H * dk * dv}


def _lengths(case, seed):
    """Sequence lengths of a packed case: long and short ones, some empty where there are many."""
    n, total = case["pack"], case["L"]
    gen = torch.Generator().manual_seed(seed)
    w = torch.randn(n, generator=gen, dtype=torch.float64).mul(1.2).exp()
    if n > 12:
        w[int(torch.randint(0, n, (1,), generator=gen))] = 0.0
    cut = (w.cumsum(0) / w.sum() * total).round().long().tolist()
    cut[-1] = total
    return [b - a for a, b in zip([0] + cut[:-1], cut)]


def prepare(case, seed):
    c = case
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    gen = torch.Generator("cuda").manual_seed(seed)
    B, H, Hk, L, dk, dv = (c[k] for k in ("B", "H", "Hk", "L", "dk", "dv"))

    def normal(*shape, dtype=torch.float32, size=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(size).to(dtype)

    # token-major, as a projection writes them; keys of about unit length
    s = {"case": c, "q": normal(B, L, Hk, dk, dtype=dt), "k": normal(B, L, Hk, dk, dtype=dt, size=dk ** -0.5),
         "v": normal(B, L, H, dv, dtype=dt), "scale": dk ** -0.5}
    if c["const"]:
        s["log_decay"] = torch.log1p(-torch.exp2(-torch.linspace(2.0, 9.0, H, device="cuda")))
        s["log_decay"] *= 1.0 + 0.05 * torch.rand(H, generator=gen, device="cuda")
    else:
        # horizons from a few steps to some thousands
        s["log_decay"] = -torch.exp(normal(B, L, H, size=1.5) - 4.0)
    if c["op"] == "step":
        for n in ("q", "k", "v"):
            s[n] = s[n][:, 0]
        if not c["const"]:
            s["log_decay"] = s["log_decay"][:, 0]
        slots = c["pack"] or B
        s["state"] = normal(slots, H, dk, dv)
        if c["pack"]:
            idx = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
            if B > 40:
                idx[-6:] = -1
            s["state_idx"] = idx
            s["rows"] = torch.nonzero(idx >= 0)[:, 0]
            s["slots"] = idx[s["rows"]].long()
        return s
    lens = _lengths(c, seed) if c["pack"] else [L] * B
    s["lens"] = lens
    if c["pack"]:
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
        s["cu_seqlens"] = cu.cuda()
    if c["state"]:
        s["h0"] = normal(len(lens), H, dk, dv)
    if c["op"] == "bwd":
        s["g_o"] = normal(B, L, H, dv, dtype=dt)
        if c["state"]:
            s["g_hL"] = normal(len(lens), H, dk, dv, size=0.1)
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import structured_sparse_state_pdssm_amd as P
    c = s["case"]
    if c["op"] == "step":
        o = P.pdssm_linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], state_idx=s.get("state_idx"), scale=s["scale"])
        return {"o": o, "state": s["state"]}
    q, k, v = (s[n].transpose(1, 2) for n in ("q", "k", "v"))
    la = s["log_decay"] if c["const"] else s["log_decay"].transpose(1, 2)
    if c["op"] == "fwd":
        o, hL = P.pdssm_linattn_fwd(q, k, v, la, h0=s.get("h0"), scale=s["scale"], cu_seqlens=s.get("cu_seqlens"))
        return {"o": o.transpose(1, 2), "h_L": hL}
    g = P.pdssm_linattn_bwd(q, k, v, la, s["g_o"].transpose(1, 2), h0=s.get("h0"), g_hL=s.get("g_hL"), scale=s["scale"],
                            cu_seqlens=s.get("cu_seqlens"), want_h0=c["state"])
    out = {n: g[n].transpose(1, 2) for n in ("g_q", "g_k", "g_v")}
    out["g_log_decay"] = g["g_log_decay"] if c["const"] else g["g_log_decay"].transpose(1, 2)
    if c["state"]:
        out["g_h0"] = g["g_h0"]
    return out


# ---------------------------------------------------------------- plain form

CHUNK = 64


def _plain(s):
    c = s["case"]
    if c["op"] == "step":
        return _plain_step(s)
    if not c["pack"]:
        parts = [{n: s[n] for n in ("q", "k", "v", "h0", "g_o", "g_hL") if n in s}]
        las = [s["log_decay"]]
    else:
        parts, las, at = [], [], 0
        for i, n in enumerate(s["lens"]):
            p = {x: s[x][:, at:at + n] for x in ("q", "k", "v", "g_o") if x in s}
            p.update({x: s[x][i:i + 1] for x in ("h0", "g_hL") if x in s})
            parts.append(p)
            las.append(s["log_decay"] if c["const"] else s["log_decay"][:, at:at + n])
            at += n
    outs = [_plain_part(p, la, c, s["scale"]) for p, la in zip(parts, las)]
    if len(outs) == 1:
        return outs[0]
    joined = {}
    for n in outs[0]:
        if n in ("h_L", "g_h0"):
            joined[n] = torch.cat([o[n] for o in outs])
        elif n == "g_log_decay" and c["const"]:
            joined[n] = torch.stack([o[n] for o in outs]).sum(0)
        else:
            joined[n] = torch.cat([o[n] for o in outs], dim=1)
    return joined


def _plain_part(p, la, c, scale):
    """One batch of sequences of one length, in chunks: token-major inputs, fp32 products, decay sums in 64 bits."""
    B, L, H, dv = p["v"].shape
    Hk, dk = p["q"].shape[2:]
    r, dt, dev = H // Hk, p["v"].dtype, p["v"].device
    nC = (L + CHUNK - 1) // CHUNK
    pad = nC * CHUNK - L

    def lay(x, rep):  # [B,L,h,d] -> [B,H,nC,C,d] fp32
        x = x.float().transpose(1, 2)
        if rep > 1:
            x = x.repeat_interleave(rep, dim=1)
        x = torch.nn.functional.pad(x, (0, 0, 0, pad))
        return x.reshape(B, H, nC, CHUNK, x.shape[-1])

    def back(x):  # and back, rounded once
        return x.reshape(B, H, nC * CHUNK, x.shape[-1])[:, :, :L]

    q, k, v = lay(p["q"], r), lay(p["k"], r), lay(p["v"], 1)
    la = la.double().expand(B, L, H) if c["const"] else la.double()
    la = torch.nn.functional.pad(la.transpose(1, 2), (0, pad)).reshape(B, H, nC, CHUNK)
    G = la.cumsum(-1)
    tot = G[..., -1:]
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    W = torch.where(tri, (G[..., :, None] - G[..., None, :]).clamp(max=0.0).exp().float(), 0.0)   # [.., i, j]
    ai, wj, A = G.exp().float()[..., None], (tot - G).exp().float()[..., None], tot.exp().float()[..., None]

    h = p["h0"] if "h0" in p else torch.zeros(B, H, dk, dv, device=dev)
    add = torch.matmul((k * wj).transpose(-1, -2), v)
    S = []
    for i in range(nC):
        S.append(h)
        h = A[:, :, i] * h + add[:, :, i]
    S = torch.stack(S, dim=2) if S else torch.zeros(B, H, 0, dk, dv, device=dev)
    QK = torch.matmul(q, k.transpose(-1, -2)) * W
    if c["op"] == "fwd":
        o = (ai * torch.matmul(q, S) + torch.matmul(QK, v)) * scale
        return {"o": back(o).transpose(1, 2).to(dt), "h_L": h}

    do = lay(p["g_o"], 1)
    d = p["g_hL"] if "g_hL" in p else torch.zeros(B, H, dk, dv, device=dev)
    add = torch.matmul((q * ai).transpose(-1, -2), do) * scale
    dS = [None] * nC
    for i in reversed(range(nC)):
        dS[i] = d
        d = A[:, :, i] * d + add[:, :, i]
    dS = torch.stack(dS, dim=2) if dS else torch.zeros(B, H, 0, dk, dv, device=dev)
    OV = torch.matmul(do, v.transpose(-1, -2)) * W * scale
    dq_far = ai * torch.matmul(do, S.transpose(-1, -2)) * scale
    dk_far = wj * torch.matmul(v, dS.transpose(-1, -2))
    dq = dq_far + torch.matmul(OV, k)
    dkk = dk_far + torch.matmul(OV.transpose(-1, -2), q)
    dvv = wj * torch.matmul(k, dS) + torch.matmul(QK.transpose(-1, -2), do) * scale
    # d log a_t: pairs with the key before t and the query at or behind it; inside the chunk, from either side, and past both
    M = torch.where(tri, (torch.matmul(q, k.transpose(-1, -2)) * OV).double(), 0.0)
    M = M.tril(-1)
    rows, cols = M.sum(-1), M.sum(-2)

    def rest(x):  # sums from t to the chunk's end
        return x.flip(-1).cumsum(-1).flip(-1)

    near = rest(rows - cols)
    r_far = rest((q * dq_far).double().sum(-1))
    c_all = (k * dk_far).double().sum(-1)
    c_far = c_all.cumsum(-1) - c_all
    far = (A * S * dS).double().sum((-1, -2))[..., None]
    dla = back((near + r_far + c_far + far)[..., None])[..., 0]

    def fold(x):  # gradients of shared heads add up
        x = back(x)
        return (x.reshape(B, Hk, r, L, x.shape[-1]).sum(2) if r > 1 else x).transpose(1, 2).to(dt)

    out = {"g_q": fold(dq), "g_k": fold(dkk), "g_v": back(dvv).transpose(1, 2).to(dt)}
    out["g_log_decay"] = dla.sum((0, 2)).float() if c["const"] else dla.transpose(1, 2).float()
    if c["state"]:
        out["g_h0"] = d
    return out


def _plain_step(s):
    q, k, v, la, pool = s["q"].float(), s["k"].float(), s["v"].float(), s["log_decay"], s["state"]
    B, H, dv = v.shape
    r = H // q.shape[1]
    if r > 1:
        q, k = q.repeat_interleave(r, dim=1), k.repeat_interleave(r, dim=1)
    a = (la.exp().expand(B, H) if la.dim() == 1 else la.exp())[..., None, None]
    if "slots" not in s:
        pool.mul_(a).add_(k[..., :, None] * v[..., None, :])
        o = (q[..., :, None] * pool).sum(-2) * s["scale"]
        return {"o": o.to(s["v"].dtype), "state": pool}
    rows, slots = s["rows"], s["slots"]
    S = a[rows] * pool[slots] + k[rows][..., :, None] * v[rows][..., None, :]
    pool[slots] = S
    o = torch.zeros(B, H, dv, device=v.device)
    o[rows] = (q[rows][..., :, None] * S).sum(-2) * s["scale"]
    return {"o": o.to(s["v"].dtype), "state": pool}


# ---------------------------------------------------------------- 64 bits, step by step

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    scale = s["scale"]
    if c["op"] == "step":
        out = torch.zeros(c["B"], c["H"], c["dv"], dtype=torch.float64, device="cuda")
        pool = s["state"].double()
        at = s["state_idx"].tolist() if "state_idx" in s else range(c["B"])
        r = c["H"] // c["Hk"]
        for b, slot in enumerate(at):
            if slot < 0:
                continue
            la = s["log_decay"] if c["const"] else s["log_decay"][b]
            q, k = (s[n][b].double()[torch.arange(c["H"], device="cuda") // r] for n in ("q", "k"))
            pool[slot] = pool[slot] * la.double().exp()[:, None, None] + torch.einsum("hi,hj->hij", k, s["v"][b].double())
            out[b] = torch.einsum("hi,hij->hj", q, pool[slot]) * scale
        return {"o": out, "state": pool}

    lens = s["lens"]
    n, most = len(lens), max(lens)
    H, Hk, dk, dv = c["H"], c["Hk"], c["dk"], c["dv"]
    if most * (2.0 if c["op"] == "bwd" else 1.0) * (40e-6 + n * H * dk * dv * 50 / 2.5e12) > 18:
        return None
    head = torch.arange(H, device="cuda") // (H // Hk)
    if c["pack"]:
        row = [torch.arange(a, a + m, device="cuda") for a, m in zip([sum(lens[:i]) for i in range(n)], lens)]

    def steps(x, rep):  # [most, n, H, ...] in 64 bits, zeros behind each end
        x = x.double()
        if rep:
            x = x[:, :, head]
        if not c["pack"]:
            return x.transpose(0, 1).contiguous()
        y = torch.zeros((most, n) + tuple(x.shape[2:]), dtype=torch.float64, device="cuda")
        for i, at in enumerate(row):
            y[:lens[i], i] = x[0, at]
        return y

    def rows(y):  # and back to the inputs' rows
        if not c["pack"]:
            return y.transpose(0, 1)
        return torch.cat([y[:lens[i], i] for i in range(n)])[None]

    q, k, v = steps(s["q"], True), steps(s["k"], True), steps(s["v"], False)
    la = s["log_decay"].double().expand(c["B"], c["L"], H) if c["const"] else s["log_decay"]
    a = steps(la, False).exp()[..., None, None]
    zero = torch.zeros(n, H, dk, dv, dtype=torch.float64, device="cuda")
    S = s["h0"].double() if "h0" in s else zero.clone()
    o = torch.empty_like(v)
    do = steps(s["g_o"], False) if c["op"] == "bwd" else None
    dq = torch.empty_like(q)
    for t in range(most):
        S = torch.addcmul(S * a[t], k[t][..., :, None], v[t][..., None, :])
        if do is None:
            torch.sum(S * q[t][..., :, None], dim=-2, out=o[t])
        else:
            torch.sum(S * do[t][..., None, :], dim=-1, out=dq[t])
    if do is None:
        return {"o": rows(o) * scale, "h_L": S}
    dq *= scale
    D = s["g_hL"].double() if "g_hL" in s else zero.clone()
    end = (S * D).sum((-1, -2))
    dk_, dv_ = torch.empty_like(k), torch.empty_like(v)
    for t in reversed(range(most)):
        D = torch.addcmul(D, q[t][..., :, None], do[t][..., None, :], value=scale)
        torch.sum(D * v[t][..., None, :], dim=-1, out=dk_[t])
        torch.sum(D * k[t][..., :, None], dim=-2, out=dv_[t])
        D = D * a[t]
    # pairs (key before t, query at or behind t): all queries from t on, without the keys from t on, and what reaches the end
    dla = ((q * dq).sum(-1) - (k * dk_).sum(-1)).flip(0).cumsum(0).flip(0) + end
    live = torch.arange(most, device="cuda")[:, None, None] < torch.tensor(lens, device="cuda")[:, None]
    dla = torch.where(live, dla, 0.0)

    def fold(x):
        x = rows(x)
        return x.reshape(x.shape[0], x.shape[1], Hk, H // Hk, x.shape[-1]).sum(3)

    out = {"g_q": fold(dq), "g_k": fold(dk_), "g_v": rows(dv_)}
    out["g_log_decay"] = dla.sum((0, 1)) if c["const"] else rows(dla)
    if c["state"]:
        out["g_h0"] = D
    return out
