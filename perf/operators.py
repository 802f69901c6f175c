"""The operators of a packed (ragged) batch around the KDA core, and the cases
they are measured on.

Three operators, as a serving or training program calls them:

  delta   kda_packed_fwd: the gated delta rule over sequences packed one after
          another (cu_seqlens), each reading and writing its state in a pool of
          slots -- chunked for prefill, recurrent for decode and verification
  conv    kda_packed_conv: the layer's causal short convolution over the same
          packed rows, its window of K - 1 tokens kept in a pool of slots
  gn_fwd, gn_bwd   kda_group_norm_fwd / kda_group_norm_bwd: group norm over
          channels-last rows with an activation or an activated gate

`own = False` computes them in elementary torch operations in 32 bits (64 where
sums of log-decays need it); `own = True` calls the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a full serving batch, the sizes of the decode workload
        dict(name="delta_decode_channel", op="delta", n=256, tokens=256, spread=0, lens_seed=0, pad=0, fresh=0,
             H=32, HV=32, Dk=128, Dv=128, dtype="bf16", gate="bounded", per_head=False),
        # a handful of requests in a batch captured for more of them, a small fp32 model with odd heads: latency
        dict(name="delta_decode_small_fp32", op="delta", n=5, tokens=5, spread=0, lens_seed=0, pad=3, fresh=1,
             H=2, HV=6, Dk=72, Dv=40, dtype="f32", gate="none", per_head=False),
        # a verification step: each request brings a few drafted tokens
        dict(name="delta_verify_channel", op="delta", n=96, tokens=389, spread=1, lens_seed=3, pad=4, fresh=0,
             H=16, HV=32, Dk=128, Dv=128, dtype="bf16", gate="bounded", per_head=False),
        # prefill of a few prompts, one decay per channel
        dict(name="delta_prefill_channel", op="delta", n=6, tokens=2900, spread=2, lens_seed=5, pad=0, fresh=6,
             H=16, HV=16, Dk=128, Dv=128, dtype="bf16", gate="bounded", per_head=False),
        # prefill and decode rows in one batch, one decay per head, unbounded gate
        dict(name="delta_mixed_head", op="delta", n=41, tokens=8203, spread=3, lens_seed=7, pad=2, fresh=5,
             H=16, HV=32, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=True),
        # the grouped-value-head training shape as four packed sequences, one decay per head
        dict(name="delta_long_head", op="delta", n=4, tokens=32768, spread=0, lens_seed=0, pad=0, fresh=2,
             H=16, HV=32, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=True),
        # the convolution of one decode step
        dict(name="conv_decode", op="conv", n=256, tokens=256, spread=0, lens_seed=0, pad=0, fresh=0,
             C=4096, K=4, head_dim=128, silu=True, dtype="bf16"),
        # the convolution of a ragged prefill batch
        dict(name="conv_prefill", op="conv", n=11, tokens=16391, spread=2, lens_seed=11, pad=1, fresh=9,
             C=4096, K=4, head_dim=128, silu=True, dtype="bf16"),
        # the layer's epilogue per token: every head's channels normalised, times silu(gate)
        dict(name="gn_token_fwd", op="gn_fwd", N=16384, L=1, C=4096, G=32, act="silu", gate=True, dtype="bf16"),
        # and its gradient in training
        dict(name="gn_token_bwd", op="gn_bwd", N=8192, L=1, C=4096, G=32, act="silu", gate=True, dtype="bf16"),
        # statistics over a whole row of positions and a group's channels, odd length, fp32
        dict(name="gn_rows_fwd_fp32", op="gn_fwd", N=3, L=1037, C=320, G=32, act="silu", gate=False, dtype="f32"),
        # the same form in training at a large size
        dict(name="gn_rows_bwd", op="gn_bwd", N=4, L=8192, C=1024, G=32, act="silu", gate=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "verify", "channel", "head", "head", "conv", "gn_fwd", "gn_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("decode", "verify", "channel", "head"):
        H = rng.choice([1, 2, 4, 8, 16, 32])
        HV = H * rng.choice([1, 1, 2, 3])
        if HV > 32:
            HV = 32
        Dk, Dv = rng.choice([(128, 128), (128, 128), (64, 128), (96, 64), (72, 40)])
        gate = rng.choice(["bounded", "softplus", "none"])
        c = dict(op="delta", H=H, HV=HV, Dk=Dk, Dv=Dv, dtype=dtype, gate=gate, per_head=rng.random() < 0.4,
                 lens_seed=rng.randrange(1 << 20))
        if op == "decode":
            n = _log(rng, 1, 256)
            return dict(c, n=n, tokens=n, spread=0, pad=rng.choice([0, 0, 1, 7]), fresh=rng.choice([0, n // 3]))
        if op == "verify":
            n = _log(rng, 1, 128)
            return dict(c, n=n, tokens=n + rng.randrange(0, 5 * n + 1), spread=1, pad=rng.choice([0, 3]), fresh=0)
        if op == "channel":
            n = rng.randrange(1, 9)
            return dict(c, n=n, tokens=n + _log(rng, 8, 2048), spread=2, pad=0, fresh=rng.randrange(0, n + 1),
                        per_head=False)
        n = rng.randrange(1, 25)
        # a packed prefill batch of one decay per head, mostly in the width of the models
        wide = rng.random() < 0.75
        return dict(c, n=n, tokens=n + _log(rng, 64, 20000), spread=rng.choice([2, 3]), pad=rng.choice([0, 2]),
                    fresh=rng.randrange(0, n + 1), per_head=True, Dk=128 if wide else Dk, Dv=128 if wide else Dv,
                    dtype="bf16" if wide else dtype)
    if op == "conv":
        n = _log(rng, 1, 256)
        head_dim = rng.choice([0, 128])
        return dict(op="conv", n=n, tokens=n + _log(rng, 1, 8192), spread=rng.choice([1, 2, 3]),
                    lens_seed=rng.randrange(1 << 20), pad=rng.choice([0, 2]), fresh=rng.randrange(0, n + 1),
                    C=128 * rng.choice([1, 2, 5, 16, 32]), K=rng.choice([2, 3, 4, 4]), head_dim=head_dim,
                    silu=rng.random() < 0.8, dtype=dtype)
    if rng.random() < 0.5:      # per token
        G = rng.choice([1, 2, 4, 8, 16, 32])
        return dict(op=op, N=_log(rng, 1, 16384), L=1, C=G * rng.choice([32, 64, 72, 128]), G=G,
                    act=rng.choice(["none", "silu", "sigmoid"]), gate=rng.random() < 0.5, dtype=dtype)
    G = rng.choice([1, 4, 16, 32])
    return dict(op=op, N=rng.randrange(1, 9), L=_log(rng, 2, 6000), C=G * rng.choice([4, 10, 16, 24, 32]), G=G,
                act=rng.choice(["none", "silu", "sigmoid"]), gate=rng.random() < 0.25, dtype=dtype)


def _lens(c):
    """The lengths of a case's sequences: equal (0), a few each (1), spread over
    a factor of ten or more (2), or mostly single tokens beside long ones (3)."""
    n, total = c["n"], c["tokens"]
    r = random.Random(c["lens_seed"])
    if c["spread"] == 0:
        return [total // n] * (n - 1) + [total - total // n * (n - 1)]
    if c["spread"] == 1:
        w = [r.random() for _ in range(n)]
    elif c["spread"] == 2:
        w = [math.exp(r.uniform(0, 3)) for _ in range(n)]
    else:
        w = [1.0 if (i % 5 == 0) else 0.0 for i in range(n)]
        w = [x * math.exp(r.uniform(0, 2)) for x in w]
    s = sum(w)
    lens = [1 + int((total - n) * x / s) for x in w]
    i = w.index(max(w))
    for _ in range(total - sum(lens)):       # what the rounding left over, one each
        lens[i % n] += 1
        i += 1
    return lens


def _packing(c):
    """cu_seqlens over the live and the padded sequences, their slots (-1: a
    padded row of a batch captured for more requests) and fresh flags."""
    lens = _lens(c) + [1] * c["pad"]
    r = random.Random(c["lens_seed"] + 1)
    P = c["n"] + 3
    slots = r.sample(range(P), c["n"]) + [-1] * c["pad"]
    fresh = [1] * c["fresh"] + [0] * (c["n"] - c["fresh"])
    r.shuffle(fresh)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return lens, cu, slots, fresh + [0] * c["pad"], P


# ---------------------------------------------------------------- inputs
def _dt(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _dt(c)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * std)

    s = {"case": dict(c)}
    if c["op"] in ("delta", "conv"):
        lens, cu, slots, fresh, P = _packing(c)
        T = cu[-1]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["slots"] = torch.tensor(slots, dtype=torch.int32, device=DEV)
        s["fresh"] = torch.tensor(fresh, dtype=torch.uint8, device=DEV)
        s["max_len"] = max(lens)
    if c["op"] == "delta":
        H, HV, Dk, Dv = c["H"], c["HV"], c["Dk"], c["Dv"]
        gk = () if c["per_head"] else (Dk,)
        s["q"], s["k"] = normal(T, H, Dk).to(dt), normal(T, H, Dk).to(dt)
        s["v"] = normal(T, HV, Dv).to(dt)
        if c["gate"] == "none":     # the log-decay itself
            s["g"] = (-torch.rand((T, HV) + gk, generator=gen, device=DEV) * 0.5).to(dt)
        else:
            s["g"] = normal(T, HV, *gk).to(dt)
        s["beta"] = normal(T, HV).to(dt)
        s["A_log"] = torch.rand(HV, generator=gen, device=DEV) * 2 - 1 if c["gate"] != "none" else None
        s["dt_bias"] = normal(HV, *gk, std=0.5) if c["gate"] != "none" else None
        s["pool"] = normal(P, HV, Dk, Dv, std=0.05)
        s["o"] = torch.zeros(T, HV, Dv, dtype=dt, device=DEV)
        s["scale"] = Dk ** -0.5
    elif c["op"] == "conv":
        C, K = c["C"], c["K"]
        s["x"] = normal(T, C).to(dt)
        s["w"] = normal(C, K, std=0.5)
        s["bias"] = normal(C, std=0.1)
        s["pool"] = normal(P, K - 1, C).to(dt)
        s["y"] = torch.zeros(T, C, dtype=dt, device=DEV)
    else:
        N, L, C, G = c["N"], c["L"], c["C"], c["G"]
        s["x"] = (normal(N, L, C) * 1.5 + 0.3).to(dt)
        s["weight"] = 1 + normal(C, std=0.2)
        s["bias"] = normal(C, std=0.2)
        s["gate"] = normal(N, L, C).to(dt) if c["gate"] else None
        if c["op"] == "gn_bwd":
            s["dy"] = normal(N, L, C).to(dt)
            xg = s["x"].double().reshape(N, L, G, C // G)    # what the forward pass saved
            mean = xg.mean(dim=(1, 3))
            var = ((xg - mean[:, None, :, None]) ** 2).mean(dim=(1, 3))
            s["mean"], s["rstd"] = mean.float(), (1 / torch.sqrt(var + 1e-5)).float()
    return s


# ---------------------------------------------------------------- plain forms
def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _decay(s, c):
    """Log-decay in 64 bits, [T, HV, Dk or 1]."""
    g = s["g"].double()
    g = g[..., None] if c["per_head"] else g
    if c["gate"] == "none":
        return g
    b = s["dt_bias"].double()
    b = b[..., None] if c["per_head"] else b
    a = torch.exp(s["A_log"].double())[:, None]
    return -5.0 / (1 + torch.exp(-a * (g + b))) if c["gate"] == "bounded" else -a * _softplus(g + b)


def _padded(s, c):
    """[N, Lmax] row numbers of the live sequences and which of them are rows."""
    lens = s["cu"][1:] - s["cu"][:-1]
    live = s["slots"] >= 0
    start, lens, slot, fresh = (t[live].long() for t in (s["cu"][:-1], lens, s["slots"], s["fresh"]))
    at = torch.arange(s["max_len"], device=DEV)
    ok = at[None] < lens[:, None]
    rows = torch.where(ok, start[:, None] + at[None], 0)
    return rows, ok, slot, fresh


def _plain_delta(s, c):
    group = c["HV"] // c["H"]
    rows, ok, slot, fresh = _padded(s, c)
    N, L = rows.shape

    def norm(x):
        x = x.float()
        return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)

    def take(x):       # [N, HV, L, D], zero behind a sequence's end
        return (x[rows] * ok[..., None, None]).transpose(1, 2).contiguous()

    q = take(norm(s["q"]) * s["scale"]).repeat_interleave(group, 1)
    k = take(norm(s["k"])).repeat_interleave(group, 1)
    v = take(s["v"].float())
    g = take(_decay(s, c))
    beta = take((1 / (1 + torch.exp(-s["beta"].float())))[..., None])
    S = s["pool"][slot] * (fresh == 0)[:, None, None, None]
    if c["per_head"] and L > 16:
        o, S = _plain_chunks(q, k, v, g, beta, S)
    else:
        a = torch.exp(g).float()
        outs = []
        for t in range(L):
            S = S * a[:, :, t, :, None]
            e = v[:, :, t] - (S * k[:, :, t, :, None]).sum(2)
            S = S + (beta[:, :, t] * k[:, :, t])[..., None] * e[:, :, None, :]
            outs.append((S * q[:, :, t, :, None]).sum(2))
        o = torch.stack(outs, 2)
    s["pool"][slot] = S
    s["o"][rows[ok]] = o.transpose(1, 2)[ok].to(s["o"].dtype)
    return {"o": s["o"], "pool": s["pool"]}


def _plain_chunks(q, k, v, g, beta, S, C=64):
    """Chunk form for one decay per head: everything that does not need the
    state for all chunks at once, then the state from chunk to chunk."""
    N, HV, L, Dk = q.shape
    M = -(-L // C)

    def cut(x):
        return torch.nn.functional.pad(x, (0, 0, 0, M * C - L)).reshape(N, HV, M, C, -1)

    q, k, v, g, beta = map(cut, (q, k, v, g, beta))
    G = g.cumsum(3)
    low = torch.ones(C, C, device=DEV).tril()
    D = torch.exp(torch.where(low > 0, G - G.transpose(3, 4), -1e30)).float()
    A = beta * (k @ k.transpose(3, 4)) * D * low.tril(-1)
    T = torch.eye(C, device=DEV).expand_as(A).clone()     # (I + A)^-1, row by row
    for i in range(1, C):
        T[..., i, :i] = -(A[..., i:i + 1, :i] @ T[..., :i, :i])[..., 0, :]
    U0, W = T @ (beta * v), T @ (beta * torch.exp(G).float() * k)
    Q = q * torch.exp(G).float()
    B = (q @ k.transpose(3, 4)) * D
    last = G[:, :, :, -1:]
    K = k * torch.exp(last - G).float()
    end = torch.exp(last).float()
    outs = []
    for m in range(M):
        U = U0[:, :, m] - W[:, :, m] @ S
        outs.append(Q[:, :, m] @ S + B[:, :, m] @ U)
        S = end[:, :, m] * S + K[:, :, m].transpose(2, 3) @ U
    return torch.cat(outs, 2)[:, :, :L], S


def _plain_conv(s, c):
    K = c["K"]
    T = s["x"].shape[0]
    t = torch.arange(T, device=DEV)
    seq = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    start, slot = s["cu"][seq].long(), s["slots"][seq].long()
    old = (s["fresh"][seq] == 0)[:, None]
    u = s["bias"].expand(T, -1)
    xf = s["x"].float()
    for j in range(K):
        at = t - (K - 1) + j
        inside = at >= start
        before = s["pool"][slot.clamp(min=0), (at - start + K - 1).clamp(0, K - 2)].float() * old
        u = u + s["w"][:, j] * torch.where(inside[:, None], xf[at.clamp(min=0)], before)
    if c["silu"]:
        u = u / (1 + torch.exp(-u))
    if c["head_dim"]:
        h = u.reshape(T, -1, c["head_dim"])
        u = (h / torch.sqrt((h * h).sum(-1, keepdim=True) + 1e-6)).reshape(T, -1)
    live = slot >= 0
    s["y"][live] = u[live].to(s["y"].dtype)
    ln = (s["cu"][1:] - s["cu"][:-1]).long()
    alive = (s["slots"] >= 0) & (ln > 0)
    ln, first, sl, fr = ln[alive], s["cu"][:-1][alive].long(), s["slots"][alive].long(), s["fresh"][alive]
    at = ln[:, None] - (K - 1) + torch.arange(K - 1, device=DEV)
    before = s["pool"][sl[:, None], (at + K - 1).clamp(0, K - 2)] * (fr == 0)[:, None, None]
    s["pool"][sl] = torch.where((at >= 0)[..., None], s["x"][(first[:, None] + at).clamp(min=0)], before)
    return {"y": s["y"], "pool": s["pool"]}


def _act(u, act):
    return u if act == "none" else 1 / (1 + torch.exp(-u)) * (u if act == "silu" else 1)


def _act_grad(u, act):
    if act == "none":
        return torch.ones_like(u)
    p = 1 / (1 + torch.exp(-u))
    return p * (1 + u * (1 - p)) if act == "silu" else p * (1 - p)


def _plain_gn_fwd(s, c):
    N, L, C, G = c["N"], c["L"], c["C"], c["G"]
    x = s["x"].float().reshape(N, L, G, C // G)
    mean = x.mean(dim=(1, 3), keepdim=True)
    var = ((x - mean) ** 2).mean(dim=(1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + 1e-5)
    u = ((x - mean) * rstd).reshape(N, L, C) * s["weight"] + s["bias"]
    y = u * _act(s["gate"].float(), c["act"]) if c["gate"] else _act(u, c["act"])
    return {"y": y.to(s["x"].dtype), "mean": mean.reshape(N, G), "rstd": rstd.reshape(N, G)}


def _plain_gn_bwd(s, c):
    N, L, C, G = c["N"], c["L"], c["C"], c["G"]
    D = C // G
    r = s["rstd"].reshape(N, 1, G, 1)
    h = ((s["x"].float().reshape(N, L, G, D) - s["mean"].reshape(N, 1, G, 1)) * r).reshape(N, L, C)
    dy = s["dy"].float()
    u = h * s["weight"] + s["bias"]
    out = {}
    if c["gate"]:
        z = s["gate"].float()
        out["dgate"] = (dy * u * _act_grad(z, c["act"])).to(s["x"].dtype)
        du = dy * _act(z, c["act"])
    else:
        du = dy * _act_grad(u, c["act"])
    out["dweight"], out["dbias"] = (du * h).sum((0, 1)), du.sum((0, 1))
    dh = (du * s["weight"]).reshape(N, L, G, D)
    h = h.reshape(N, L, G, D)
    dx = r * (dh - dh.mean(dim=(1, 3), keepdim=True) - h * (dh * h).mean(dim=(1, 3), keepdim=True))
    out["dx"] = dx.reshape(N, L, C).to(s["x"].dtype)
    return out


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"delta": _plain_delta, "conv": _plain_conv, "gn_fwd": _plain_gn_fwd, "gn_bwd": _plain_gn_bwd}[
            c["op"]](s, c)
    import gated_delta_rule_157_b200 as kda
    if c["op"] == "delta":
        o = kda.kda_packed_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], cu_seqlens=s["cu"],
                               slots=s["slots"], fresh=s["fresh"], max_seqlen=s["max_len"], A_log=s["A_log"],
                               dt_bias=s["dt_bias"], scale=s["scale"],
                               gate_in_kernel=False if c["gate"] == "none" else c["gate"],
                               g_per_head=c["per_head"], o=s["o"])
        return {"o": o, "pool": s["pool"]}
    if c["op"] == "conv":
        y = kda.kda_packed_conv(s["x"], s["w"], s["pool"], s["bias"], cu_seqlens=s["cu"], slots=s["slots"],
                                fresh=s["fresh"], head_dim=c["head_dim"], silu=c["silu"], y=s["y"])
        return {"y": y, "pool": s["pool"]}
    if c["op"] == "gn_fwd":
        y, mean, rstd = kda.kda_group_norm_fwd(s["x"], c["G"], s["weight"], s["bias"], s["gate"], act=c["act"])
        return {"y": y, "mean": mean, "rstd": rstd}
    d = kda.kda_group_norm_bwd(s["dy"], s["x"], c["G"], s["mean"], s["rstd"], s["weight"], s["bias"], s["gate"],
                               act=c["act"])
    return {n: t for n, t in d.items() if t is not None}


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "delta":
        T, H, HV, Dk, Dv = c["tokens"], c["H"], c["HV"], c["Dk"], c["Dv"]
        gk = 1 if c["per_head"] else Dk
        state = HV * Dk * Dv * 4
        return {"bytes": T * (2 * H * Dk + 2 * HV * Dv + HV * gk + HV) * es + (2 * c["n"] - c["fresh"]) * state,
                "flops": 6 * T * HV * Dk * Dv}
    if c["op"] == "conv":
        T, C, K, n = c["tokens"], c["C"], c["K"], c["n"]
        return {"bytes": 2 * T * C * es + (2 * n - c["fresh"]) * (K - 1) * C * es + C * (K + 1) * 4,
                "flops": T * C * (2 * K + 6)}
    n = c["N"] * c["L"] * c["C"]
    stats = 8 * c["N"] * c["G"] + 8 * c["C"]
    if c["op"] == "gn_fwd":
        return {"bytes": n * es * (3 if c["gate"] else 2) + stats, "flops": 12 * n}
    return {"bytes": n * es * (5 if c["gate"] else 3) + stats + 8 * c["C"], "flops": 25 * n}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "delta":
        return _exact_delta(s, c)
    if c["op"] == "conv":
        return _exact_conv(s, c)
    return _exact_gn(s, c)


def _exact_delta(s, c):
    """Token by token, every live sequence that still has one."""
    d = lambda t: None if t is None else t.double()       # noqa: E731
    lens, cu, slots, fresh, _ = _packing(c)
    pool, o = s["pool"].double(), torch.zeros_like(s["o"], dtype=torch.float64)
    group = c["HV"] // c["H"]
    order = sorted((i for i in range(len(lens)) if slots[i] >= 0), key=lambda i: -lens[i])
    slot = torch.tensor([slots[i] for i in order], device=DEV)
    keep = torch.tensor([0.0 if fresh[i] else 1.0 for i in order], device=DEV, dtype=torch.float64)
    start = torch.tensor([cu[i] for i in order], device=DEV)
    S = pool[slot] * keep[:, None, None, None]
    A, b = d(s["A_log"]), d(s["dt_bias"])
    active = len(order)
    for t in range(max(lens)):
        while active and lens[order[active - 1]] <= t:
            active -= 1
        if not active:
            break
        r = start[:active] + t
        q, k = s["q"][r].double(), s["k"][r].double()
        q = q * (q.square().sum(-1, keepdim=True) + 1e-6).rsqrt() * s["scale"]
        k = k * (k.square().sum(-1, keepdim=True) + 1e-6).rsqrt()
        q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
        g = s["g"][r].double()
        if c["gate"] == "bounded":
            e = A.exp() if c["per_head"] else A.exp()[:, None]
            g = -5.0 * torch.sigmoid(e * (g + b))
        elif c["gate"] == "softplus":
            e = A.exp() if c["per_head"] else A.exp()[:, None]
            g = -e * torch.logaddexp(g + b, torch.zeros((), device=DEV, dtype=torch.float64))
        a = g.exp()[..., None, None] if c["per_head"] else g.exp()[..., None]
        beta = torch.sigmoid(s["beta"][r].double())[..., None]
        now = S[:active].mul_(a)
        err = s["v"][r].double() - torch.einsum("nhkv,nhk->nhv", now, k)
        now.add_(torch.einsum("nhk,nhv->nhkv", k, beta * err))
        o[r] = torch.einsum("nhkv,nhk->nhv", now, q)
    pool[slot] = S
    return {"o": o, "pool": pool}


def _exact_conv(s, c):
    """Each sequence behind its own window."""
    lens, cu, slots, fresh, _ = _packing(c)
    K = c["K"]
    y, pool = torch.zeros_like(s["y"], dtype=torch.float64), s["pool"].double()
    w = s["w"].double()
    for i, n in enumerate(lens):
        if slots[i] < 0 or n == 0:
            continue
        before = torch.zeros_like(pool[slots[i]]) if fresh[i] else pool[slots[i]]
        row = torch.cat([before, s["x"][cu[i]:cu[i + 1]].double()])
        u = (row.unfold(0, K, 1) * w).sum(-1) + s["bias"].double()
        u = u * torch.sigmoid(u) if c["silu"] else u
        if c["head_dim"]:
            h = u.view(n, -1, c["head_dim"])
            u = (h * (h.square().sum(-1, keepdim=True) + 1e-6).rsqrt()).view(n, -1)
        y[cu[i]:cu[i + 1]] = u
        pool[slots[i]] = row[n:]
    return {"y": y, "pool": pool}


def _exact_gn(s, c):
    """The forward formula in 64 bits, the gradient by differentiating it."""
    N, L, C, G = c["N"], c["L"], c["C"], c["G"]
    back = c["op"] == "gn_bwd"
    leaf = lambda t: t.double().requires_grad_(back)      # noqa: E731
    x, w, b = leaf(s["x"]), leaf(s["weight"]), leaf(s["bias"])
    z = leaf(s["gate"]) if c["gate"] else None
    f = {"none": lambda u: u, "silu": lambda u: u * torch.sigmoid(u), "sigmoid": torch.sigmoid}[c["act"]]
    by_group = x.view(N, L, G, C // G).transpose(1, 2).reshape(N, G, -1)
    mean = by_group.mean(-1, keepdim=True)
    rstd = (by_group - mean).square().mean(-1, keepdim=True).add(1e-5).rsqrt()
    h = ((by_group - mean) * rstd).view(N, G, L, C // G).transpose(1, 2).reshape(N, L, C)
    u = h * w + b
    y = u * f(z) if c["gate"] else f(u)
    if not back:
        return {"y": y, "mean": mean.view(N, G), "rstd": rstd.view(N, G)}
    got = torch.autograd.grad(y, [x, w, b] + ([z] if c["gate"] else []), s["dy"].double())
    return dict(zip(["dx", "dweight", "dbias", "dgate"], got))
