"""FP64 oracle of the packed operators and of group norm -- TEST INFRASTRUCTURE.

  * ``packed_fwd``  -- every live sequence of a packed batch through the C
    oracle's recurrence, the gate applied by ``gates``.
  * ``packed_conv`` -- every live sequence through ``layer``'s prologue behind
    its slot's window.
  * ``group_norm`` / ``group_norm_backward`` -- the formulas in NumPy.

A sequence is live if it has rows, its bounds lie in [0, T], its slot is in the
pool and no earlier sequence with rows names that slot.
"""
import numpy as np

import oracle

from . import gates, layer


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def live(cu, slots, T, P, n):
    """[(sequence, begin, end, slot)] of the live sequences, and whether any is reported."""
    out, report, seen = [], False, set()
    for s in range(n):
        b, e = (s, s + 1) if cu is None else (int(cu[s]), int(cu[s + 1]))
        slot = s if slots is None else int(slots[s])
        bad = b < 0 or e < b or e > T or slot >= P
        repeat = slots is not None and slot >= 0 and slot in seen
        if e != b:
            seen.add(slot)
        report |= bad or (repeat and e > b)
        if not bad and not repeat and slot >= 0 and e > b:
            out.append((s, b, e, slot))
    return out, report


def log_decay(g, A_log, dt_bias, gate, per_head, Dk, g_min=-5.0):
    """[T, HV, Dk] from the gate input (gate: False, "bounded" or "softplus")."""
    z = _f64(g)[..., None] if per_head else _f64(g)
    if gate:
        b = None if dt_bias is None else (_f64(dt_bias)[:, None] if per_head else _f64(dt_bias))
        b = np.zeros(z.shape[-2:]) if b is None else b
        z = gates.bounded_gate(z, A_log, b, g_min) if gate == "bounded" else gates.softplus_gate(z, A_log, b)
    return np.ascontiguousarray(np.broadcast_to(z, z.shape[:-1] + (Dk,)))


def packed_fwd(q, k, v, g, beta, pool, o, *, cu=None, slots=None, fresh=None, A_log=None, dt_bias=None,
               gate="bounded", per_head=False, scale=1.0, l2norm=True, beta_sigmoid=True, g_min=-5.0, l2_eps=1e-6):
    """Returns (o, pool) in float64: copies of the given o and pool with the live
    sequences' rows and slots replaced."""
    T, Dk = q.shape[0], q.shape[2]
    n = T if cu is None else len(cu) - 1
    gl = log_decay(g, A_log, dt_bias, gate, per_head, Dk, g_min)
    o, pool = _f64(o).copy(), _f64(pool).copy()
    for s, b, e, slot in live(cu, slots, T, len(pool), n)[0]:
        S0 = None if fresh is not None and fresh[s] else pool[slot][None]
        r = oracle.kda_fwd(q[None, b:e], k[None, b:e], v[None, b:e], gl[None, b:e], beta[None, b:e], S0=S0,
                           scale=scale, qk_l2norm=l2norm, beta_sigmoid=beta_sigmoid, gate_in=False, l2_eps=l2_eps)
        o[b:e], pool[slot] = r["o"][0], r["S_T"][0]
    return o, pool


def packed_conv(x, w, pool, y, bias=None, *, cu=None, slots=None, fresh=None, head_dim=0, silu=True, l2_eps=1e-6):
    """Returns (y, pool) in float64, as packed_fwd."""
    x, T, K = _f64(x), x.shape[0], w.shape[1]
    n = T if cu is None else len(cu) - 1
    y, pool = _f64(y).copy(), _f64(pool).copy()
    for s, b, e, slot in live(cu, slots, T, len(pool), n)[0]:
        before = np.zeros_like(pool[slot]) if fresh is not None and fresh[s] else pool[slot].copy()
        u, after = layer.short_conv(x[None, b:e], w, bias, before[None])
        u = u[0]
        if silu:
            u = u / (1 + np.exp(-u))
        if head_dim:
            h = u.reshape(e - b, -1, head_dim)
            u = (h / np.sqrt((h * h).sum(-1, keepdims=True) + l2_eps)).reshape(e - b, -1)
        y[b:e], pool[slot] = u, after[0]
    return y, pool


def _act(u, act):
    p = 1 / (1 + np.exp(-u))
    if act == "none":
        return u, np.ones_like(u)
    return (u * p, p * (1 + u * (1 - p))) if act == "silu" else (p, p * (1 - p))


def _normalised(x, G, eps):
    N, L, C = x.shape
    xg = _f64(x).reshape(N, L, G, C // G)
    mean = xg.mean(axis=(1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean(axis=(1, 3))
    rstd = 1 / np.sqrt(var + eps)
    return (xg - mean[:, None, :, None]) * rstd[:, None, :, None], mean, rstd


def group_norm(x, G, weight=None, bias=None, gate=None, act="none", eps=1e-5):
    """Returns y [N, L, C], mean and rstd [N, G]."""
    h, mean, rstd = _normalised(x, G, eps)
    u = h.reshape(x.shape)
    u = u * (1.0 if weight is None else _f64(weight)) + (0.0 if bias is None else _f64(bias))
    y = u * _act(_f64(gate), act)[0] if gate is not None else _act(u, act)[0]
    return y, mean, rstd


def group_norm_backward(dy, x, G, weight=None, bias=None, gate=None, act="none", eps=1e-5):
    """Gradient of <dy, y>: dict dx, dgate, dweight, dbias, and l1, the sums of
    the magnitudes of the terms of dweight and dbias."""
    N, L, C = x.shape
    hg, _, rstd = _normalised(x, G, eps)
    h, dy = hg.reshape(x.shape), _f64(dy)
    w = np.ones(C) if weight is None else _f64(weight)
    u = h * w + (0.0 if bias is None else _f64(bias))
    out = {}
    if gate is not None:
        f, d = _act(_f64(gate), act)
        du, out["dgate"] = dy * f, dy * u * d
    else:
        du = dy * _act(u, act)[1]
    out["dweight"], out["dbias"] = (du * h).sum((0, 1)), du.sum((0, 1))
    out["l1"] = np.maximum(np.abs(du * h).sum((0, 1)), np.abs(du).sum((0, 1)))
    dh = (du * w).reshape(hg.shape)
    m1, m2 = dh.mean(axis=(1, 3), keepdims=True), (dh * hg).mean(axis=(1, 3), keepdims=True)
    out["dx"] = (rstd[:, None, :, None] * (dh - m1 - hg * m2)).reshape(x.shape)
    return out
