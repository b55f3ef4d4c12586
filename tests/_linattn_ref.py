"""Plain 64-bit references of linear attention with decays, of the grouped norm and of a serving batch's maps.

Linear attention steps the recurrence token by token, forward and backward, as the
formulas are written.  Its bounds are those of _layer_ref.check: half a step of the
output's type relative to the value, and 2^-15 of the sum of the magnitudes of its
terms (the same functions on magnitudes) for fp32 sums, operands in bf16 parts and decays.
"""
import numpy as np


def linattn_rows(q, k, v, g, scale, h0):
    """One sequence: q (n, H, dk), k (n, G, dk), v (n, G, dv), g (H,), h0 (H, dv, dk).  Returns y and the last state."""
    rep = q.shape[1] // k.shape[1]
    a, H, y = np.exp(g)[:, None, None], h0.copy(), np.zeros((q.shape[0], q.shape[1], v.shape[2]))
    for t in range(q.shape[0]):
        kt, vt = np.repeat(k[t], rep, 0), np.repeat(v[t], rep, 0)
        H = a * H + vt[:, :, None] * kt[:, None, :]
        y[t] = scale * np.einsum("hpn,hn->hp", H, q[t])
    return y, H


def linattn_grads(q, k, v, g, scale, h0, dy, dfinal):
    """Gradients of sum(dy y) + sum(dfinal H_last): dq, dk, dv, dh0."""
    n, H, dk = q.shape
    G, rep = k.shape[1], H // k.shape[1]
    a = np.exp(g)[:, None, None]
    states, st = [], h0
    for t in range(n):
        st = a * st + np.repeat(v[t], rep, 0)[:, :, None] * np.repeat(k[t], rep, 0)[:, None, :]
        states.append(st)
    D, dq, dkk, dv = dfinal.copy(), np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for t in range(n - 1, -1, -1):
        D = D + scale * dy[t][:, :, None] * q[t][:, None, :]
        dq[t] = scale * np.einsum("hpn,hp->hn", states[t], dy[t])
        dkk[t] = np.einsum("hpn,hp->hn", D, np.repeat(v[t], rep, 0)).reshape(G, rep, dk).sum(1)
        dv[t] = np.einsum("hpn,hn->hp", D, np.repeat(k[t], rep, 0)).reshape(G, rep, v.shape[2]).sum(1)
        D = a * D
    return dq, dkk, dv, D


def _silu(x):
    return x / (1.0 + np.exp(-x))


def norm(x, w, b, z, groups, eps, center, mode):
    """y, and the magnitude that its error is measured by.

    A group's mean is a tree of fp32 sums: off by up to some 20 * 2^-24 of mean|u|; its deviation by
    20 * 2^-24 of itself; o by those of ((|u| + mean|u|) rstd) |w| + |b|, and what follows is a product."""
    rows, C = x.shape
    u = x * _silu(z) if mode == "gate_first" else x
    u = u.reshape(rows, groups, -1)
    m = u.mean(2, keepdims=True) if center else 0.0 * u[:, :, :1]
    r = 1.0 / np.sqrt(((u - m) ** 2).mean(2, keepdims=True) + eps)
    n = ((u - m) * r).reshape(rows, C)
    big = ((np.abs(u) + np.abs(u).mean(2, keepdims=True)) * r).reshape(rows, C)
    o, mag = n * w + b, big * np.abs(w) + np.abs(b)
    if mode == "silu":
        return _silu(o), 1.2 * mag                     # SiLU's slope is at most 1.1
    if mode == "gate":
        return o * _silu(z), mag * np.abs(_silu(z))
    return o, mag


def norm_grads(x, w, b, z, dy, groups, eps, center, mode):
    """Gradients and their magnitudes, by name."""
    rows, C = x.shape
    sig = 1.0 / (1.0 + np.exp(-z)) if z is not None else None
    ds = sig * (1.0 + z * (1.0 - sig)) if z is not None else None
    dm = sig * (1.0 + np.abs(z)) if z is not None else None            # of the terms of ds
    u = x * z * sig if mode == "gate_first" else x
    g3 = lambda a: a.reshape(rows, groups, -1)
    flat = lambda a: a.reshape(rows, C)
    u = g3(u)
    m = u.mean(2, keepdims=True) if center else 0.0 * u[:, :, :1]
    r = 1.0 / np.sqrt(((u - m) ** 2).mean(2, keepdims=True) + eps)
    n = (u - m) * r
    big = (np.abs(u) + np.abs(u).mean(2, keepdims=True)) * r
    o, om = flat(n) * w + b, flat(big) * np.abs(w) + np.abs(b)
    out = {}
    if mode == "silu":
        so = 1.0 / (1.0 + np.exp(-o))
        do = dy * so * (1.0 + o * (1.0 - so))
        dom = np.abs(dy) * (1.0 + om)                  # the slope's slope is at most 1/2
    elif mode == "gate":
        do, dom = dy * z * sig, np.abs(dy * z * sig)
        out["dz"] = dy * o * ds, np.abs(dy) * om * dm
    else:
        do, dom = dy, np.abs(dy)
    out["dweight"] = (do * flat(n)).sum(0), (dom * flat(big)).sum(0)
    out["dbias"] = do.sum(0), dom.sum(0)
    dn, dnm = g3(do * w), g3(dom * np.abs(w))
    mean = lambda a: a.mean(2, keepdims=True)
    du = r * (dn - (mean(dn) if center else 0.0) - n * mean(dn * n))
    dum = r * (dnm + mean(dnm) + big * mean(dnm * big))
    du, dum = flat(du), flat(dum)
    if mode == "gate_first":
        out["dz"] = du * x * ds, dum * np.abs(x) * dm
        du, dum = du * z * sig, dum * np.abs(z * sig)
    out["dx"] = du, dum
    return out


def pack(new, slots, seen, tokens):
    """The maps of a batch, a request after the other."""
    n = len(new)
    out = dict(rows=[-1] * n, taken=[0] * n, step_slots=[], cu_seqlens=[], prompt_slots=[], has_state=[], row_request=[],
               row_position=[])
    at = 0
    for prompts in (False, True):
        for i in range(n):
            step = new[i] == 1 and seen[i] > 0
            if slots[i] < 0 or new[i] <= 0 or step == prompts or at >= tokens:
                continue
            take = min(new[i], tokens - at)
            out["rows"][i], out["taken"][i] = at, take
            if step:
                out["step_slots"].append(slots[i])
            else:
                out["cu_seqlens"].append(at)
                out["prompt_slots"].append(slots[i])
                out["has_state"].append(int(seen[i] > 0))
            out["row_request"] += [i] * take
            out["row_position"] += range(max(seen[i], 0), max(seen[i], 0) + take)
            at += take
    for key, fill, size in (("step_slots", -1, n), ("cu_seqlens", at, n + 1), ("prompt_slots", -1, n), ("has_state", 0, n),
                            ("row_request", -1, tokens), ("row_position", -1, tokens)):
        out[key] += [fill] * (size - len(out[key]))
    return {k: np.asarray(v, dtype=np.int64) for k, v in out.items()}
