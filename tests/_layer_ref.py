"""Plain 64-bit references of a Mamba-2 layer's serving and gradient operators, and their error bounds.

The scans come from the C oracle (one call per sequence); the gradients step the
recurrence backwards as the formulas are written.  `abs` runs of the same functions
(every input replaced by its magnitude) give the sum of the magnitudes of an output's
terms, the measure of the bounds below.

Bounds.  An output is a sum of products; its error is at most
  half a step of the output's type, relative to the value, plus
  2^-15 of the sum of its terms' magnitudes:
    2^-16 for fp32 sums of up to 256 terms one after the other (n * 2^-24),
    2^-17 for operands in two bf16 parts (2^-18 of each of two),
    2^-17 for the decays (an exponent of size up to 16, beyond which a weight is
    below 2^-23 of its neighbour, rounded to 2^-24 of it, and a few roundings more).
"""
import numpy as np
import torch

import oracle
from _util import f64

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SUM = 2.0 ** -15
# softplus, SiLU and their derivatives on the fp32 pipeline: a few units of 2^-24 each
ELEMENT = 2.0 ** -20


def check(got, ref, mag, name, terms=SUM):
    """|got - ref| <= half a step of got's type * |ref| + terms * mag, element by element."""
    ref, mag = np.asarray(ref, dtype=np.float64), np.asarray(mag, dtype=np.float64)
    half = HALF[got.dtype]
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), "%s: non-finite values" % name
    # below a type's normal range values step by a fixed amount (fp16: half of it 2^-25); bf16 and fp32 end at
    # 2^-126, below which a factor (sigmoid(-100), say) is 0 in fp32 arithmetic: times factors of up to 2^16, 2^-110
    tiny = 2.0 ** -25 if half == 2.0 ** -11 else 2.0 ** -110
    over = np.abs(got - ref) - (half * np.abs(ref) + terms * mag + tiny)
    worst = float(over.max()) if over.size else 0.0
    scale = float(np.max(np.abs(got - ref) / (half * np.abs(ref) + terms * mag + tiny + 1e-300))) if over.size else 0.0
    print("  %-12s error / bound %.3f" % (name, scale), flush=True)
    assert worst <= 0.0, (name, scale)


def silu(v):
    return v / (1.0 + np.exp(-v))


def softplus(v):
    return np.logaddexp(v, 0.0)


# ---- convolution of packed prompts ------------------------------------------------


def conv_rows(x, w, bias, win, use_silu=True):
    """One sequence: x (n, D), win (D, W-1).  Returns (out, the magnitudes of its terms, the window behind it)."""
    W = w.shape[1]
    rows = np.concatenate([win.T, x])
    n = x.shape[0]
    pre = np.zeros((n, x.shape[1])) + (0.0 if bias is None else bias)
    mag = np.zeros_like(pre) + (0.0 if bias is None else np.abs(bias))
    for k in range(W):
        pre = pre + rows[k:k + n] * w[:, k]
        mag = mag + np.abs(rows[k:k + n] * w[:, k])
    out = silu(pre) if use_silu else pre
    return out, mag, rows[rows.shape[0] - (W - 1):].T if W > 1 else win


# ---- scan of packed prompts ---------------------------------------------------------


def ssd_rows(x, dt, A, Bm, Cm, D, z, dt_bias, h0):
    """One sequence (no batch axis) through the oracle: y, its terms' magnitudes, state, its magnitudes."""
    b = lambda a: None if a is None else a[None]
    if x.shape[0] == 0:
        return x, np.abs(x), h0, np.abs(h0)
    y, fin = oracle.ssd_fwd(b(x), b(dt), A, b(Bm), b(Cm), D=D, z=b(z), dt_bias=dt_bias, h0=b(h0))
    m = lambda a: None if a is None else np.abs(a)
    ym, fm = oracle.ssd_fwd(b(m(x)), b(dt), A, b(m(Bm)), b(m(Cm)), D=m(D), dt_bias=dt_bias, h0=b(m(h0)))
    if z is not None:
        ym = ym * np.abs(silu(z))
    return y[0], ym[0], fin[0], fm[0]


# ---- gradients of the scan --------------------------------------------------------------


def _ssd_grad_core(x, delta, loga, Bm, Cm, g, keep, h0, dfinal):
    """Of the recurrence H_t = exp(loga_t) keep_t H_{t-1} + delta_t x_t B_t^T, y0_t = H_t C_t, with the gradient g
    of y0: y0, G_t B_t, da_t, dB, dC (per head), dh0."""
    Bsz, L, H, P = x.shape
    N = Bm.shape[3]
    Hs = np.zeros((L + 1, Bsz, H, P, N))
    if h0 is not None:
        Hs[0] = h0
    a = np.exp(loga) * keep[:, :, None]
    for t in range(L):
        Hs[t + 1] = a[:, t, :, None, None] * Hs[t] + (delta[:, t, :, None] * x[:, t])[..., None] * Bm[:, t, :, None, :]
    y0 = np.stack([(Hs[t + 1] * Cm[:, t, :, None, :]).sum(3) for t in range(L)], 1)
    G = np.zeros((Bsz, H, P, N)) if dfinal is None else dfinal.copy()
    gB, da, dB, dC = np.zeros_like(x), np.zeros_like(delta), np.zeros_like(Bm), np.zeros_like(Cm)
    for t in range(L - 1, -1, -1):
        dC[:, t] = (Hs[t + 1] * g[:, t][..., None]).sum(2)
        G = G + g[:, t][..., None] * Cm[:, t, :, None, :]
        gB[:, t] = (G * Bm[:, t, :, None, :]).sum(3)
        dB[:, t] = delta[:, t, :, None] * (G * x[:, t][..., None]).sum(2)
        da[:, t] = a[:, t] * (G * Hs[t]).sum((2, 3))
        G = a[:, t, :, None, None] * G
    return y0, gB, da, dB, dC, G


def ssd_grad(q, use_softplus=True):
    """q: dict of 64-bit x, dt, A, Bm, Cm, dy and optional D, z, dt_bias, seq_idx, h0, dfinal.  Returns the gradients
    and the magnitudes of their terms."""
    x, dt, A, Bm, Cm, dy = (q[k] for k in ("x", "dt", "A", "Bm", "Cm", "dy"))
    D, z, dt_bias, ids, h0, dfinal = (q.get(k) for k in ("D", "z", "dt_bias", "seq_idx", "h0", "dfinal"))
    Bsz, L, H, P = x.shape
    Gn = Bm.shape[2]
    rep = H // Gn
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    delta = softplus(raw) if use_softplus else raw
    slope = 1.0 / (1.0 + np.exp(-raw)) if use_softplus else np.ones_like(raw)
    keep = np.ones((Bsz, L))
    if ids is not None:
        keep[:, 1:] = ids[:, 1:] == ids[:, :-1]
    Dv = np.zeros(H) if D is None else D
    sz = None if z is None else silu(z)
    m = lambda a: None if a is None else np.abs(a)

    def run(x, Bm, Cm, g, h0, dfinal, Dv, Aw, ry):
        Bh, Ch = np.repeat(Bm, rep, 2), np.repeat(Cm, rep, 2)
        y0, gB, da, dB, dC, dh0 = _ssd_grad_core(x, delta, delta * A, Bh, Ch, g, keep, h0, dfinal)
        sum_heads = lambda v: v.reshape(Bsz, L, Gn, rep, -1).sum(3)
        dd = (x * gB).sum(3) + Aw * da
        out = dict(dx=delta[..., None] * gB + Dv[:, None] * g, dB=sum_heads(dB), dC=sum_heads(dC),
                   dA=(delta * da).sum((0, 1)), ddt=dd * slope, ddt_bias=(dd * slope).sum((0, 1)),
                   dD=(g * x).sum((0, 1, 3)), dh0=dh0)
        if ry is not None:
            out["dz"] = ry * (y0 + Dv[:, None] * x)
        return out

    g = dy if z is None else dy * sz
    ry = None
    if z is not None:
        sg = 1.0 / (1.0 + np.exp(-z))
        ry = dy * sg * (1.0 + z * (1.0 - sg))
    ref = run(x, Bm, Cm, g, h0, dfinal, Dv, A, ry)
    mag = run(m(x), m(Bm), m(Cm), m(g), m(h0), m(dfinal), m(Dv), m(A), m(ry))
    return ref, mag


# ---- gradients of the convolution ----------------------------------------------------------


def conv_grad(x, w, dout, bias=None, use_silu=True, ids=None, init=None, dfinal=None):
    """Returns (gradients, their terms' magnitudes): dx, dw, dbias, dconv_init."""
    Bsz, D, L = x.shape
    W = w.shape[1]
    win = np.zeros((Bsz, D, W - 1)) if init is None else init
    wide = np.concatenate([win, x], 2)
    ids = np.zeros((Bsz, L), dtype=np.int64) if ids is None else ids
    idw = np.concatenate([np.repeat(ids[:, :1], W - 1, 1), ids], 1)

    def terms(k):  # inputs k - (W-1) steps away, 0 across documents
        same = (idw[:, k:k + L] == ids)[:, None, :]
        return wide[:, :, k:k + L] * same, same

    pre = np.zeros_like(x) + (0.0 if bias is None else bias[None, :, None])
    pm = np.abs(pre)
    for k in range(W):
        pre = pre + w[None, :, k, None] * terms(k)[0]
        pm = pm + np.abs(w[None, :, k, None] * terms(k)[0])
    if use_silu:
        s = 1.0 / (1.0 + np.exp(-pre))
        dpre = dout * s * (1.0 + pre * (1.0 - s))
    else:
        dpre = dout
    # an error of pre moves SiLU's slope by at most half of it
    dm = np.abs(dout) * (1.2 + (pm if use_silu else 0.0))

    def back(d, wt, fin):
        dw = np.stack([(d * (np.abs(terms(k)[0]) if wt is not w else terms(k)[0])).sum((0, 2)) for k in range(W)], 1)
        dwide = np.zeros_like(wide)
        for k in range(W):
            dwide[:, :, k:k + L] += wt[None, :, k, None] * d * terms(k)[1]
        if fin is not None:
            dwide[:, :, L:] += fin * (idw[:, None, L:] == ids[:, None, -1:])
        return dict(dx=dwide[:, :, W - 1:], dw=dw, dbias=d.sum((0, 2)), dconv_init=dwide[:, :, :W - 1])

    return back(dpre, w, dfinal), back(dm, np.abs(w), None if dfinal is None else np.abs(dfinal))
