"""The 64-bit gradient references of the layer tests, pinned by finite differences of the oracle's forwards (CPU)."""
import numpy as np
import pytest

import _layer_ref as ref
import oracle


def _ssd_problem(seed, docs, state, gate, L=13, Bsz=2, H=4, G=2, P=3, N=4):
    r = np.random.default_rng(seed)
    q = dict(x=r.standard_normal((Bsz, L, H, P)), dt=r.standard_normal((Bsz, L, H)) * 0.5, A=-r.uniform(0.5, 2.0, H),
             Bm=r.standard_normal((Bsz, L, G, N)), Cm=r.standard_normal((Bsz, L, G, N)),
             dy=r.standard_normal((Bsz, L, H, P)), D=r.standard_normal(H), dt_bias=r.standard_normal(H) * 0.1)
    if gate:
        q["z"] = r.standard_normal((Bsz, L, H, P))
    if docs:
        q["seq_idx"] = np.cumsum(r.random((Bsz, L)) < 0.25, 1)
    if state:
        q["h0"], q["dfinal"] = r.standard_normal((Bsz, H, P, N)), r.standard_normal((Bsz, H, P, N))
    return q, r


def _loss(q):
    y, fin = oracle.ssd_fwd(q["x"], q["dt"], q["A"], q["Bm"], q["Cm"], D=q["D"], z=q.get("z"), dt_bias=q["dt_bias"],
                            seq_idx=q.get("seq_idx"), h0=q.get("h0"))
    return (y * q["dy"]).sum() + (0.0 if q.get("dfinal") is None else (fin * q["dfinal"]).sum())


@pytest.mark.parametrize("docs,state,gate", [(False, False, False), (True, True, True), (True, False, False),
                                             (False, True, True)])
def test_ssd_gradient_by_differences(docs, state, gate):
    q, r = _ssd_problem(3, docs, state, gate)
    g, mag = ref.ssd_grad(q)
    names = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", dt_bias="ddt_bias")
    if gate:
        names["z"] = "dz"
    if state:
        names["h0"] = "dh0"
    h = 1e-5
    for k, name in names.items():
        d = r.standard_normal(q[k].shape)
        up, down = dict(q), dict(q)
        up[k], down[k] = q[k] + h * d, q[k] - h * d
        fd = (_loss(up) - _loss(down)) / (2 * h)
        assert abs(fd - (g[name] * d).sum()) <= 1e-7 * (1.0 + np.abs(mag[name] * d).sum()), name
        assert np.all(np.abs(g[name]) <= mag[name] * (1 + 1e-12) + 1e-12), name


@pytest.mark.parametrize("W", [1, 2, 4])
@pytest.mark.parametrize("L", [1, 2, 9])
@pytest.mark.parametrize("docs", [False, True])
def test_conv_gradient_by_differences(W, L, docs):
    r = np.random.default_rng(5)
    Bsz, D, h = 2, 3, 1e-5
    x, w, b = r.standard_normal((Bsz, D, L)), r.standard_normal((D, W)), r.standard_normal(D)
    dout, init, dfin = (r.standard_normal(s) for s in ((Bsz, D, L), (Bsz, D, W - 1), (Bsz, D, W - 1)))
    ids = np.cumsum(r.random((Bsz, L)) < 0.3, 1).astype(np.int32) if docs else None

    def loss(x, w, b, init):
        out, fin = oracle.conv1d_fwd(x, w, b, seq_idx=ids, conv_init=init if W > 1 else None)
        return (out * dout).sum() + ((fin * dfin).sum() if W > 1 else 0.0)

    g, mag = ref.conv_grad(x, w, dout, bias=b, ids=ids, init=init, dfinal=dfin)
    args = dict(x=x, w=w, b=b, init=init)
    for k, name in (("x", "dx"), ("w", "dw"), ("b", "dbias"), ("init", "dconv_init")):
        if k == "init" and W == 1:
            continue
        d = r.standard_normal(args[k].shape)
        fd = (loss(**{**args, k: args[k] + h * d}) - loss(**{**args, k: args[k] - h * d})) / (2 * h)
        assert abs(fd - (g[name] * d).sum()) <= 1e-7 * (1.0 + np.abs(mag[name] * d).sum()), name


def test_chunk_places_stay_inside_for_any_offsets():
    """The chunk places of packed sequences (first row / Q + sequence, from clamped offsets): for ordered
    offsets every chunk has a place of its own, and for any content at all every place that a sequence
    can name, its chunks included, lies below tokens / Q + nseqs, the size of the workspace."""
    r = np.random.default_rng(0)
    for trial in range(3000):
        Q = (16, 256)[trial % 2]
        tokens, nseqs = int(r.integers(1, 5000)), int(r.integers(1, 40))
        ordered = trial % 3 != 0
        cu = r.integers(-50, tokens + 50, nseqs + 1)
        cu = np.sort(cu) if ordered else cu
        c = np.clip(cu, 0, tokens)
        places = set()
        for s in range(nseqs):
            n = max(0, int(c[s + 1] - c[s]))
            for k in range(-(-n // Q)):
                place = c[s] // Q + s + k
                assert 0 <= place < tokens // Q + nseqs
                if ordered:
                    assert place not in places
                    places.add(place)


def _find(cu, nseqs, tokens, Q, place):
    """The kernels' search of a place's sequence, step by step (64 probes a step)."""
    lo, n, rounds = 0, nseqs, 0
    while n > 1:
        rounds += 1
        assert rounds < 8
        step = (n + 63) // 64
        cnt = sum(min(max(int(cu[lo + k]), 0), tokens) // Q + lo + k <= place for k in range(0, min(n, 64 * step), step))
        cnt = max(cnt, 1)
        lo += (cnt - 1) * step
        n = min(n - (cnt - 1) * step, step)
        assert 0 <= lo < nseqs and n >= 1
    return lo


def test_chunk_search_finds_every_chunk():
    r = np.random.default_rng(1)
    for trial in range(60):
        Q = (16, 256)[trial % 2]
        nseqs = int(r.integers(1, 400))
        lens = r.integers(0, 4 * Q, nseqs) * (r.random(nseqs) < 0.8)
        cu = np.concatenate([[int(r.integers(0, 50))], lens]).cumsum()
        tokens = int(cu[-1]) + 7
        for s in range(nseqs):
            for k in range(-(-int(lens[s]) // Q)):
                assert _find(cu, nseqs, tokens, Q, int(cu[s]) // Q + s + k) == s
        wild = r.integers(-1000, 9000, nseqs + 1)
        for place in range(0, tokens // Q + nseqs, 7):
            _find(wild, nseqs, tokens, Q, place)
