"""GPU parity of linear attention with decays (prompts, tokens, training and its gradients) with the recurrences in
64 bits, one sequence at a time; bounds in _layer_ref.py."""
import numpy as np
import pytest
import torch

import _linattn_ref as ref
from _layer_ref import SUM, check
from _util import f64, say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _ss():
    from mamba_selective_scan_fwd_amd import ss
    ss.load_library()
    return ss


def _problem(lens, H, G, dk, dv, io, seed, lead=0, tail=0, g=None):
    """Operands on the host, q, k and v as columns of common rows, one of them an odd piece away from the next."""
    r = np.random.default_rng(seed)
    cu = np.concatenate([[lead], lens]).cumsum()
    T = int(cu[-1]) + tail
    t = lambda *s: torch.from_numpy(r.standard_normal(s))
    row = t(T, H * dk + 8 + G * (dk + dv)).to(DT[io])
    q, k, v = row[:, :H * dk], row[:, H * dk + 8:H * dk + 8 + G * dk], row[:, H * dk + 8 + G * dk:]
    S = len(lens)
    return dict(row=row, q=q.unflatten(1, (H, dk)), k=k.unflatten(1, (G, dk)), v=v.unflatten(1, (G, dv)),
                g=torch.from_numpy(-np.exp(r.uniform(np.log(2.0 ** -12), np.log(0.7), H))).float() if g is None else g,
                scale=dk ** -0.5, cu=torch.tensor(cu, dtype=torch.int32), T=T, dims=(H, G, dk, dv),
                state=(t(S + 2, H, dv, dk) * 0.5).float(), slots=torch.tensor(r.permutation(S + 2)[:S], dtype=torch.int32),
                has=torch.tensor(r.integers(0, 2, S), dtype=torch.int32), dy=t(T, H, dv).to(DT[io]),
                h0=(t(S, H, dv, dk) * 0.5).float(), df=(t(S, H, dv, dk) * 0.1).float())


def _dev(q):
    """On the device, q, k and v as slices of the rows again."""
    g = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in q.items()}
    H, G, dk, dv = q["dims"]
    g["q"] = g["row"][:, :H * dk].unflatten(1, (H, dk))
    g["k"] = g["row"][:, H * dk + 8:H * dk + 8 + G * dk].unflatten(1, (G, dk))
    g["v"] = g["row"][:, H * dk + 8 + G * dk:].unflatten(1, (G, dv))
    return g


def _rows(q, s):
    a, b = int(q["cu"][s]), int(q["cu"][s + 1])
    return a, b, {n: f64(q[n][a:b]) for n in ("q", "k", "v")}


def _magnitudes(p):
    return {k: np.abs(v) for k, v in p.items()}


def _forward(q, h0s):
    """y of every row (7 outside the sequences) and the last states, each with its terms' magnitudes."""
    H, G, dk, dv = q["dims"]
    y, ym = np.full((q["T"], H, dv), 7.0), np.zeros((q["T"], H, dv))
    last, lm = [], []
    g = f64(q["g"])
    for s, h0 in enumerate(h0s):
        a, b, p = _rows(q, s)
        y[a:b], L = ref.linattn_rows(**p, g=g, scale=q["scale"], h0=h0)
        ym[a:b], M = ref.linattn_rows(**_magnitudes(p), g=g, scale=abs(q["scale"]), h0=np.abs(h0))
        last.append(L)
        lm.append(M)
    return y, ym, np.array(last), np.array(lm)


def _check_prompts(q, got, state, slots=True, has=True):
    st = f64(q["state"])
    at = [int(q["slots"][s]) if slots else s for s in range(len(q["cu"]) - 1)]
    h0s = [st[i] if 0 <= i < len(st) and has and int(q["has"][s]) else np.zeros(st.shape[1:]) for s, i in enumerate(at)]
    y, ym, last, lm = _forward(q, h0s)
    check(got, y, ym, "y")
    new, nm = st.copy(), np.zeros(st.shape)
    for s, i in enumerate(at):
        if 0 <= i < len(st):
            new[i], nm[i] = last[s], lm[s]
    check(state, new, nm, "state")                       # other slots untouched: magnitude 0


LENS = [3, 0, 1, 64, 65, 63, 0, 130, 200, 7]


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,dk,dv", [(4, 4, 64, 64), (4, 2, 64, 128), (3, 1, 128, 64), (2, 2, 128, 128)])
def test_prompts(io, H, G, dk, dv):
    """Lengths around a chunk's, empty ones, rows of no sequence before and behind, which stay as they were."""
    ss = _ss()
    say("prompts %s %d %d %d %d" % (io, H, G, dk, dv))
    q = _problem(LENS, H, G, dk, dv, io, seed=H, lead=5, tail=9)
    g = _dev(q)
    y = torch.full((q["T"], H, dv), 7.0, dtype=DT[io], device="cuda")
    ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"], scale=q["scale"], slots=g["slots"],
                      has_state=g["has"], y=y)
    torch.cuda.synchronize()
    _check_prompts(q, y, g["state"])


@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_prompts_in_segments(io):
    """Few heads and long sequences among short ones: walked in segments, their states joined."""
    ss = _ss()
    q = _problem([700, 3, 0, 129, 1500, 128], 2, 1, 64, 128, io, seed=5, tail=2)
    g = _dev(q)
    g["has"][0] = q["has"][0] = 1
    y = torch.full((q["T"], 2, 128), 7.0, dtype=DT[io], device="cuda")
    ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"], slots=g["slots"], has_state=g["has"], y=y)
    torch.cuda.synchronize()
    _check_prompts(q, y, g["state"])


def test_prompts_options():
    """Default slots and scale, no states carried; slots outside the pool; contiguous operands give the same."""
    ss = _ss()
    q = _problem([5, 70, 1], 2, 2, 64, 64, "bf16", seed=9)
    g = _dev(q)
    y = ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"])
    torch.cuda.synchronize()
    _check_prompts(q, y, g["state"], slots=False, has=False)
    q["slots"] = torch.tensor([-1, 4, 99], dtype=torch.int32)
    g = _dev(q)
    other = g["state"].clone()
    y = ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"], slots=g["slots"], has_state=g["has"])
    z = ss.linattn_prompt(g["q"].contiguous(), g["k"].contiguous(), g["v"].contiguous(), g["g"], g["cu"], other,
                          slots=g["slots"], has_state=g["has"])
    torch.cuda.synchronize()
    _check_prompts(q, y, g["state"])
    assert torch.equal(y, z) and torch.equal(other, g["state"])


def test_many_sequences():
    ss = _ss()
    r = np.random.default_rng(2)
    q = _problem((r.integers(0, 4, 3000) * (r.random(3000) < 0.2)).tolist() + [90], 1, 1, 64, 64, "f16", seed=3, tail=2)
    g = _dev(q)
    y = torch.full((q["T"], 1, 64), 7.0, dtype=torch.float16, device="cuda")
    ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"], slots=g["slots"], has_state=g["has"], y=y)
    torch.cuda.synchronize()
    _check_prompts(q, y, g["state"])


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("decay", [0.0, -1e-6, -3.0, -200.0, -float("inf")])
def test_decays(io, decay):
    """No decay, hardly any, one that forgets within tokens, and no memory at all; in one walk and in segments."""
    ss = _ss()
    for lens in ([70, 1, 130], [600]):
        q = _problem(lens, 1, 1, 64, 64, io, seed=4, g=torch.tensor([decay]))
        g = _dev(q)
        y = ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"], slots=g["slots"], has_state=g["has"])
        torch.cuda.synchronize()
        _check_prompts(q, y, g["state"])


@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_states_hold_fp32(io):
    """The last states of long memories: three bf16 parts leave 2^-26 of a term and n fp32 sums of random sign about
    sqrt(n) 2^-25 of the whole; 3 * 2048 of them 2^-18.7, which a state in two parts (2^-17 of every term) exceeds."""
    ss = _ss()
    q = _problem([2048], 2, 2, 64, 64, io, seed=6, g=torch.tensor([-1e-3, -0.3]))
    g = _dev(q)
    ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"])
    torch.cuda.synchronize()
    _, _, last, _ = _forward(q, [np.zeros((2, 64, 64))])
    off = np.linalg.norm(f64(g["state"][0]) - last[0], axis=(1, 2)) / np.linalg.norm(last[0], axis=(1, 2))
    say("  states off by %s" % off)
    assert np.all(off <= 2.0 ** -18.7)


# ---- training -----------------------------------------------------------------------


def _train(q, B, L, cu, state, seed_scale=None):
    """Forward and gradients on the device as (B, L, ..) tensors."""
    ss = _ss()
    g = _dev(q)
    H, G, dk, dv = q["dims"]
    a = tuple(g[n].unflatten(0, (B, L)) for n in ("q", "k", "v")) + (g["g"],)
    kw = dict(scale=q["scale"], cu_seqlens=g["cu"] if cu else None, h0=g["h0"] if state else None)
    out = ss.linattn_fwd(*a, return_final_state=state, **kw)
    y, fin = out if state else (out, None)
    gr = ss.linattn_bwd(*a, g["dy"].unflatten(0, (B, L)), dfinal=g["df"] if state else None, want_dh0=state, **kw)
    torch.cuda.synchronize()
    return y.flatten(0, 1), fin, {n: v if n == "dh0" else v.flatten(0, 1) for n, v in gr.items()}


def _check_train(q, y, fin, gr, state):
    H, G, dk, dv = q["dims"]
    S = len(q["cu"]) - 1
    zero = np.zeros((S, H, dv, dk))
    h0, df = (f64(q["h0"]), f64(q["df"])) if state else (zero, zero)
    want, mag, last, lm = _forward(q, h0)
    inside = np.zeros(q["T"], dtype=bool)
    inside[int(q["cu"][0]):int(q["cu"][-1])] = True
    want[~inside] = 0.0
    check(y, want, mag, "y")
    grads = [np.zeros((q["T"], n, d)) for n, d in ((H, dk), (G, dk), (G, dv))] + [np.zeros((S, H, dv, dk))]
    mags = [np.zeros_like(x) for x in grads]
    for s in range(S):
        a, b, p = _rows(q, s)
        dy = f64(q["dy"][a:b])
        one = ref.linattn_grads(**p, g=f64(q["g"]), scale=q["scale"], h0=h0[s], dy=dy, dfinal=df[s])
        big = ref.linattn_grads(**_magnitudes(p), g=f64(q["g"]), scale=q["scale"], h0=np.abs(h0[s]), dy=np.abs(dy),
                                dfinal=np.abs(df[s]))
        for i in range(4):
            at = slice(a, b) if i < 3 else s
            grads[i][at], mags[i][at] = one[i], big[i]
    for i, n in enumerate(("dq", "dk", "dv", "dh0") if state else ("dq", "dk", "dv")):
        check(gr[n], grads[i], mags[i], n)
    if state:
        check(fin, last, lm, "final")


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,dk,dv", [(4, 4, 64, 64), (4, 2, 64, 128), (3, 1, 128, 64), (2, 2, 128, 128)])
@pytest.mark.parametrize("state", [False, True])
def test_training_rows(io, H, G, dk, dv, state):
    B, L = 3, 150
    q = _problem([L] * B, H, G, dk, dv, io, seed=20 + H)
    _check_train(q, *_train(q, B, L, False, state), state)


@pytest.mark.parametrize("io,G,dk,dv", [("f16", 2, 64, 128), ("bf16", 4, 128, 128)])
def test_training_walks_beyond_a_round(io, G, dk, dv):
    """22 rows of 4 heads have 264 walks of gradients: 256 run whole beside the last 8, those of the last row, in pieces."""
    B, L = 22, 1537
    q = _problem([L] * B, 4, G, dk, dv, io, seed=50)
    y, fin, gr = _train(q, B, L, False, True)
    t = (B - 2) * L
    last = dict(q, cu=q["cu"][:3], T=2 * L, h0=q["h0"][B - 2:], df=q["df"][B - 2:], **{n: q[n][t:] for n in ("q", "k", "v", "dy")})
    _check_train(last, y[t:], fin[B - 2:], {n: v[B - 2:] if n == "dh0" else v[t:] for n, v in gr.items()}, True)


@pytest.mark.parametrize("L", [1, 2, 63, 64, 65, 129, 500])
def test_training_lengths(L):
    q = _problem([L] * 2, 2, 1, 64, 64, "bf16", seed=L)
    _check_train(q, *_train(q, 2, L, False, True), True)


@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_training_documents(io):
    """Documents across rows of the batch, empty ones, and tokens of none: outputs and gradients of zero there."""
    q = _problem([40, 0, 200, 1, 64, 90], 2, 1, 128, 128, io, seed=31, lead=3, tail=402)
    _check_train(q, *_train(q, 2, 400, True, True), True)
    q = _problem([700, 300, 9], 2, 2, 64, 128, io, seed=32, lead=1, tail=10)   # in segments
    _check_train(q, *_train(q, 1, 1020, True, True), True)


@pytest.mark.parametrize("decay", [0.0, -3.0, -200.0])
def test_gradients_of_decays(decay):
    q = _problem([150, 70], 1, 1, 64, 64, "bf16", seed=33, g=torch.tensor([decay]))
    _check_train(q, *_train(q, 1, 220, True, True), True)


def test_linattn_fn():
    """autograd reaches q, k, v, h0 through both outputs, views of a projection among them; log_decay is refused."""
    ss = _ss()
    q = _problem([70, 70], 2, 1, 64, 64, "bf16", seed=40)
    g = _dev(q)
    row = g["row"].detach().clone().requires_grad_()
    h0 = g["h0"].clone().requires_grad_()
    cols = row.unflatten(0, (2, 70))
    a, b, c = cols[..., :128].unflatten(2, (2, 64)), cols[..., 136:200].unflatten(2, (1, 64)), cols[..., 200:].unflatten(2, (1, 64))
    y, fin = ss.linattn_fn(a, b, c, g["g"], h0=h0, return_final_state=True)
    torch.autograd.backward([y, fin], [g["dy"].unflatten(0, (2, 70)), g["df"]])
    torch.cuda.synchronize()
    gr = {"dq": row.grad[:, :128].unflatten(1, (2, 64)), "dk": row.grad[:, 136:200].unflatten(1, (1, 64)),
          "dv": row.grad[:, 200:].unflatten(1, (1, 64)), "dh0": h0.grad}
    assert int(row.grad[:, 128:136].count_nonzero()) == 0
    _check_train(q, y.detach().flatten(0, 1), fin.detach(), gr, True)
    with pytest.raises(ValueError):
        ss.linattn_fn(a, b, c, g["g"].clone().requires_grad_())
    with pytest.raises(RuntimeError):                    # once differentiable
        p = g["q"].clone().unflatten(0, (2, 70)).requires_grad_()
        o = ss.linattn_fn(p, b.detach(), c.detach(), g["g"])
        d, = torch.autograd.grad(o.float().square().sum(), p, create_graph=True)
        d.float().sum().backward()


# ---- single tokens --------------------------------------------------------------------


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,dk,dv,n", [(4, 4, 64, 64, 3), (4, 2, 64, 128, 70), (3, 1, 128, 64, 1), (2, 2, 128, 128, 9),
                                         (16, 4, 128, 128, 130)])
def test_step(io, H, G, dk, dv, n):
    """Both counts of workgroups; slots out of order, none (-1, beyond the pool) and rows at odd elements."""
    ss = _ss()
    q = _problem([1] * n, H, G, dk, dv, io, seed=n)
    if n > 2:
        q["slots"][1], q["slots"][2] = -1, n + 2
    g = _dev(q)
    wide = torch.zeros(n, q["row"].shape[1] + 3, dtype=DT[io], device="cuda")
    wide[:, 3:] = g["row"]
    cols = wide[:, 3:]
    a = (cols[:, :H * dk].unflatten(1, (H, dk)), cols[:, H * dk + 8:H * dk + 8 + G * dk].unflatten(1, (G, dk)),
         cols[:, H * dk + 8 + G * dk:].unflatten(1, (G, dv)))
    y = torch.full((n, H, dv), 7.0, dtype=DT[io], device="cuda")
    ss.linattn_step(*a, g["g"], g["state"], scale=q["scale"], slots=g["slots"], y=y)
    torch.cuda.synchronize()
    st, (qq, kk, vv) = f64(q["state"]), (f64(q[x]) for x in ("q", "k", "v"))
    want, mag, new, nm = np.full((n, H, dv), 7.0), np.zeros((n, H, dv)), st.copy(), np.zeros(st.shape)
    for i in range(n):
        s = int(q["slots"][i])
        if not 0 <= s < len(st):
            continue
        r = lambda f: (f(qq[i:i + 1]), f(kk[i:i + 1]), f(vv[i:i + 1]), f64(q["g"]), q["scale"], f(st[s]))
        want[i:i + 1], new[s] = ref.linattn_rows(*r(lambda x: x))
        mag[i:i + 1], nm[s] = ref.linattn_rows(*r(np.abs))
    # two roundings a state element, 2^-22 of its terms; a sum of at most 128 products
    check(y, want, mag, "y")
    check(g["state"], new, nm, "state", terms=2.0 ** -22)


def test_prompts_then_tokens():
    """A prompt in one piece equals its pieces, the last one token by token."""
    ss = _ss()
    q = _problem([150], 2, 2, 64, 128, "f16", seed=50)
    g = _dev(q)
    whole = torch.zeros(3, 2, 128, 64, device="cuda")
    y = ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], whole)
    st = torch.zeros(3, 2, 128, 64, device="cuda")
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    a = tuple(g[n] for n in ("q", "k", "v"))
    parts = [ss.linattn_prompt(*(x[:90] for x in a), g["g"], cu(90), st, slots=one),
             ss.linattn_prompt(*(x[90:140] for x in a), g["g"], cu(50), st, slots=one, has_state=one)]
    parts += [ss.linattn_step(*(x[t:t + 1] for x in a), g["g"], st, slots=one) for t in range(140, 150)]
    torch.cuda.synchronize()
    want, mag, last, lm = _forward(q, [np.zeros((2, 128, 64))])
    check(y, want, mag, "whole")
    check(torch.cat(parts), want, mag, "pieces")
    check(whole[0], last[0], lm[0], "state")
    check(st[1], last[0], lm[0], "state")


# ---- memory -----------------------------------------------------------------------------


def test_sequences_do_not_touch_each_other():
    """Values that are not finite stay in their sequence, and in their rows' neighbourhood of slots and outputs."""
    ss = _ss()
    q = _problem([70, 40, 200], 2, 2, 64, 64, "bf16", seed=60)
    g = _dev(q)
    clean = ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"].clone(), slots=g["slots"], has_state=g["has"])
    g["row"][75] = float("nan")
    g["row"][80] = float("inf")
    st = g["state"].clone()
    st[int(g["slots"][1])] = float("nan")
    y = ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], st, slots=g["slots"], has_state=g["has"])
    dy = g["dy"].unsqueeze(0)
    a = tuple(g[n].unsqueeze(0) for n in ("q", "k", "v")) + (g["g"],)
    gr = ss.linattn_bwd(*a, dy, cu_seqlens=g["cu"])
    torch.cuda.synchronize()
    assert torch.equal(y[:70], clean[:70]) and torch.equal(y[110:], clean[110:])
    for n in ("dq", "dk", "dv"):
        assert bool(torch.isfinite(gr[n][0, :70]).all()) and bool(torch.isfinite(gr[n][0, 110:]).all())


def test_offsets_out_of_order_stay_inside():
    """Offsets beyond the rows, below them and decreasing: calls that end, and guard rows that stay."""
    ss = _ss()
    q = _problem([700, 100], 2, 1, 64, 64, "f16", seed=61)
    g = _dev(q)
    for cu in ([900, -5, 300], [0, 100000, 3], [-7, 2 ** 31 - 1, 2 ** 31 - 1], [500, 400, 300], [800, 800, 800]):
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        guard = torch.full((q["T"] + 20, 2, 64), 7.0, dtype=torch.float16, device="cuda")
        pool = torch.full((6, 2, 64, 64), 3.0, device="cuda")
        ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], bad, pool[1:5], y=guard[10:-10])
        a = tuple(g[n].unsqueeze(0) for n in ("q", "k", "v")) + (g["g"],)
        ss.linattn_bwd(*a, g["dy"].unsqueeze(0), cu_seqlens=bad, want_dh0=True)
        torch.cuda.synchronize()
        assert bool((guard[:10] == 7).all()) and bool((guard[-10:] == 7).all())
        assert bool((pool[0] == 3).all()) and bool((pool[5] == 3).all())


def test_pool_offsets_past_32_bits():
    """Slots whose states lie more than 2^32 bytes into the pool."""
    ss = _ss()
    H, n = 16, 4200                                      # 1 MiB a slot
    pool = torch.zeros(n, H, 128, 128, device="cuda")
    q = _problem([3, 1], H, H, 128, 128, "bf16", seed=62)
    g = _dev(q)
    slots = torch.tensor([n - 1, n - 3], dtype=torch.int32, device="cuda")
    small = torch.zeros(2, H, 128, 128, device="cuda")
    y = ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], pool, slots=slots)
    z = ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], small)
    assert torch.equal(y, z) and torch.equal(pool[n - 1], small[0]) and torch.equal(pool[n - 3], small[1])
    a = tuple(g[x][:2] for x in ("q", "k", "v"))
    y = ss.linattn_step(*a, g["g"], pool, slots=slots)
    z = ss.linattn_step(*a, g["g"], small)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(pool[n - 1], small[0])
    assert int(pool[:n - 3].count_nonzero()) == 0


def test_streams_and_graph_replays_match_eager():
    """A captured training step and a captured token, replayed with new inputs and eager work in between, and two calls
    on streams of their own."""
    ss = _ss()
    q = _problem([300, 300], 2, 1, 64, 128, "bf16", seed=63)
    g = _dev(q)
    a = tuple(g[n].unflatten(0, (2, 300)) for n in ("q", "k", "v"))
    dy = g["dy"].unflatten(0, (2, 300))
    step = tuple(g[n][:2] for n in ("q", "k", "v"))

    def work(state):
        y, fin = ss.linattn_fwd(*a, g["g"], h0=g["h0"], return_final_state=True)
        gr = ss.linattn_bwd(*a, g["g"], dy, h0=g["h0"], dfinal=g["df"], want_dh0=True)
        return [y, fin, *gr.values(), ss.linattn_step(*step, g["g"], state), state]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(g["state"].clone())
    torch.cuda.current_stream().wait_stream(side)
    st = g["state"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(st)
    for k in range(3):
        g["row"].normal_()
        g["dy"].normal_()
        st.copy_(g["state"])
        graph.replay()
        want = work(g["state"].clone())
        torch.cuda.synchronize()
        for x, z in zip(outs, want):
            assert torch.equal(x, z), k
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            both.append(work(g["state"].clone()))
    torch.cuda.synchronize()
    for x in both:
        for u, z in zip(x, want):
            assert torch.equal(u, z)


def test_python_refusals():
    ss = _ss()
    q = _problem([20], 2, 1, 64, 64, "bf16", seed=64)
    g = _dev(q)
    a = (g["q"], g["k"], g["v"], g["g"], g["cu"])
    with pytest.raises(ValueError):
        ss.linattn_prompt(*a, g["state"], y=torch.zeros(20, 2, 128, dtype=torch.bfloat16, device="cuda")[:, :, :64])
    with pytest.raises(TypeError):
        ss.linattn_prompt(g["q"], g["k"].half(), *a[2:], g["state"])
    with pytest.raises(ValueError):
        ss.linattn_prompt(*a, g["state"][:, :, :, :32])
    with pytest.raises(ValueError):
        ss.linattn_prompt(g["q"], g["k"][:10], *a[2:], g["state"])
    with pytest.raises(TypeError):
        ss.linattn_prompt(*a[:3], g["g"].double(), g["cu"], g["state"])
    with pytest.raises(ValueError):
        ss.linattn_fwd(g["q"], g["k"], g["v"], g["g"])
    with pytest.raises(RuntimeError):                    # 3 heads for 2 of q
        three = torch.zeros(20, 3, 64, dtype=torch.bfloat16, device="cuda")
        ss.linattn_prompt(g["q"], three, three, *a[3:], g["state"])
    with pytest.raises(RuntimeError):                    # a size that is not there
        x = torch.zeros(20, 2, 32, dtype=torch.bfloat16, device="cuda")
        ss.linattn_step(x, x, x, g["g"], torch.zeros(20, 2, 32, 32, device="cuda"))
