"""GPU parity of the packed-prompt convolution and scan and of the decode step over state slots, against the
64-bit oracle, one sequence at a time; bounds in _layer_ref.py."""
import numpy as np
import pytest
import torch

import _layer_ref as ref
from _layer_ref import ELEMENT, SUM, check
from _util import f64, say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _ss():
    from mamba_selective_scan_fwd_amd import ss
    ss.load_library()
    return ss


def _cut(lens, lead=0, tail=0):
    cu = np.concatenate([[lead], lens]).cumsum()
    return torch.tensor(cu, dtype=torch.int32), int(cu[-1]) + tail


# ---- convolution of packed prompts --------------------------------------------------


def _conv_problem(lens, dim, W, io, seed, lead=0, tail=0, wide=0):
    r = np.random.default_rng(seed)
    cu, T = _cut(lens, lead, tail)
    t = lambda *s: torch.from_numpy(r.standard_normal(s))
    row = t(T, dim + wide).to(DT[io])
    return dict(x=row[:, wide:], w=(t(dim, W) * 0.5).float(), b=(t(dim) * 0.1).float(), cu=cu,
                state=t(len(lens) + 2, dim, W - 1).float(), slots=torch.tensor(r.permutation(len(lens) + 2)[:len(lens)],
                                                                               dtype=torch.int32),
                has=torch.tensor(r.integers(0, 2, len(lens)), dtype=torch.int32))


def _conv_check(q, got, state, slots=True, has=True, use_silu=True, bias=True, fill=None):
    x, w, b, st = f64(q["x"]), f64(q["w"]), f64(q["b"]) if bias else None, f64(q["state"])
    out, mag = np.full(x.shape, 0.0 if fill is None else fill), np.zeros(x.shape)
    new = st.copy()
    cu = q["cu"].tolist()
    for s in range(len(cu) - 1):
        slot = int(q["slots"][s]) if slots else s
        inside = 0 <= slot < st.shape[0]
        win = st[slot] if inside and has and int(q["has"][s]) else np.zeros(st.shape[1:])
        out[cu[s]:cu[s + 1]], mag[cu[s]:cu[s + 1]], last = ref.conv_rows(x[cu[s]:cu[s + 1]], w, b, win, use_silu)
        if inside:
            new[slot] = last
    # W + 1 fp32 terms, then SiLU, whose slope is at most 1.1
    check(got, out, mag, "out", terms=ELEMENT)
    assert np.array_equal(f64(state), new)          # inputs as they were, other slots untouched


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,wide", [(8, 8), (64, 0), (600, 40), (1, 0), (65, 3), (100, 7)])
def test_conv_prompt(io, dim, wide):
    """Vector and scalar rows, slices of wider rows, sequences shorter than the window, empty ones, chunk edges."""
    ss = _ss()
    q = _conv_problem([3, 0, 1, 16, 17, 2, 0, 40, 15, 33], dim, 4, io, seed=dim, lead=5, tail=6, wide=wide)
    say("conv prompt io=%s dim=%d" % (io, dim))
    g = {k: v.cuda() for k, v in q.items()}
    row = torch.zeros(g["x"].shape[0], dim + wide, dtype=DT[io], device="cuda")
    row[:, wide:] = g["x"]
    out = torch.full((row.shape[0], dim), 7.0, dtype=DT[io], device="cuda")
    ss.conv1d_prompt(row[:, wide:], g["w"], g["cu"], g["state"], bias=g["b"], slots=g["slots"], has_state=g["has"],
                     out=out)
    torch.cuda.synchronize()
    _conv_check(q, out, g["state"], fill=7.0)       # rows of no sequence stay as they were


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("start,wide", [(1, 9), (2, 8), (3, 12), (0, 1)])
def test_conv_prompt_rows_at_any_element(io, start, wide):
    """Rows that begin and lie at odd elements give what whole rows give, bit for bit, and nothing beside them is
    written."""
    ss = _ss()
    q = _conv_problem([20, 0, 3, 40], 66, 4, io, seed=start)
    g = {k: v.cuda() for k, v in q.items()}
    T = q["x"].shape[0]
    args = (g["w"], g["cu"])
    kw = dict(bias=g["b"], slots=g["slots"], has_state=g["has"])
    a, b = g["state"].clone(), g["state"].clone()
    want = ss.conv1d_prompt(g["x"].contiguous(), *args, a, **kw)
    src = torch.full((T, 66 + wide), 7.0, dtype=DT[io], device="cuda")
    src[:, start:start + 66] = g["x"]
    dst = torch.full((T, 66 + wide), 5.0, dtype=DT[io], device="cuda")
    ss.conv1d_prompt(src[:, start:start + 66], *args, b, out=dst[:, start:start + 66], **kw)
    torch.cuda.synchronize()
    assert torch.equal(dst[:, start:start + 66], want) and torch.equal(a, b)
    dst[:, start:start + 66] = 5.0
    assert bool((dst == 5.0).all())


@pytest.mark.parametrize("W", [1, 2, 3, 4])
def test_conv_prompt_options(W):
    ss = _ss()
    q = _conv_problem([5, 1, 30], 24, W, "bf16", seed=W)
    g = {k: v.cuda() for k, v in q.items()}
    out = ss.conv1d_prompt(g["x"], g["w"], g["cu"], g["state"], silu=False)       # slot = index, none carried
    torch.cuda.synchronize()
    _conv_check(q, out, g["state"], slots=False, has=False, use_silu=False, bias=False)
    q["slots"] = torch.tensor([-1, 4, 99], dtype=torch.int32)                      # -1 and 99: no slot
    g = {k: v.cuda() for k, v in q.items()}
    wide = torch.zeros(36, 40, dtype=torch.bfloat16, device="cuda")
    ss.conv1d_prompt(g["x"], g["w"], g["cu"], g["state"], bias=g["b"], slots=g["slots"], has_state=g["has"],
                     out=wide[:, 16:])
    torch.cuda.synchronize()
    _conv_check(q, wide[:, 16:], g["state"])
    assert int(wide[:, :16].count_nonzero()) == 0


def test_conv_prompt_many_sequences():
    """More sequences than one search step covers, most of them tiny."""
    ss = _ss()
    r = np.random.default_rng(2)
    q = _conv_problem((r.integers(0, 5, 5000) * (r.random(5000) < 0.3)).tolist() + [70], 16, 4, "f32", seed=3, tail=2)
    g = {k: v.cuda() for k, v in q.items()}
    out = torch.zeros(g["x"].shape, device="cuda")
    ss.conv1d_prompt(g["x"], g["w"], g["cu"], g["state"], bias=g["b"], slots=g["slots"], has_state=g["has"], out=out)
    torch.cuda.synchronize()
    _conv_check(q, out, g["state"])


# ---- scan of packed prompts ------------------------------------------------------------


def _ssd_problem(lens, H, G, N, io, seed, lead=0, tail=0, gate=True, skip=True):
    r = np.random.default_rng(seed)
    cu, T = _cut(lens, lead, tail)
    t = lambda *s: torch.from_numpy(r.standard_normal(s))
    row = t(T, H * 64 + 2 * G * N + 8).to(DT[io])
    dt0 = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), H))
    q = dict(row=row, dt=(t(T, H) * 0.5).to(DT[io]), A=torch.from_numpy(-r.uniform(1.0, 16.0, H)).float(),
             bias=torch.from_numpy(np.log(np.expm1(dt0))).float(), cu=cu,
             state=(t(len(lens) + 2, H, 64, N) * 0.5).float(),
             slots=torch.tensor(r.permutation(len(lens) + 2)[:len(lens)], dtype=torch.int32),
             has=torch.tensor(r.integers(0, 2, len(lens)), dtype=torch.int32))
    if skip:
        q["D"] = t(H).float()
    if gate:
        q["z"] = t(T, H, 64).to(DT[io])
    return q


def _parts(row, H, G, N):
    T = row.shape[0]
    return (row[:, :H * 64].view(T, H, 64), row[:, H * 64:H * 64 + G * N].view(T, G, N),
            row[:, H * 64 + G * N:H * 64 + 2 * G * N].view(T, G, N))


def _ssd_run(ss, q, H, G, N, y, **kw):
    g = {k: v.cuda() for k, v in q.items()}
    x, Bm, Cm = _parts(g["row"], H, G, N)
    ss.ssd_prompt(x, g["dt"], g["A"], Bm, Cm, g["cu"], g["state"], D=g.get("D"), z=g.get("z"), dt_bias=g["bias"], y=y,
                  **{**dict(slots=g["slots"], has_state=g["has"]), **kw})
    torch.cuda.synchronize()
    return g["state"]


def _ssd_check(q, H, G, N, y, state, slots=True, has=True, fill=0.0):
    x, Bm, Cm = (f64(v) for v in _parts(q["row"], H, G, N))
    A, dt, bias, st = f64(q["A"]), f64(q["dt"]), f64(q["bias"]), f64(q["state"])
    D, z = (f64(q[k]) if k in q else None for k in ("D", "z"))
    yr, ym = np.full(x.shape, fill), np.zeros(x.shape)
    sr, sm = st.copy(), np.zeros_like(st)
    cu = q["cu"].tolist()
    for s in range(len(cu) - 1):
        a, e = cu[s], cu[s + 1]
        slot = int(q["slots"][s]) if slots else s
        inside = 0 <= slot < st.shape[0]
        h0 = st[slot] if inside and has and int(q["has"][s]) else np.zeros(st.shape[1:])
        yr[a:e], ym[a:e], last, lm = ref.ssd_rows(x[a:e], dt[a:e], A, Bm[a:e], Cm[a:e], D, None if z is None else z[a:e],
                                                  bias, h0)
        if inside:
            sr[slot], sm[slot] = last, lm
    check(y, yr, ym, "y")
    check(state, sr, sm, "state")


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("N", [32, 64, 96, 128])
def test_ssd_prompt(io, N):
    """Lengths around the chunk's and its pieces' edges, empty sequences, rows of none, strided operands."""
    ss = _ss()
    H, G = 4, 2
    q = _ssd_problem([1, 0, 255, 256, 257, 64, 65, 15, 0, 300], H, G, N, io, seed=N, lead=3, tail=9)
    say("ssd prompt io=%s N=%d" % (io, N))
    y = torch.full((q["row"].shape[0], H, 64), 5.0, dtype=DT[io], device="cuda")
    state = _ssd_run(ss, q, H, G, N, y)
    _ssd_check(q, H, G, N, y, state, fill=5.0)


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (6, 3), (5, 5)])
def test_ssd_prompt_heads_and_options(H, G):
    ss = _ss()
    q = _ssd_problem([40, 530], H, G, 64, "bf16", seed=H, gate=False, skip=False)
    y = torch.zeros(570, H, 64, dtype=torch.bfloat16, device="cuda")
    state = _ssd_run(ss, q, H, G, 64, y, slots=None, has_state=None)
    _ssd_check(q, H, G, 64, y, state, slots=False, has=False)
    q["slots"] = torch.tensor([-1, 3], dtype=torch.int32)
    q["has"][:] = 1
    state = _ssd_run(ss, q, H, G, 64, y)
    _ssd_check(q, H, G, 64, y, state)


def test_ssd_prompt_single_tokens_and_many():
    ss = _ss()
    r = np.random.default_rng(4)
    q = _ssd_problem((r.integers(0, 3, 150)).tolist(), 2, 1, 32, "f16", seed=9)
    y = torch.zeros(q["row"].shape[0], 2, 64, dtype=torch.float16, device="cuda")
    state = _ssd_run(ss, q, 2, 1, 32, y)
    _ssd_check(q, 2, 1, 32, y, state)


def test_ssd_prompt_long():
    """Many chunks of one sequence: the states' way between them."""
    ss = _ss()
    q = _ssd_problem([5000], 2, 1, 64, "bf16", seed=11)
    q["A"] = torch.tensor([-0.02, -4.0])           # one head that forgets little
    y = torch.zeros(5000, 2, 64, dtype=torch.bfloat16, device="cuda")
    state = _ssd_run(ss, q, 2, 1, 64, y)
    _ssd_check(q, 2, 1, 64, y, state)


@pytest.mark.parametrize("io", ["bf16", "f16"])
def test_ssd_prompt_long_among_short(io):
    """A long prompt between an empty and two short ones, on average long: chunk numbers on both sides of 16."""
    ss = _ss()
    for lens in ([100, 9 * 1024, 0, 300], [0, 16 * 256, 16 * 256 + 1, 15 * 256]):
        q = _ssd_problem(lens, 2, 1, 32, io, seed=len(lens) + lens[0])
        y = torch.zeros(sum(lens), 2, 64, dtype=DT[io], device="cuda")
        state = _ssd_run(ss, q, 2, 1, 32, y)
        _ssd_check(q, 2, 1, 32, y, state)


@pytest.mark.parametrize("lens", [[256], [255, 1], [0, 100, 0], [256, 257, 0, 1], [0, 0]])
def test_ssd_prompt_one_chunk_or_none(lens):
    """Prompts of one chunk, of none and of two, carried and not, with and without a slot: the states in the slots
    and every output, and the slots that no prompt names stay as they were."""
    ss = _ss()
    H, G, N = 3, 1, 64
    q = _ssd_problem(lens, H, G, N, "bf16", seed=41 + len(lens) + lens[0])
    T = max(sum(lens), 1)
    if sum(lens) == 0:                                   # a row of no prompt
        q = _ssd_problem([1], H, G, N, "bf16", seed=40)
        q["cu"] = torch.zeros(len(lens) + 1, dtype=torch.int32)
    S = len(lens)
    g = {k: v.cuda() for k, v in q.items()}
    g.update(zip(("x", "Bm", "Cm"), _parts(g["row"], H, G, N)))
    pool = torch.randn(2 * S + 2, H, 64, N, generator=torch.Generator().manual_seed(5)).cuda()
    for use in (True, False):
        slots = torch.tensor([2 * k + 1 if k != 1 else -1 for k in range(S)], dtype=torch.int32, device="cuda")
        has = torch.full((S,), int(use), dtype=torch.int32, device="cuda")
        state = pool.clone()
        y = torch.zeros(T, H, 64, dtype=torch.bfloat16, device="cuda")
        ss.ssd_prompt(g["x"], g["dt"], g["A"], g["Bm"], g["Cm"], g["cu"], state, D=g.get("D"), z=g.get("z"),
                      dt_bias=g["bias"], slots=slots, has_state=has, y=y)
        torch.cuda.synchronize()
        at = 0
        for k, n in enumerate(lens):
            slot = int(slots[k])
            if n:                                        # the same prompt alone, in a pool of its own
                one = pool[slot:slot + 1].clone() if slot >= 0 and use else torch.zeros_like(pool[:1])
                cut = lambda v: g[v][at:at + n].contiguous() if v in g else None
                yk = torch.zeros(n, H, 64, dtype=torch.bfloat16, device="cuda")
                ss.ssd_prompt(cut("x"), cut("dt"), g["A"], cut("Bm"), cut("Cm"),
                              torch.tensor([0, n], dtype=torch.int32, device="cuda"), one, D=g.get("D"), z=cut("z"),
                              dt_bias=g["bias"], has_state=torch.ones(1, dtype=torch.int32, device="cuda"),
                              y=yk)
                assert torch.equal(y[at:at + n], yk), (k, n)
                if slot >= 0:
                    assert torch.equal(state[slot], one[0]), (k, n)
            elif slot >= 0:
                assert torch.equal(state[slot], pool[slot] if use else torch.zeros_like(pool[slot])), k
            at += n
        named = {int(v) for v in slots if v >= 0}
        for k in range(pool.shape[0]):
            if k not in named:
                assert torch.equal(state[k], pool[k])


def test_ssd_prompt_strong_and_no_decay():
    """Steps that forget everything (the weights underflow) and steps that change nothing (Delta = 0)."""
    ss = _ss()
    q = _ssd_problem([270, 300], 2, 1, 64, "bf16", seed=12)
    q["dt"][:270] = 60.0                            # exp(-16 * 60) = 0
    q["A"] = torch.tensor([-16.0, -1.0])
    q["dt"][270:] = -200.0                          # softplus(-200) = 0
    q["has"][:] = 1
    y = torch.zeros(570, 2, 64, dtype=torch.bfloat16, device="cuda")
    state = _ssd_run(ss, q, 2, 1, 64, y)
    _ssd_check(q, 2, 1, 64, y, state)


def test_sequences_do_not_touch_each_other():
    """A sequence full of infinities and NaN leaves the others' results as they are, bit for bit."""
    ss = _ss()
    q = _ssd_problem([100, 70, 300], 2, 1, 64, "bf16", seed=13)
    q["slots"] = torch.tensor([0, 3, 2], dtype=torch.int32)
    y0, y1 = (torch.zeros(470, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s0 = _ssd_run(ss, q, 2, 1, 64, y0)
    bad = dict(q, row=q["row"].clone(), dt=q["dt"].clone())
    bad["row"][100:170, ::3] = float("nan")
    bad["row"][100:170, 1::3] = float("inf")
    s1 = _ssd_run(ss, bad, 2, 1, 64, y1)
    keep = torch.ones(470, dtype=torch.bool)
    keep[100:170] = False
    assert torch.equal(y0[keep.cuda()], y1[keep.cuda()]) and torch.equal(s0[[0, 1, 2, 4]], s1[[0, 1, 2, 4]])


def test_offsets_out_of_order_stay_inside():
    """Offsets that are no offsets (negative, past the rows, decreasing) are clamped: nothing outside the rows
    and the pool changes."""
    ss = _ss()
    q = _ssd_problem([40, 30, 60], 2, 1, 32, "bf16", seed=14)
    guard = torch.full((130 + 64, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    pool = torch.full((5 + 4, 2, 64, 32), 2.0, device="cuda")
    for cu in ([-7, 50, 20, 9999], [90, 60, 30, 0], [200, 300, -1, 130]):
        q["cu"] = torch.tensor(cu, dtype=torch.int32)
        g = {k: v.cuda() for k, v in q.items()}
        x, Bm, Cm = _parts(g["row"], 2, 1, 32)
        ss.ssd_prompt(x, g["dt"], g["A"], Bm, Cm, g["cu"], pool[2:7], D=g["D"], z=g["z"], dt_bias=g["bias"],
                      slots=g["slots"], has_state=g["has"], y=guard[32:162])
        w, cs = torch.ones(64, 4, device="cuda"), torch.ones(5, 64, 3, device="cuda")
        ss.conv1d_prompt(guard[32:162, 0], w, g["cu"], cs, slots=g["slots"], out=torch.empty(130, 64, device="cuda").bfloat16())
        torch.cuda.synchronize()
        assert bool((guard[:32] == 3.0).all()) and bool((guard[162:] == 3.0).all())
        assert bool((pool[:2] == 2.0).all()) and bool((pool[7:] == 2.0).all())


# ---- decode step ----------------------------------------------------------------------------


def _step_problem(n, H, G, N, W, io, seed, slots, gate=True):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s))
    ch = H * 64 + 2 * G * N
    dt0 = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), H))
    q = dict(row=t(n, H * 64 + ch + H + 3).to(DT[io]), A=torch.from_numpy(-r.uniform(1.0, 16.0, H)).float(),
             D=t(H).float(), bias=torch.from_numpy(np.log(np.expm1(dt0))).float(), w=(t(ch, W) * 0.5).float(),
             cb=(t(ch) * 0.1).float(), conv=t(slots, ch, W - 1).float(), state=(t(slots, H, 64, N) * 0.5).float(),
             slots=torch.tensor(r.permutation(slots)[:n], dtype=torch.int32))
    return q


def _step_ref(q, H, G, N, gate, order):
    """The convolution and one step of the oracle's scan, row by row."""
    row = f64(q["row"])
    ch = H * 64 + 2 * G * N
    conv, state = f64(q["conv"]), f64(q["state"])
    cm, sm = np.zeros_like(conv), np.zeros_like(state)
    y, ym = np.zeros((row.shape[0], H, 64)), np.zeros((row.shape[0], H, 64))
    for i, slot in enumerate(order):
        if not 0 <= slot < state.shape[0]:
            continue
        z = row[i, :H * 64].reshape(H, 64) if gate else None
        out, mag, conv[slot] = ref.conv_rows(row[i:i + 1, H * 64:H * 64 + ch], f64(q["w"]), f64(q["cb"]), conv[slot])
        b = lambda v: (v[:, :H * 64].reshape(1, H, 64), v[:, H * 64:H * 64 + G * N].reshape(1, G, N),
                       v[:, H * 64 + G * N:].reshape(1, G, N))
        dt = row[i:i + 1, H * 64 + ch:H * 64 + ch + H]
        x, Bm, Cm = b(out)
        y_, _, s_, _ = ref.ssd_rows(x, dt, f64(q["A"]), Bm, Cm, f64(q["D"]), None if z is None else z[None],
                                    f64(q["bias"]), state[slot])
        # every convolved channel carries its own terms' rounding (magnitudes 1.1 mag above |out|)
        x, Bm, Cm = b(np.abs(out) + 1.1 * mag)
        _, m_, _, n_ = ref.ssd_rows(x, dt, f64(q["A"]), Bm, Cm, f64(q["D"]), None if z is None else z[None],
                                    f64(q["bias"]), np.abs(state[slot]))
        y[i], ym[i], state[slot], sm[slot] = y_[0], m_[0], s_, n_
    return y, ym, conv, state, sm


def _step_args(q, H, G, N, gate):
    g = {k: v.cuda() for k, v in q.items()}
    ch = H * 64 + 2 * G * N
    n = g["row"].shape[0]
    return g, dict(xbc=g["row"][:, H * 64:H * 64 + ch], dt=g["row"][:, H * 64 + ch:H * 64 + ch + H], A=g["A"],
                   conv_w=g["w"], conv_state=g["conv"], state=g["state"], ngroups=G, conv_bias=g["cb"], D=g["D"],
                   z=g["row"][:, :H * 64].view(n, H, 64) if gate else None, dt_bias=g["bias"])


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("N", [32, 64, 96, 128])
@pytest.mark.parametrize("W", [1, 2, 4])
def test_ssd_step(io, N, W):
    """Rows at odd offsets, permuted slots, padding rows (-1, past the pool) that nothing is written for."""
    ss = _ss()
    H, G, gate = 4, 2, N != 64
    q = _step_problem(7, H, G, N, W, io, seed=N + W, slots=11)
    q["slots"][2], q["slots"][5] = -1, 11
    say("step io=%s N=%d W=%d" % (io, N, W))
    g, a = _step_args(q, H, G, N, gate)
    y = torch.full((7, H, 64), 9.0, dtype=DT[io], device="cuda")
    ss.ssd_step(slots=g["slots"], y=y, **a)
    torch.cuda.synchronize()
    yr, ym, conv, state, sm = _step_ref(q, H, G, N, gate, q["slots"].tolist())
    yr[[2, 5]] = 9.0
    # all in fp32: a dozen roundings, and a sum of N
    check(y, yr, ym, "y", terms=2.0 ** -17)
    check(g["state"], state, sm, "state", terms=ELEMENT)
    assert np.array_equal(f64(g["conv"]), conv)


def test_ssd_step_call_and_default_slots():
    ss = _ss()
    q = _step_problem(3, 2, 1, 64, 4, "bf16", seed=5, slots=4)
    g, a = _step_args(q, 2, 1, 64, True)
    y0 = ss.ssd_step(**a)
    h, b = _step_args(q, 2, 1, 64, True)
    y1 = torch.empty_like(y0)
    ss.SsdStepCall(y=y1, slots=torch.arange(3, dtype=torch.int32, device="cuda"), **b)()
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(g["state"], h["state"]) and torch.equal(g["conv"], h["conv"])
    yr, ym, _, state, sm = _step_ref(q, 2, 1, 64, True, [0, 1, 2])
    check(y0, yr, ym, "y", terms=2.0 ** -17)
    check(g["state"], state, sm, "state", terms=ELEMENT)


def test_python_refusals():
    ss = _ss()
    q = _step_problem(3, 2, 1, 64, 4, "bf16", seed=5, slots=4)
    g, a = _step_args(q, 2, 1, 64, True)
    with pytest.raises(RuntimeError):                                 # fewer slots than rows, none named
        ss.ssd_step(**dict(a, conv_state=g["conv"][:2], state=g["state"][:2]))
    with pytest.raises(ValueError):                                   # a pool is never copied
        ss.ssd_step(**dict(a, state=g["state"].transpose(2, 3)))
    with pytest.raises(ValueError):
        ss.ssd_step(**dict(a, conv_state=g["conv"].double()))
    with pytest.raises(ValueError):
        ss.ssd_step(**dict(a, y=torch.empty(3, 2, 128, dtype=torch.bfloat16, device="cuda")[..., ::2]))
    with pytest.raises(ValueError):
        ss.ssd_step(**dict(a, xbc=a["xbc"][:, :-1]))
    with pytest.raises(ValueError):
        ss.SsdStepCall(y=None, **a)
    with pytest.raises(ValueError):
        ss.SsdStepCall(y=torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda"), **dict(a, xbc=a["xbc"].t().contiguous().t()))
    with pytest.raises(RuntimeError):                                 # output inside the pool
        ss.ssd_step(**dict(a, y=g["state"].view(torch.bfloat16).view(-1)[:384].view(3, 2, 64)))


# ---- the three together ------------------------------------------------------------------------


def _layer(seed, H=4, G=2, N=64, W=4):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s))
    ch = H * 64 + 2 * G * N
    dt0 = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), H))
    return dict(w=(t(ch, W) * 0.5).float(), cb=(t(ch) * 0.1).float(), A=torch.from_numpy(-r.uniform(1, 16, H)).float(),
                D=t(H).float(), bias=torch.from_numpy(np.log(np.expm1(dt0))).float()), ch, t


def test_prompts_then_tokens():
    """A serving batch as it runs: ragged prompts through convolution and scan into slots, one prompt in two
    pieces, then tokens one by one; against whole sequences in 64 bits.  The prompts' convolved channels are
    rounded to bf16 in between, so the bound has one more half step of every factor (x, B and C)."""
    ss = _ss()
    H, G, N, W = 4, 2, 64, 4
    lay, ch, t = _layer(21)
    lens, extra = [300, 5, 70], 6
    full = [t(n + extra, ch).to(torch.bfloat16) for n in lens]
    dts = [(t(n + extra, H) * 0.5).to(torch.bfloat16) for n in lens]
    zs = [t(n + extra, H, 64).to(torch.bfloat16) for n in lens]
    g = {k: v.cuda() for k, v in lay.items()}
    conv, state = torch.ones(5, ch, W - 1, device="cuda"), torch.ones(5, H, 64, N, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")

    def prompts(pieces, has):
        xbc = torch.cat([full[i][a:e] for i, a, e in pieces]).cuda()
        dt = torch.cat([dts[i][a:e] for i, a, e in pieces]).cuda()
        z = torch.cat([zs[i][a:e] for i, a, e in pieces]).cuda()
        cu = torch.tensor(np.concatenate([[0], [e - a for _, a, e in pieces]]).cumsum(), dtype=torch.int32).cuda()
        sl, hs = slots[[i for i, _, _ in pieces]], torch.tensor(has, dtype=torch.int32).cuda()
        out = ss.conv1d_prompt(xbc, g["w"], cu, conv, bias=g["cb"], slots=sl, has_state=hs)
        x, Bm, Cm = _parts(out, H, G, N)
        return ss.ssd_prompt(x, dt, g["A"], Bm, Cm, cu, state, D=g["D"], z=z, dt_bias=g["bias"], slots=sl, has_state=hs)

    first = prompts([(0, 0, 131), (1, 0, 5), (2, 0, 70)], [0, 0, 0])
    second = prompts([(0, 131, 300)], [1])
    got = [[first[:131], second], [first[131:136]], [first[136:]]]
    for k in range(extra):
        xbc = torch.stack([full[i][lens[i] + k] for i in range(3)]).cuda()
        dt = torch.stack([dts[i][lens[i] + k] for i in range(3)]).cuda()
        z = torch.stack([zs[i][lens[i] + k] for i in range(3)]).cuda()
        y = ss.ssd_step(xbc, dt, g["A"], g["w"], conv, state, ngroups=G, conv_bias=g["cb"], D=g["D"], z=z,
                        dt_bias=g["bias"], slots=slots)
        for i in range(3):
            got[i].append(y[i:i + 1])
    torch.cuda.synchronize()
    for i in range(3):
        out, _, _ = ref.conv_rows(f64(full[i]), f64(lay["w"]), f64(lay["cb"]), np.zeros((ch, W - 1)))
        b = lambda v: (v[:, :H * 64].reshape(-1, H, 64), v[:, H * 64:H * 64 + G * N].reshape(-1, G, N),
                       v[:, H * 64 + G * N:].reshape(-1, G, N))
        x, Bm, Cm = b(out)
        yr, ym, sr, sm = ref.ssd_rows(x, f64(dts[i]), f64(lay["A"]), Bm, Cm, f64(lay["D"]), f64(zs[i]),
                                      f64(lay["bias"]), np.zeros((H, 64, N)))
        check(torch.cat(got[i]), yr, ym, "y %d" % i, terms=3 * 2.0 ** -8 + SUM)
        check(state[int(slots[i])], sr, sm, "state %d" % i, terms=2 * 2.0 ** -8 + SUM)
    assert bool((state[[1, 3]] == 1.0).all()) and bool((conv[[1, 3]] == 1.0).all())


def _one_round(ss, g, xbc, dt, z, cu, slots, has, conv, state, tok, H, G, N, ws=None):
    out = ss.conv1d_prompt(xbc, g["w"], cu, conv, bias=g["cb"], slots=slots, has_state=has)
    x, Bm, Cm = _parts(out, H, G, N)
    y = ss.ssd_prompt(x, dt, g["A"], Bm, Cm, cu, state, D=g["D"], z=z, dt_bias=g["bias"], slots=slots, has_state=has)
    yt = ss.ssd_step(tok, dt[:2], g["A"], g["w"], conv, state, ngroups=G, conv_bias=g["cb"], D=g["D"], z=z[:2],
                     dt_bias=g["bias"], slots=slots)
    return y, yt


def test_streams_and_graph_replays_match_eager():
    """The same round of calls on the default stream, on a side stream, as two rounds at once on two streams, and
    captured and replayed with eager work in between, slots and lengths changed in place: all bit for bit."""
    ss = _ss()
    H, G, N = 4, 2, 64
    lay, ch, t = _layer(22)
    g = {k: v.cuda() for k, v in lay.items()}
    xbc, tok = t(400, ch).to(torch.bfloat16).cuda(), t(2, ch).to(torch.bfloat16).cuda()
    dt, z = (t(400, H) * 0.5).to(torch.bfloat16).cuda(), t(400, H, 64).to(torch.bfloat16).cuda()
    conv0, state0 = t(4, ch, 3).float().cuda(), t(4, H, 64, N).float().cuda()
    plans = [([0, 300, 400], [2, 0], [1, 0]), ([0, 10, 390], [1, 3], [1, 1]), ([5, 5, 261], [3, 2], [0, 1])]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")

    def fresh(plan):
        conv, state = conv0.clone(), state0.clone()
        r = _one_round(ss, g, xbc, dt, z, i32(plan[0]), i32(plan[1]), i32(plan[2]), conv, state, tok, H, G, N)
        return (*r, conv, state)

    def same(a, b, plan):
        lo, hi = plan[0][0], plan[0][-1]
        return torch.equal(a[0][lo:hi], b[0][lo:hi]) and all(torch.equal(u, v) for u, v in zip(a[1:], b[1:]))

    want = [fresh(p) for p in plans]
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (one, two):
        s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(one):
        a = fresh(plans[0])
    with torch.cuda.stream(two):
        b = fresh(plans[1])
    one.synchronize()
    two.synchronize()
    assert same(a, want[0], plans[0]) and same(b, want[1], plans[1])
    cu, sl, hs = i32(plans[0][0]), i32(plans[0][1]), i32(plans[0][2])
    conv, state = conv0.clone(), state0.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y, yt = _one_round(ss, g, xbc, dt, z, cu, sl, hs, conv, state, tok, H, G, N)
    for k in (0, 1, 2, 1, 0):
        for dst, src in ((cu, plans[k][0]), (sl, plans[k][1]), (hs, plans[k][2])):
            dst.copy_(i32(src))
        conv.copy_(conv0)
        state.copy_(state0)
        graph.replay()
        torch.cuda.synchronize()
        say("replay of plan %d" % k)
        assert same((y, yt, conv, state), want[k], plans[k])
        fresh(plans[(k + 1) % 3])                       # eager work between replays
        torch.cuda.synchronize()


def test_pool_offsets_past_32_bits():
    """Slots whose states lie past 2^31 elements of the pool."""
    ss = _ss()
    H, G, N = 64, 1, 128
    n = (1 << 31) // (H * 64 * N) + 3                   # 4099 slots of 2 MiB: 8.6 GB
    state = torch.zeros(n, H, 64, N, device="cuda")
    q = _step_problem(2, H, G, N, 2, "bf16", seed=8, slots=3)
    small = {k: v.cuda() for k, v in q.items()}
    ch = H * 64 + 2 * G * N
    conv = torch.zeros(n, ch, 1, device="cuda")
    far = torch.tensor([n - 1, 1], dtype=torch.int32, device="cuda")
    near = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    for pool, cv, sl in ((state, conv, far), (small["state"], small["conv"], near)):
        pool[sl.long()] = q["state"][[2, 1]].cuda()
        cv[sl.long()] = q["conv"][[2, 1]].cuda()
    _, a = _step_args(q, H, G, N, True)
    y0 = ss.ssd_step(**dict(a, conv_state=conv, state=state, slots=far))
    y1 = ss.ssd_step(**dict(a, conv_state=small["conv"], state=small["state"], slots=near))
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(state[n - 1], small["state"][2]) and torch.equal(conv[n - 1], small["conv"][2])
    row = torch.randn(40, ch, device="cuda").bfloat16()
    x, Bm, Cm = _parts(row, H, G, N)
    dt = torch.zeros(40, H, device="cuda").bfloat16()
    cu = torch.tensor([0, 17, 40], dtype=torch.int32, device="cuda")
    has = torch.ones(2, dtype=torch.int32, device="cuda")
    y0 = ss.ssd_prompt(x, dt, small["A"], Bm, Cm, cu, state, slots=far, has_state=has)
    y1 = ss.ssd_prompt(x, dt, small["A"], Bm, Cm, cu, small["state"], slots=near, has_state=has)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(state[n - 1], small["state"][2])
