"""GPU parity of ss_ssd_bwd and ss_conv1d_bwd against the 64-bit references (their pins: test_layer_grad_pins.py),
by differences of the oracle's forward, through autograd, on streams and in graphs; bounds in _layer_ref.py."""
import numpy as np
import pytest
import torch

import _layer_ref as ref
import oracle
from _layer_ref import ELEMENT, SUM, check
from _util import f64, say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _ss():
    from mamba_selective_scan_fwd_amd import ss
    ss.load_library()
    return ss


def _ssd(Bsz, L, H, G, N, io, seed, gate=False, docs=False, state=False, skip=True, bias=True):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s))
    dt0 = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), H))
    q = dict(x=t(Bsz, L, H, 64).to(DT[io]), dt=(t(Bsz, L, H) * 0.5).to(DT[io]),
             A=torch.from_numpy(-r.uniform(1.0, 16.0, H)).float(), Bm=t(Bsz, L, G, N).to(DT[io]),
             Cm=t(Bsz, L, G, N).to(DT[io]), dy=t(Bsz, L, H, 64).to(DT[io]))
    if skip:
        q["D"] = t(H).float()
    if bias:
        q["dt_bias"] = torch.from_numpy(np.log(np.expm1(dt0))).float()
    if gate:
        q["z"] = t(Bsz, L, H, 64).to(DT[io])
    if docs:
        q["seq_idx"] = torch.from_numpy(np.cumsum(r.random((Bsz, L)) < 4.0 / L, 1)).to(torch.int32)
    if state:
        q["h0"], q["dfinal"] = (t(Bsz, H, 64, N) * 0.5).float(), (t(Bsz, H, 64, N) * 0.1).float()
    return q


def _bwd(ss, q, **kw):
    g = {k: v.cuda() for k, v in q.items()}
    opt = {k: g.get(k) for k in ("D", "z", "dt_bias", "seq_idx", "h0", "dfinal")}
    return ss.ssd_bwd(g["x"], g["dt"], g["A"], g["Bm"], g["Cm"], g["dy"], **{**opt, **kw})


def _check_ssd(q, got, softplus=True):
    want, mag = ref.ssd_grad({k: (v.numpy() if k == "seq_idx" else f64(v)) for k, v in q.items()}, softplus)
    for k, v in got.items():
        check(v, want[k], mag[k], k)


@pytest.mark.parametrize("io,gate", [("bf16", False), ("bf16", True), ("f16", False), ("f16", True)])
@pytest.mark.parametrize("N", [32, 64, 96, 128])
def test_ssd_bwd(io, gate, N):
    """Every type, gate and state size, a length across two chunk edges, documents, states in and out."""
    ss = _ss()
    say("ssd bwd io=%s N=%d gate=%d" % (io, N, gate))
    q = _ssd(2, 530, 4, 2, N, io, seed=N + gate, gate=gate, docs=True, state=True)
    got = _bwd(ss, q, want_dh0=True)
    torch.cuda.synchronize()
    assert set(got) == {"dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"} | ({"dz"} if gate else set())
    _check_ssd(q, got)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 128, 193, 255, 256, 257, 512])
def test_ssd_bwd_lengths(L):
    ss = _ss()
    q = _ssd(1, L, 2, 1, 64, "bf16", seed=L)
    got = _bwd(ss, q, want_dh0=True)                  # the gradient of a zero initial state
    torch.cuda.synchronize()
    _check_ssd(q, got)


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (6, 3), (5, 5)])
def test_ssd_bwd_shared_heads_and_missing_operands(H, G):
    ss = _ss()
    q = _ssd(2, 300, H, G, 32, "f16", seed=H, skip=False, bias=False, state=True)
    del q["h0"]
    got = _bwd(ss, q)
    torch.cuda.synchronize()
    assert set(got) == {"dx", "ddt", "dA", "dB", "dC"}
    _check_ssd(q, got)


def test_ssd_bwd_without_softplus_and_every_step_a_document():
    ss = _ss()
    q = _ssd(1, 300, 2, 1, 64, "bf16", seed=3, bias=False)
    q["dt"] = (q["dt"].float().abs() * 0.05 + 0.001).to(torch.bfloat16)
    got = _bwd(ss, q, dt_softplus=False)
    torch.cuda.synchronize()
    _check_ssd(q, got, softplus=False)
    q = _ssd(1, 300, 2, 1, 64, "bf16", seed=4, state=True)
    q["seq_idx"] = torch.arange(300, dtype=torch.int32)[None].flip(1).contiguous()
    got = _bwd(ss, q, want_dh0=True)
    torch.cuda.synchronize()
    _check_ssd(q, got)
    assert int(got["dA"].count_nonzero()) <= 2 and np.abs(f64(got["dA"])).max() < 1e3


def test_ssd_bwd_strong_and_weak_decay():
    """Decays that leave nothing, heads that forget nothing over many chunks (their decay's gradient is a small
    difference of large sums), and a head of constant state."""
    ss = _ss()
    q = _ssd(1, 1400, 3, 1, 32, "bf16", seed=6, state=True)
    q["A"] = torch.tensor([-200.0, -0.01, -1.0])
    q["dt"][:, :, 2] = -100.0                          # softplus = 0: exactly no step
    got = _bwd(ss, q, want_dh0=True)
    torch.cuda.synchronize()
    _check_ssd(q, got)


def test_decay_gradient_keeps_fp32_accuracy():
    """dA and ddt_bias against 64 bits in relative terms, over a length where errors that add up along a chunk
    would show: 4 units of 2^-20 of the whole vector (fp32 sums of a few thousand terms of either sign)."""
    ss = _ss()
    for io, gate in (("bf16", False), ("f16", True)):
        q = _ssd(2, 1024, 4, 1, 64, io, seed=7, gate=gate)
        got = _bwd(ss, q)
        torch.cuda.synchronize()
        want, _ = ref.ssd_grad({k: f64(v) for k, v in q.items()})
        for k in ("dA", "ddt_bias", "dD"):
            e = np.linalg.norm(f64(got[k]) - want[k]) / np.linalg.norm(want[k])
            say("%s %s %.2e" % (io, k, e))
            assert e <= 2.0 ** -18


def test_ssd_bwd_by_differences():
    """The device's gradients along a random direction against central differences of the oracle's forward."""
    ss = _ss()
    q = _ssd(1, 280, 2, 1, 32, "f16", seed=8, gate=True, docs=True, state=True)
    got = _bwd(ss, q, want_dh0=True)
    torch.cuda.synchronize()
    r = np.random.default_rng(9)
    p = {k: (v.numpy() if k == "seq_idx" else f64(v)) for k, v in q.items()}
    _, mag = ref.ssd_grad(p)
    d = {k: r.standard_normal(p[k].shape) * (np.abs(p[k]) if k == "A" else 1.0)
         for k in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "z", "h0")}

    def loss(s):
        v = {k: p[k] + s * d.get(k, 0.0) for k in p}
        y, fin = oracle.ssd_fwd(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], D=v["D"], z=v["z"], dt_bias=v["dt_bias"],
                                seq_idx=p["seq_idx"], h0=v["h0"])
        return (y * p["dy"]).sum() + (fin * p["dfinal"]).sum()

    h = 1e-6
    fd = (loss(h) - loss(-h)) / (2 * h)
    name = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", dt_bias="ddt_bias", z="dz", h0="dh0")
    an = sum((f64(got[name[k]]) * d[k]).sum() for k in d)
    # the rounding of 16-bit gradients and the sums' errors, each in any direction, and the difference's own
    bound = sum(((ref.HALF[got[name[k]].dtype] * np.abs(f64(got[name[k]])) + SUM * mag[name[k]]) * np.abs(d[k])).sum()
                for k in d) + 1e-6 * abs(fd)
    say("differences %.6e gradients %.6e bound %.1e" % (fd, an, bound))
    assert abs(fd - an) <= bound


def test_ssd_scan_fn():
    """Autograd: forward and backward of the training call, a shared (broadcast) input among them."""
    ss = _ss()
    q = _ssd(2, 300, 4, 2, 64, "bf16", seed=10, gate=True, docs=True, state=True)
    leaf = {k: v.cuda().requires_grad_(k not in ("seq_idx", "dfinal", "dy")) if v.is_floating_point() else v.cuda()
            for k, v in q.items()}
    row = leaf["h0"].detach()[:1].clone().requires_grad_()       # one initial state for both rows
    y, fin = ss.ssd_scan_fn(leaf["x"], leaf["dt"], leaf["A"], leaf["Bm"], leaf["Cm"], D=leaf["D"], z=leaf["z"],
                            dt_bias=leaf["dt_bias"], seq_idx=leaf["seq_idx"], h0=row.expand(2, -1, -1, -1),
                            return_final_state=True)
    torch.autograd.backward([y, fin], [leaf["dy"], leaf["dfinal"]])
    torch.cuda.synchronize()
    q["h0"] = q["h0"][:1].expand(2, -1, -1, -1).contiguous()
    want, mag = ref.ssd_grad({k: (v.numpy() if k == "seq_idx" else f64(v)) for k, v in q.items()})
    for k, n in dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", dt_bias="ddt_bias", z="dz").items():
        check(leaf[k].grad, want[n], mag[n], n)
    check(row.grad, want["dh0"].sum(0, keepdims=True), mag["dh0"].sum(0, keepdims=True), "dh0")


# ---- convolution ------------------------------------------------------------------------------


def _conv(Bsz, D, L, W, io, seed, docs=False, state=False, bias=True):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s))
    q = dict(x=t(Bsz, D, L).to(DT[io]), w=(t(D, W) * 0.5).float(), dout=t(Bsz, D, L).to(DT[io]))
    if bias:
        q["bias"] = (t(D) * 0.1).float()
    if docs:
        q["seq_idx"] = torch.from_numpy(np.cumsum(r.random((Bsz, L)) < 4.0 / L, 1)).to(torch.int32)
    if state:
        q["conv_init"], q["dconv_final"] = t(Bsz, D, W - 1).float(), t(Bsz, D, W - 1).float()
    return q


def _check_conv(q, got, use_silu=True):
    n = {k: (v.numpy() if k == "seq_idx" else f64(v)) for k, v in q.items()}
    want, mag = ref.conv_grad(n["x"], n["w"], n["dout"], n.get("bias"), use_silu, n.get("seq_idx"), n.get("conv_init"),
                              n.get("dconv_final"))
    check(got["dx"], want["dx"], mag["dx"], "dx", terms=ELEMENT)
    for k in ("dw", "dbias"):
        if k in got:                                   # fp32 sums, a few hundred terms one after the other
            check(got[k], want[k], mag[k], k, terms=SUM)
    if "dconv_init" in got:
        check(got["dconv_init"], want["dconv_init"], mag["dconv_init"], "dconv_init", terms=ELEMENT)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 3, 4, 7, 8, 9, 12, 16, 19, 64, 2048, 2051])
@pytest.mark.parametrize("docs", [False, True])
def test_conv_bwd(io, L, docs):
    """Rows shorter than the window, whole and cut chunks of 8, several units of a channel."""
    ss = _ss()
    q = _conv(3, 5, L, 4, io, seed=L, docs=docs, state=True)
    g = {k: v.cuda() for k, v in q.items()}
    got = ss.conv1d_bwd(want_dconv_init=True, **g)
    torch.cuda.synchronize()
    _check_conv(q, got)


@pytest.mark.parametrize("W", [1, 2, 3])
@pytest.mark.parametrize("silu", [False, True])
def test_conv_bwd_widths(W, silu):
    ss = _ss()
    q = _conv(2, 33, 100, W, "bf16", seed=W, docs=W > 1, state=W > 1, bias=silu)
    g = {k: v.cuda() for k, v in q.items()}
    got = ss.conv1d_bwd(silu=silu, want_dconv_init=W > 1, **g)
    torch.cuda.synchronize()
    assert ("dbias" in got) == silu
    _check_conv(q, got, use_silu=silu)


def test_conv_bwd_one_part_per_channel():
    """Enough channels that no partial sums are kept."""
    ss = _ss()
    q = _conv(2, 4100, 24, 4, "f16", seed=1)
    got = ss.conv1d_bwd(**{k: v.cuda() for k, v in q.items()})
    torch.cuda.synchronize()
    _check_conv(q, got)


def test_conv1d_fn():
    ss = _ss()
    q = _conv(2, 6, 50, 4, "f32", seed=2, docs=True, state=True)
    leaf = {k: v.cuda().requires_grad_(k in ("x", "w", "bias", "conv_init")) if v.is_floating_point() else v.cuda()
            for k, v in q.items()}
    out, fin = ss.conv1d_fn(leaf["x"], leaf["w"], leaf["bias"], seq_idx=leaf["seq_idx"], conv_init=leaf["conv_init"],
                            return_final=True)
    torch.autograd.backward([out, fin], [leaf["dout"], leaf["dconv_final"]])
    torch.cuda.synchronize()
    _check_conv(q, dict(dx=leaf["x"].grad, dw=leaf["w"].grad, dbias=leaf["bias"].grad,
                        dconv_init=leaf["conv_init"].grad))
    leaf["x"].grad = None
    ss.conv1d_fn(leaf["x"], leaf["w"], leaf["bias"]).sum().backward()       # an expanded gradient, no final window
    torch.cuda.synchronize()
    _check_conv(dict(x=q["x"], w=q["w"], bias=q["bias"], dout=torch.ones(2, 6, 50)), dict(dx=leaf["x"].grad))


# ---- a layer, streams, graphs ---------------------------------------------------------------------


def test_layer_gradients_through_both():
    """conv1d_fn into ssd_scan_fn, as a Mamba-2 block trains: the chain's gradients by the two references.  The
    convolution's output is rounded to bf16 between them; the reference takes the rounded values."""
    ss = _ss()
    Bsz, L, H, G, N = 2, 270, 2, 1, 32
    ch = H * 64 + 2 * G * N
    q = _ssd(Bsz, L, H, G, N, "bf16", seed=12, docs=True)
    c = _conv(Bsz, ch, L, 4, "bf16", seed=13)
    ids = q["seq_idx"]
    x = c["x"].cuda().requires_grad_()
    w, b = c["w"].cuda().requires_grad_(), c["bias"].cuda().requires_grad_()
    mid = ss.conv1d_fn(x, w, b, seq_idx=ids.cuda())
    tm = mid.transpose(1, 2).contiguous()
    sx, sB, sC = (v.contiguous().view(Bsz, L, -1, n) for v, n in
                  ((tm[..., :H * 64], 64), (tm[..., H * 64:H * 64 + G * N], N), (tm[..., H * 64 + G * N:], N)))
    g = {k: v.cuda() for k, v in q.items()}
    y = ss.ssd_scan_fn(sx, g["dt"], g["A"], sB, sC, D=g["D"], dt_bias=g["dt_bias"], seq_idx=g["seq_idx"])
    mid.retain_grad()
    y.backward(g["dy"])
    torch.cuda.synchronize()
    p = {k: (v.numpy() if k == "seq_idx" else f64(v)) for k, v in q.items()}
    p.update(x=f64(sx.detach()), Bm=f64(sB.detach()), Cm=f64(sC.detach()))
    want, mag = ref.ssd_grad(p)
    cat = lambda d: np.concatenate([d[k].reshape(Bsz, L, -1) for k in ("dx", "dB", "dC")], 2).transpose(0, 2, 1)
    check(mid.grad, cat(want), cat(mag), "between")
    _check_conv(dict(c, seq_idx=ids, dout=mid.grad.cpu()), dict(dx=x.grad, dw=w.grad, dbias=b.grad))


def test_gradients_repeat_on_streams_and_in_graphs():
    """No sum depends on timing: repeated, on a side stream, two at once on two streams, and captured and replayed
    with eager work in between, all gradients are equal bit for bit."""
    ss = _ss()
    problems = [_ssd(2, 300, 4, 2, 64, "bf16", seed=20, state=True), _ssd(1, 530, 4, 1, 64, "f16", seed=21, gate=True,
                                                                         docs=True)]
    dev = [{k: v.cuda() for k, v in q.items()} for q in problems]
    conv = {k: v.cuda() for k, v in _conv(3, 40, 700, 4, "bf16", seed=22, docs=True, state=True).items()}

    def ssd(g):
        opt = {k: g.get(k) for k in ("D", "z", "dt_bias", "seq_idx", "h0", "dfinal")}
        return ss.ssd_bwd(g["x"], g["dt"], g["A"], g["Bm"], g["Cm"], g["dy"], want_dh0=True, **opt)

    run = [lambda: ssd(dev[0]), lambda: ssd(dev[1]), lambda: ss.conv1d_bwd(want_dconv_init=True, **conv)]
    want = [f() for f in run]
    same = lambda a, b: all(torch.equal(a[k], b[k]) for k in b)
    torch.cuda.synchronize()
    assert all(same(f(), v) for f, v in zip(run, want))
    streams = [torch.cuda.Stream() for _ in run]
    got = []
    for s, f in zip(streams, run):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(f())
    for s in streams:
        s.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        caught = [f() for f in run]
    for k in range(4):
        for d in caught:
            for v in d.values():
                v.fill_(float("nan"))
        dev[0]["dy"].mul_(-1.0)                          # another input, then back
        graph.replay()
        torch.cuda.synchronize()
        say("replay %d" % k)
        assert same(caught[1], want[1]) and same(caught[2], want[2])
        if k % 2:
            assert same(caught[0], want[0])
        run[k % 3]()
        torch.cuda.synchronize()


def test_training_step_captured_and_replayed():
    """Forward and backward of both operators through autograd inside one graph: every replay leaves the gradients
    that an eager pass over other leaves of the same values gives, new inputs among them."""
    ss = _ss()
    Bsz, L, H, N = 2, 270, 2, 32
    ch = H * 64 + 2 * N
    q = {k: v.cuda() for k, v in _ssd(Bsz, L, H, 1, N, "bf16", seed=31).items()}
    c = {k: v.cuda() for k, v in _conv(Bsz, ch, L, 4, "bf16", seed=32).items()}

    def leaves():
        return [c[k].clone().requires_grad_() for k in ("x", "w", "bias")] + [q["A"].clone().requires_grad_()]

    def step(x, w, b, A):
        tm = ss.conv1d_fn(x, w, b).transpose(1, 2)
        sx, sB, sC = (v.reshape(Bsz, L, -1, n) for v, n in zip(tm.split([H * 64, N, N], 2), (64, N, N)))
        y = ss.ssd_scan_fn(sx, q["dt"], A, sB, sC, D=q["D"], dt_bias=q["dt_bias"])
        y.backward(q["dy"])

    def eager(x):
        v = leaves()
        with torch.no_grad():
            v[0].copy_(x)
        step(*v)
        return [t.grad for t in v]

    inputs = [c["x"].clone(), c["x"].flip(2).contiguous(), c["x"].clone()]
    want = [eager(x) for x in inputs]
    torch.cuda.synchronize()
    mine = leaves()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*mine)
    for x, w in zip(inputs, want):
        with torch.no_grad():
            mine[0].copy_(x)
        graph.replay()
        eager(x)
        torch.cuda.synchronize()
        assert all(torch.equal(t.grad, v) for t, v in zip(mine, w))


def test_second_derivatives_and_strided_workspaces_are_refused():
    ss = _ss()
    c = {k: v.cuda() for k, v in _conv(1, 8, 40, 4, "f32", seed=33).items()}
    x = c["x"].requires_grad_()
    (dx,) = torch.autograd.grad(ss.conv1d_fn(x, c["w"], c["bias"]).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()
    q = {k: v.cuda() for k, v in _ssd(1, 40, 2, 1, 32, "bf16", seed=34).items()}
    x = q["x"].requires_grad_()
    (dx,) = torch.autograd.grad(ss.ssd_scan_fn(x, q["dt"], q["A"], q["Bm"], q["Cm"]).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()
    room = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        ss.ssd_bwd(q["x"].detach(), q["dt"], q["A"], q["Bm"], q["Cm"], q["dy"], workspace=room[::2])
    with pytest.raises(ValueError):
        ss.ssd_bwd(q["x"].detach(), q["dt"], q["A"], q["Bm"], q["Cm"], q["dy"], workspace=room.cpu())


@pytest.mark.parametrize("L", [3, 8, 9, 16, 21, 4096])
def test_conv_bwd_values_that_are_not_finite_stay_in_their_reach(L):
    """An infinity or NaN in x at one step of one row reaches the gradients of the steps that its window meets, its
    channel's dw and dbias, and nothing else."""
    ss = _ss()
    W, D = 4, 4
    q = _conv(2, D, L, W, "f32", seed=L)
    g = {k: v.cuda() for k, v in q.items()}
    clean = ss.conv1d_bwd(**g)
    for t in sorted({0, L // 2, max(L - 4, 0), L - 1}):
        for bad in (float("inf"), float("nan")):
            x = g["x"].clone()
            x[1, 2, t] = bad
            got = ss.conv1d_bwd(**dict(g, x=x))
            far = torch.ones(2, D, L, dtype=torch.bool, device="cuda")
            far[1, 2, max(t - (W - 1), 0):t + W] = False       # dpre of steps t .. t + W - 1, dx W - 1 before them
            assert torch.equal(got["dx"][far], clean["dx"][far]), (t, bad)
            others = [0, 1, 3]
            assert torch.equal(got["dw"][others], clean["dw"][others])
            assert torch.equal(got["dbias"][others], clean["dbias"][others])
