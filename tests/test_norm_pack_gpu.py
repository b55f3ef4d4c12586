"""GPU parity of the grouped norm and its gradients and of a serving batch's maps, and the new operators in one run."""
import numpy as np
import pytest
import torch

import _linattn_ref as ref
from _layer_ref import check
from _util import f64, say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# sums of a group, a tree over some 18 roundings, twice (mean, deviation), the root, SiLU's few units and the products
# behind: 64 roundings of 2^-24
FORWARD = 2.0 ** -18
# the same again for the two sums of the gradients and their products; sums over rows add up to 64 in a row and 16 of those
BACKWARD = 2.0 ** -16


def _ss():
    from mamba_selective_scan_fwd_amd import ss
    ss.load_library()
    return ss


def _draw(rows, C, io, mode, seed, mean=0.0, weight=True, bias=True):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s))
    return dict(x=(2 * t(rows, C) + mean).to(DT[io]), z=t(rows, C).to(DT[io]) if mode.startswith("gate") else None,
                dy=t(rows, C).to(DT[io]), w=(1 + 0.2 * t(C)).float() if weight else None,
                b=(0.2 * t(C)).float() if bias else None)


def _both(q, groups, eps, center, mode, dev=None):
    ss = _ss()
    d = dev or {k: v.cuda() if v is not None else None for k, v in q.items()}
    how = dict(bias=d["b"], z=d["z"], ngroups=groups, eps=eps, center=center, silu=mode == "silu", gate_first=mode == "gate_first")
    y = ss.group_norm(d["x"], d["w"], **how)
    g = ss.group_norm_bwd(d["x"], d["w"], d["dy"], **how)
    torch.cuda.synchronize()
    C = q["x"].shape[1]
    a = dict(x=f64(q["x"]), w=f64(q["w"]) if q["w"] is not None else np.ones(C),
             b=f64(q["b"]) if q["b"] is not None else np.zeros(C), z=f64(q["z"]) if q["z"] is not None else None)
    want, mag = ref.norm(**a, groups=groups, eps=eps, center=center, mode=mode)
    check(y, want, mag, "y", terms=FORWARD)
    grads = ref.norm_grads(**a, dy=f64(q["dy"]), groups=groups, eps=eps, center=center, mode=mode)
    assert set(g) == {k for k in grads if not (k == "dweight" and q["w"] is None or k == "dbias" and q["b"] is None)}
    for k, v in g.items():
        check(v, *grads[k], k, terms=BACKWARD)
    return y, g


MODES = ["plain", "silu", "gate", "gate_first"]


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("center", [False, True])
def test_norm(io, mode, center):
    """A group a head, odd groups, one group of a row, groups of one channel and rows of many groups."""
    for rows, C, groups in ((37, 128, 2), (5, 700, 7), (3, 1536, 1), (130, 48, 16), (2, 75, 3), (1, 64, 64)):
        say("norm %s %s %d rows of %d in %d" % (io, mode, rows, C, groups))
        _both(_draw(rows, C, io, mode, seed=C), groups, 1e-5, center, mode)


@pytest.mark.parametrize("io,C,groups", [("bf16", 2056, 1), ("f16", 8192, 1), ("f16", 8200, 1), ("bf16", 2061, 1), ("f32", 4096, 1),
                                         ("f32", 5000, 1), ("f32", 2050, 2), ("bf16", 16400, 2), ("f16", 12, 1)])
def test_norm_group_sizes(io, C, groups):
    """Groups of more than a wave's vectors, of more than a workgroup's, and odd ones element by element."""
    for rows, mode in ((3, "gate"), (70, "gate_first")):
        _both(_draw(rows, C, io, mode, seed=C), groups, 1e-5, True, mode)


def test_norm_many_rows():
    """Rows beyond one round of the workgroups."""
    _both(_draw(3001, 64, "f32", "silu", seed=1), 2, 1e-5, True, "silu")
    _both(_draw(40001, 8, "bf16", "plain", seed=2), 1, 1e-5, False, "plain")


def test_norm_without_weights_far_means_and_constant_rows():
    _both(_draw(9, 256, "f32", "plain", seed=3, mean=1000.0, weight=False, bias=False), 2, 1e-5, True, "plain")
    _both(_draw(9, 256, "bf16", "gate", seed=4, weight=False), 4, 1e-3, False, "gate")
    q = _draw(4, 64, "f32", "plain", seed=5, bias=False)
    q["x"][:] = 3.0
    _both(q, 2, 1e-5, True, "plain")
    q["x"][:] = 0.0
    _both(q, 2, 1e-5, False, "plain")


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("start", [0, 1, 8])
def test_norm_strided_rows(io, start):
    """Columns of wider rows, at odd elements too; nothing beside y is written; leading dimensions are rows."""
    ss = _ss()
    q = _draw(24, 64, io, "gate", seed=start)
    d = {k: v.cuda() for k, v in q.items()}
    for n in ("x", "z", "dy"):
        wide = torch.full((24, 64 + 16 + start), 7.0, dtype=DT[io], device="cuda")
        wide[:, start:start + 64] = d[n]
        d[n] = wide[:, start:start + 64]
    y, g = _both(q, 4, 1e-5, True, "gate", dev=d)
    out = torch.full((24, 90), 5.0, dtype=DT[io], device="cuda")
    at = out[:, start:start + 64]
    ss.group_norm(d["x"], d["w"], bias=d["b"], z=d["z"], ngroups=4, y=at)
    three = ss.group_norm(d["x"].unflatten(0, (4, 6)), d["w"], bias=d["b"], z=d["z"].unflatten(0, (4, 6)), ngroups=4)
    torch.cuda.synchronize()
    assert torch.equal(three.flatten(0, 1), y)
    # rows of 90 elements go element by element, whose lanes' sums come in another order
    want, mag = ref.norm(f64(q["x"]), f64(q["w"]), f64(q["b"]), f64(q["z"]), 4, 1e-5, True, "gate")
    check(at, want, mag, "y", terms=FORWARD)
    at.fill_(5.0)
    assert bool((out == 5.0).all())


def test_norm_rows_are_their_own():
    """A row that is not finite, and rows behind the last: nobody else sees them."""
    ss = _ss()
    q = _draw(40, 64, "bf16", "gate", seed=8)
    d = {k: v.cuda() for k, v in q.items()}
    how = dict(bias=d["b"], z=d["z"], ngroups=4)
    clean, gc = ss.group_norm(d["x"], d["w"], **how), ss.group_norm_bwd(d["x"], d["w"], d["dy"], **how)
    d["x"][7, 20] = float("inf")
    y, g = ss.group_norm(d["x"], d["w"], **how), ss.group_norm_bwd(d["x"], d["w"], d["dy"], **how)
    torch.cuda.synchronize()
    keep = torch.arange(40, device="cuda") != 7
    assert torch.equal(y[keep], clean[keep]) and torch.equal(g["dx"][keep], gc["dx"][keep])
    assert torch.equal(y[7, 32:], clean[7, 32:])         # other groups of that row
    assert not bool(torch.isfinite(y[7, 16:32]).all())


def test_group_norm_fn():
    ss = _ss()
    q = _draw(20, 96, "f32", "gate_first", seed=9)
    d = {k: v.cuda().requires_grad_() for k, v in q.items()}
    y = ss.group_norm_fn(d["x"], d["w"], d["b"], d["z"], ngroups=3, center=False, gate_first=True)
    y.backward(d["dy"].detach())
    g = ss.group_norm_bwd(d["x"].detach(), d["w"].detach(), d["dy"].detach(), bias=d["b"].detach(), z=d["z"].detach(), ngroups=3,
                          center=False, gate_first=True)
    torch.cuda.synchronize()
    for n, k in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("z", "dz")):
        assert torch.equal(d[n].grad, g[k])
    x = d["x"].detach().requires_grad_()
    ss.group_norm_fn(x, silu=True).sum().backward()
    assert x.grad is not None
    with pytest.raises(ValueError):
        ss.group_norm(d["x"].detach(), silu=True, z=d["z"].detach())
    with pytest.raises(ValueError):
        ss.group_norm(d["x"].detach(), gate_first=True)
    with pytest.raises(RuntimeError):
        ss.group_norm(d["x"].detach(), ngroups=5)
    with pytest.raises(ValueError):
        ss.group_norm(d["x"].detach(), d["w"].detach()[:50])


# ---- maps -------------------------------------------------------------------------------


def _pack(new, slots, seen, tokens):
    ss = _ss()
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    got = ss.pack_requests(i(new), i(slots), i(seen), tokens)
    torch.cuda.synchronize()
    want = ref.pack(new, slots, seen, tokens)
    assert set(got) == set(want)
    for k, v in want.items():
        assert np.array_equal(got[k].cpu().numpy(), v), k


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 255, 256, 257, 1000, 1024, 1025, 2500, 4095, 4096, 4097, 9000])
def test_pack(n):
    r = np.random.default_rng(n)
    new = np.where(r.random(n) < 0.6, 1, r.integers(0, 40, n))
    seen = r.integers(0, 3, n)
    slots = np.where(r.random(n) < 0.9, r.permutation(n), -1)
    total = int(new[slots >= 0].sum())
    for tokens in sorted({1, max(1, total // 3), max(1, total - 1), max(1, total), total + 77}):
        say("pack %d requests into %d rows" % (n, tokens))
        _pack(new.tolist(), slots.tolist(), seen.tolist(), tokens)


def test_pack_edges():
    """No rows at all, steps beyond the batch, lengths whose sum passes 32 bits, and negative numbers."""
    most = 2 ** 31 - 1
    _pack([0] * 70, list(range(70)), [5] * 70, 9)
    _pack([1] * 70, list(range(70)), [5] * 70, 9)
    _pack([1] * 70, [-1] * 70, [5] * 70, 9)
    _pack([most] * 2000, list(range(2000)), [0] * 2000, 10000)
    _pack([1, most, -4, most, 1, 3], [0, 1, 2, 3, 4, 5], [1, -7, 3, 2, 0, -1], 9000)
    _pack([20000, 1, 30000], [2, 1, 0], [4, 4, 0], 60000)


# ---- together ----------------------------------------------------------------------------


def test_a_serving_layer():
    """A batch's maps, linear attention of its single tokens and prompts and the norm behind, over three batches, eager
    and as one captured graph whose replays take new requests, against each request alone in 64 bits."""
    ss = _ss()
    R, T, H, d, io = 6, 200, 2, 64, torch.bfloat16
    r = np.random.default_rng(11)
    g = torch.tensor([-0.02, -0.3])
    w = torch.from_numpy(1 + 0.2 * r.standard_normal(H * d)).float()
    dev = dict(g=g.cuda(), w=w.cuda(), new=torch.zeros(R, dtype=torch.int32, device="cuda"),
               slots=torch.zeros(R, dtype=torch.int32, device="cuda"), seen=torch.zeros(R, dtype=torch.int32, device="cuda"),
               row=torch.zeros(T, 4 * H * d, dtype=io, device="cuda"), state=torch.zeros(R + 2, H, d, d, device="cuda"),
               y=torch.zeros(T, H, d, dtype=io, device="cuda"))

    def layer():
        m = ss.pack_requests(dev["new"], dev["slots"], dev["seen"], T)
        q, k, v = (dev["row"][:, i * H * d:(i + 1) * H * d].unflatten(1, (H, d)) for i in range(3))
        y = dev["y"]
        ss.linattn_prompt(q, k, v, dev["g"], m["cu_seqlens"], dev["state"], slots=m["prompt_slots"], has_state=m["has_state"], y=y)
        ss.linattn_step(q[:R], k[:R], v[:R], dev["g"], dev["state"], slots=m["step_slots"], y=y[:R])
        out = ss.group_norm(y.flatten(1), dev["w"], z=dev["row"][:, 3 * H * d:], ngroups=H)
        return m["rows"], m["taken"], out

    batches = [([40, 1, 0, 30, 7, 1], [0, 0, 0, 0, 0, 0]), ([1, 1, 50, 1, 1, 1], [40, 1, 0, 30, 7, 1]),
               ([1, 0, 100, 1, 90, 1], [41, 2, 50, 31, 8, 2])]
    slots = [3, 0, 7, 1, 5, 2]
    draws = [torch.from_numpy(r.standard_normal((T, 4 * H * d))).to(io) for _ in batches]

    def run(step):
        dev["state"].zero_()
        outs = []
        for (new, seen), row in zip(batches, draws):
            dev["new"].copy_(torch.tensor(new, dtype=torch.int32))
            dev["seen"].copy_(torch.tensor(seen, dtype=torch.int32))
            dev["slots"].copy_(torch.tensor(slots, dtype=torch.int32))
            dev["row"].copy_(row)
            outs.append([t.clone() for t in step()])
        torch.cuda.synchronize()
        return outs, dev["state"].clone()

    eager, state = run(layer)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer()

    def replay():
        graph.replay()
        return outs

    for _ in range(2):
        again, st = run(replay)
        assert torch.equal(st, state)
        for a, b, (new, _) in zip(again, eager, batches):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            n = int(a[1].sum())
            assert torch.equal(a[2][:n], b[2][:n])
    # each request alone
    hist = {i: [] for i in range(R)}
    for (new, seen), row, (rows, taken, out) in zip(batches, draws, eager):
        rows, taken = rows.tolist(), taken.tolist()
        assert taken == [min(n, t) for n, t in zip(new, taken)] and sum(taken) <= T
        for i in range(R):
            if not taken[i]:
                continue
            x = f64(row[rows[i]:rows[i] + taken[i]])
            hist[i].append(x)
            x = np.concatenate(hist[i])
            q, k, v = (x[:, j * H * d:(j + 1) * H * d].reshape(-1, H, d) for j in range(3))
            y, _ = ref.linattn_rows(q, k, v, f64(g), d ** -0.5, np.zeros((H, d, d)))
            y = y[-taken[i]:].reshape(-1, H * d)
            want, mag = ref.norm(y, f64(w), np.zeros(H * d), x[-taken[i]:, 3 * H * d:], H, 1e-5, True, "gate")
            # y is rounded to bf16 in between: half a step of it goes through the norm, whose gain the bound has
            check(out[rows[i]:rows[i] + taken[i]], want, mag, "request %d" % i, terms=2.0 ** -7)
