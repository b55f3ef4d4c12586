"""Linear attention where values of one channel are infinite or far from the others': the other channels hold their bounds."""
import numpy as np
import pytest
import torch

import _linattn_ref as ref
import test_linattn_gpu as base
from _layer_ref import check
from _util import f64, say

pytestmark = pytest.mark.gpu

IOS = ["f16", "bf16"]
LENS = {"whole": [200, 70], "pieces": [700, 70]}


def _prompts(g, q):
    y = torch.zeros(q["T"], *g["dy"].shape[1:], dtype=g["q"].dtype, device="cuda")
    base._ss().linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"], slots=g["slots"], has_state=g["has"], y=y)
    torch.cuda.synchronize()
    return y


def _prompts_want(q):
    st = f64(q["state"])
    h0s = [st[int(i)] * int(h) for i, h in zip(q["slots"], q["has"])]
    return base._forward(q, h0s)


def _others(n, bad):
    keep = np.ones(n, dtype=bool)
    keep[bad] = False
    return keep


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("H,G,dk,dv", [(2, 2, 64, 64), (2, 1, 128, 128), (2, 2, 64, 128), (2, 1, 128, 64)])
def test_an_infinite_value(io, lens, H, G, dk, dv):
    """An infinity in one channel of v: the other channels' y and states are those of v without it."""
    say("infinite v %s %s %d %d" % (io, lens, dk, dv))
    q = base._problem(LENS[lens], H, G, dk, dv, io, seed=70)
    q["has"][:] = 1
    q["v"][10, 0, 5] = 0.0
    g = base._dev(q)
    g["v"][10, 0, 5] = float("inf")
    y = _prompts(g, q)
    want, mag, last, lm = _prompts_want(q)
    ok = _others(dv, 5)
    check(y[:, :, ok], want[:, :, ok], mag[:, :, ok], "y")
    check(y[LENS[lens][0]:], want[LENS[lens][0]:], mag[LENS[lens][0]:], "y, the next")
    for s in range(2):
        i = int(q["slots"][s])
        check(g["state"][i][:, ok], last[s][:, ok], lm[s][:, ok], "state")
    bad = g["state"][int(q["slots"][0])][:H // G, 5]
    assert not bool(torch.isfinite(bad).any())           # and it shows where it is


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("lens", list(LENS))
def test_an_infinite_state(io, lens):
    """An infinity in one element of the state that enters: the other rows of it, and their y, are as without."""
    q = base._problem(LENS[lens], 2, 2, 64, 128, io, seed=71)
    q["has"][:] = 1
    q["g"] = torch.tensor([-0.02, -0.01])
    i = int(q["slots"][0])
    q["state"][i, 0, 7, 3] = 0.0
    g = base._dev(q)
    g["state"][i, 0, 7, 3] = float("inf")
    y = _prompts(g, q)
    want, mag, last, lm = _prompts_want(q)
    ok = _others(128, 7)
    check(y[:, :, ok], want[:, :, ok], mag[:, :, ok], "y")
    check(g["state"][i][:, ok], last[0][:, ok], lm[0][:, ok], "state")
    assert not bool(torch.isfinite(g["state"][i, 0, 7, 3]))


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("which", ["q", "k", "dy"])
def test_an_infinite_value_in_the_gradients(io, which):
    """An infinity in one channel of q, k or dy: the gradients' other channels that it does not meet are as without."""
    dims = (2, 2, 64, 128)
    q = base._problem([200, 150], *dims, io, seed=72)
    q[which][100, 0, 9] = 0.0
    g = base._dev(q)
    g[which][100, 0, 9] = float("inf")
    ss = base._ss()
    gr = ss.linattn_bwd(*(g[n].unsqueeze(0) for n in ("q", "k", "v")), g["g"], g["dy"].unsqueeze(0), cu_seqlens=g["cu"], h0=g["h0"],
                        dfinal=g["df"], want_dh0=True)
    torch.cuda.synchronize()
    # dq contracts dy and v and leaves k's channels, dk leaves q's, dv dy's; dh0 has dy's rows and q's columns
    clean = {"q": {"dq": None, "dk": 2, "dh0": 3}, "k": {"dk": None, "dq": 2, "dh0": None}, "dy": {"dv": 2, "dh0": 2}}[which]
    for s in range(2):
        a, b, p = base._rows(q, s)
        args = dict(p, g=f64(q["g"]), h0=f64(q["h0"])[s], dy=f64(q["dy"][a:b]), dfinal=f64(q["df"])[s])
        want = ref.linattn_grads(**args, scale=q["scale"])
        mag = ref.linattn_grads(**{n: np.abs(v) if n != "g" else v for n, v in args.items()}, scale=q["scale"])
        for i, n in enumerate(("dq", "dk", "dv", "dh0")):
            if n not in clean:
                continue
            got, w, m = (gr[n][0, a:b] if n != "dh0" else gr[n][s]), want[i], mag[i]
            axis = clean[n] - (1 if n == "dh0" else 0) if clean[n] is not None else None
            if axis is not None:
                ok = _others(w.shape[axis], 9)
                got, w, m = got.movedim(axis, 0)[ok], np.moveaxis(w, axis, 0)[ok], np.moveaxis(m, axis, 0)[ok]
            check(got, w, m, "%s of %d" % (n, s))


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("lens", list(LENS))
def test_channels_of_other_sizes(io, lens):
    """v's channels from 2^-12 to 2^12 and entering states' from 2^-30 to 2^30 times the usual: each is bounded by its own terms."""
    q = base._problem(LENS[lens], 2, 2, 64, 128, io, seed=73)
    q["has"][:] = 1
    of = lambda most: torch.tensor([2.0 ** ((p * 7) % (2 * most + 1) - most) for p in range(128)])
    q["v"] *= of(12).to(q["v"].dtype)
    q["state"] *= of(30)[:, None]
    g = base._dev(q)
    y = _prompts(g, q)
    want, mag, last, lm = _prompts_want(q)
    ok = np.abs(want).max((0, 1)) < 60000.0              # what fp16 holds
    check(y[:, :, ok], want[:, :, ok], mag[:, :, ok], "y")
    for s in range(2):
        check(g["state"][int(q["slots"][s])], last[s], lm[s], "state")


@pytest.mark.parametrize("io", IOS)
def test_terms_below_the_largest_of_their_channel(io):
    """Keys of zero behind the first rows, whose weights a strong decay then takes far below the others': bf16 holds its
    bounds there too, fp16 what its parts leave, 2^-38 of a channel's largest row for each of up to 64 of them."""
    q = base._problem([64, 100, 300], 3, 3, 64, 128, io, seed=74, g=torch.tensor([-0.05, -0.3, -0.7]))
    for a, n in zip((0, 64, 164), (64, 100, 300)):
        q["k"][a + 5:a + n] = 0
    g = base._dev(q)
    y = _prompts(g, q)
    want, mag, last, lm = _prompts_want(q)
    check(y, want, mag, "y")
    most = float(q["k"].abs().max()) * float(q["v"].abs().max())
    floor = 64 * 2.0 ** -38 * most if io == "f16" else 0.0
    for s in range(3):
        check(g["state"][int(q["slots"][s])], last[s], lm[s] + floor * 2.0 ** 15, "state")
