"""Linear attention in pieces at every pair of head sizes, and every sequence of a batch whose last walks alone are cut."""
import numpy as np
import pytest
import torch

import _linattn_ref as ref
import test_linattn_gpu as base
from _layer_ref import check
from _util import f64, say

pytestmark = pytest.mark.gpu

DIMS = [(2, 2, 64, 64), (2, 1, 64, 128), (2, 1, 128, 64), (2, 2, 128, 128)]


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,dk,dv", DIMS)
def test_prompts_in_pieces(io, H, G, dk, dv):
    say("pieces %s %d %d" % (io, dk, dv))
    q = base._problem([700, 129, 3, 0, 450], H, G, dk, dv, io, seed=120, lead=4, tail=2)
    q["has"][0] = 1
    g = base._dev(q)
    y = torch.full((q["T"], H, dv), 7.0, dtype=g["q"].dtype, device="cuda")
    base._ss().linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"], slots=g["slots"], has_state=g["has"], y=y)
    torch.cuda.synchronize()
    base._check_prompts(q, y, g["state"])


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,dk,dv", DIMS)
@pytest.mark.parametrize("state", [False, True])
def test_training_in_pieces(io, H, G, dk, dv, state):
    """Packed documents, and rows of one length."""
    say("pieces %s %d %d %s" % (io, dk, dv, state))
    q = base._problem([600, 0, 65, 300], H, G, dk, dv, io, seed=121, lead=1, tail=10)
    base._check_train(q, *base._train(q, 1, q["T"], True, state), state)
    q = base._problem([501, 501], H, G, dk, dv, io, seed=122)
    base._check_train(q, *base._train(q, 2, 501, False, state), state)


@pytest.mark.parametrize("io,G,dk,dv", [("bf16", 2, 64, 64), ("f16", 4, 128, 64)])
def test_every_walk_beyond_a_round(io, G, dk, dv):
    """22 rows of 4 heads, 264 walks of gradients: the 256 that run whole and the 8 in pieces, all of them."""
    B, L, H, at_once = 22, 1537, 4, 3
    say("walks beyond a round %s %d %d" % (io, dk, dv))
    q = base._problem([L] * B, H, G, dk, dv, io, seed=123)
    y, fin, gr = base._train(q, B, L, False, True)
    one = lambda t, b: np.concatenate([f64(t[i * L:(i + 1) * L]) for i in b], 1)       # sequences beside each other, as heads
    for b0 in range(0, B, at_once):
        b = range(b0, min(b0 + at_once, B))
        x = {n: one(q[n], b) for n in ("q", "k", "v")}
        g, h0, df = np.tile(f64(q["g"]), len(b)), np.concatenate(f64(q["h0"][b0:b0 + at_once])), np.concatenate(
            f64(q["df"][b0:b0 + at_once]))
        dy = one(q["dy"], b)
        a = np.abs
        both = lambda f, *r: zip(f(x["q"], x["k"], x["v"], g, q["scale"], h0, *r),
                                 f(a(x["q"]), a(x["k"]), a(x["v"]), g, q["scale"], a(h0), *(a(t) for t in r)))
        (wy, my), (wf, mf) = both(ref.linattn_rows)
        check(torch.cat([y[i * L:(i + 1) * L] for i in b], 1), wy, my, "y %d" % b0)
        check(fin[b0:b0 + at_once].flatten(0, 1), wf, mf, "final")
        for n, (w, m) in zip(("dq", "dk", "dv", "dh0"), both(ref.linattn_grads, dy, df)):
            got = gr[n][b0:b0 + at_once].flatten(0, 1) if n == "dh0" else torch.cat([gr[n][i * L:(i + 1) * L] for i in b], 1)
            check(got, w, m, n)
