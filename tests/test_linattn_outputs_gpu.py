"""What is asked for beside them does not change a gradient's bits where it has no part in it."""
import pytest
import torch

import test_linattn_gpu as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("G,dk,dv", [(2, 64, 64), (1, 128, 128), (2, 64, 128), (1, 128, 64)])
@pytest.mark.parametrize("B,L", [(3, 150), (1, 700)])
def test_dq_and_dk_without_dh0(io, G, dk, dv, B, L):
    ss = base._ss()
    q = base._problem([L] * B, 2, G, dk, dv, io, seed=110)
    g = base._dev(q)
    a = tuple(g[n].unflatten(0, (B, L)) for n in ("q", "k", "v")) + (g["g"], g["dy"].unflatten(0, (B, L)))
    with_, without = (ss.linattn_bwd(*a, h0=g["h0"], dfinal=g["df"], want_dh0=w) for w in (True, False))
    torch.cuda.synchronize()
    assert set(with_) - set(without) == {"dh0"}
    for n in ("dq", "dk"):
        assert torch.equal(with_[n], without[n]), n
    # dv's walk leaves dh0: its rows are added to the state in three bf16 parts for it, in two without
    d = (with_["dv"].float() - without["dv"].float()).abs()
    assert bool((d <= 2.0 ** -7 * with_["dv"].float().abs() + 2.0 ** -16 * float(with_["dv"].float().abs().max())).all())
