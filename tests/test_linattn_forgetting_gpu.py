"""Decays that forget within a chunk or a token, over rows that add nothing: what is left of the old state is its product
with the decay."""
import numpy as np
import pytest
import torch

import test_linattn_gpu as base
from _layer_ref import check
from _util import f64

pytestmark = pytest.mark.gpu

DECAYS = [-1e-3, -3.9e-3, -4e-3, -0.02, -0.15, -0.24, -0.3, -0.7]


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[64], [100], [200, 3, 64], [700]])
def test_chunks(io, lens):
    """Prompts whose keys are zero; 700 rows are walked in pieces."""
    q = base._problem(lens, len(DECAYS), 2, 64, 64, io, seed=80, g=torch.tensor(DECAYS))
    q["k"][:] = 0
    q["has"][:] = 1
    g = base._dev(q)
    y = base._ss().linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"], slots=g["slots"], has_state=g["has"])
    torch.cuda.synchronize()
    base._check_prompts(q, y, g["state"])


@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_gradients(io):
    """The gradients' states, from dfinal through rows whose q is zero, whole and in pieces."""
    for B, L in ((3, 150), (1, 700)):
        q = base._problem([L] * B, len(DECAYS), 2, 64, 128, io, seed=81, g=torch.tensor(DECAYS))
        q["q"][:] = 0
        q["k"][:, 0] = 0
        base._check_train(q, *base._train(q, B, L, False, True), True)


@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_tokens(io):
    """A token of zeros leaves exp(log_decay) times the state: one product of it, two roundings and the decay's few."""
    decays = [-1e-6, -0.1, -0.2499, -0.25, -0.5, -3.0, -8.0, -12.0, -16.5, -40.0, -60.0, -float("inf")]
    H, n = len(decays), 5
    st = torch.randn(n, H, 128, 64, generator=torch.Generator().manual_seed(82))
    x = torch.zeros(n, H, 64, dtype=base.DT[io], device="cuda")
    v = torch.ones(n, H, 128, dtype=base.DT[io], device="cuda")
    got = st.cuda()
    base._ss().linattn_step(x, x, v, torch.tensor(decays).cuda(), got)
    torch.cuda.synchronize()
    want = f64(st) * np.exp(f64(torch.tensor(decays)))[None, :, None, None]
    check(got, want, np.abs(want), "state", terms=2.0 ** -22)
