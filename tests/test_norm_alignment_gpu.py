"""The grouped norm of 16-bit rows on 8-byte boundaries: groups of 4 channels at a time, whatever their size."""
import pytest
import torch

import test_norm_pack_gpu as base
from _util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("C,groups", [(1536, 1), (96, 3), (4096, 1), (4104, 1), (20, 5)])
@pytest.mark.parametrize("start", [4, 2, 3])
def test_norm_at_part_of_a_vector(io, C, groups, start):
    """x, z and dy as columns from the 4th, 2nd and 3rd element of their rows on, of a multiple of 4, of 2 and odd."""
    say("norm %s %d in %d from %d" % (io, C, groups, start))
    for mode in ("gate", "gate_first"):
        q = base._draw(9, C, io, mode, seed=C)
        d = {k: v.cuda() for k, v in q.items()}
        for n in ("x", "z", "dy"):
            wide = torch.full((9, C + 8 + (start if start != 4 else 0)), 7.0, dtype=base.DT[io], device="cuda")
            wide[:, start:start + C] = d[n]
            d[n] = wide[:, start:start + C]
        base._both(q, groups, 1e-5, True, mode, dev=d)
