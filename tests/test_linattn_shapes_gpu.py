"""k, v, y and dy of other rows than q's are refused, also where their product is the same."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_rows_of_other_shapes():
    from mamba_selective_scan_fwd_amd import ss
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    q, kv, g = t(2, 64, 2, 64), t(2, 64, 2, 64), torch.zeros(2, device="cuda")
    for other in (t(4, 32, 2, 64), t(1, 128, 2, 64), t(64, 2, 2, 64)):
        for call in (ss.linattn_fwd, ss.linattn_fn, lambda *a: ss.linattn_bwd(*a, q)):
            with pytest.raises(ValueError):
                call(q, other, kv, g)
            with pytest.raises(ValueError):
                call(q, kv, other, g)
            with pytest.raises(ValueError):
                call(q, other, other, g)
        with pytest.raises(ValueError):
            ss.linattn_bwd(q, kv, kv, g, other)
    ss.linattn_fwd(q, kv, kv, g)
    torch.cuda.synchronize()
