"""Gradients of so many rows that their tensors lie past 32 bits of bytes, without shared heads."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_gradients_of_many_rows():
    """256 equal sequences of 16384 rows and 17 heads, every operand 9 GB: what one gives the others give, to the bit."""
    from mamba_selective_scan_fwd_amd import ss
    S, L, H = 256, 16384, 17
    torch.manual_seed(90)
    one = torch.randn(1, L, H, 64, device="cuda").bfloat16()
    x = one.expand(S, L, H, 64).contiguous()
    g = -torch.logspace(-4, 0, H, device="cuda")
    y = ss.linattn_fwd(x, x, x, g)
    gr = ss.linattn_bwd(x, x, x, g, x)
    torch.cuda.synchronize()
    for t in (y, gr["dq"], gr["dk"], gr["dv"]):
        assert bool(torch.isfinite(t[0]).all()) and float(t[0].float().abs().max()) > 0
        for s in (1, S // 2, S - 1):
            assert torch.equal(t[s], t[0])
    del x, y, gr
    torch.cuda.empty_cache()
