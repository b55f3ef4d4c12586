"""A batch's maps are tensors of their own: a change of one in place is none of another."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_outputs_change_alone():
    from mamba_selective_scan_fwd_amd import ss
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for n in (3, 4):                                     # with and without gaps between them
        new, slots, seen = i(2, 1, 70, 5)[:n], i(1, 0, 3, 2)[:n], i(0, 4, 0, 1)[:n]
        m = ss.pack_requests(new, slots, seen, 80)
        was = {k: (t.clone(), t._version) for k, t in m.items()}
        for k, t in m.items():
            t.add_(1)
            for j, u in m.items():
                if j != k:
                    assert u._version == was[j][1], (k, j)
            t.copy_(was[k][0])
            was[k] = was[k][0], t._version
        # a training step over the packed documents, with a map changed before its backward
        q = torch.randn(1, 80, 2, 64, device="cuda").bfloat16().requires_grad_()
        y = ss.linattn_fn(q, q.detach(), q.detach(), torch.full((2,), -0.1, device="cuda"), cu_seqlens=m["cu_seqlens"])
        m["rows"].add_(1)
        y.sum().backward()
        torch.cuda.synchronize()
        assert bool(torch.isfinite(q.grad).all())
