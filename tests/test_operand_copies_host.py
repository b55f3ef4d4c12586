"""Operands that a call has to copy outlive its launch (CPU: the launch is replaced by a look at who owns each address)."""
import gc

import pytest
import torch

from mamba_selective_scan_fwd_amd import ss


@pytest.fixture
def launches(monkeypatch):
    """Every address that reaches a launch, with whether a tensor that is alive holds it."""
    seen = []

    def launch(dev, fn, problem, *args):
        spans = []
        for t in gc.get_objects():
            if issubclass(type(t), torch.Tensor):
                at = t.untyped_storage().data_ptr()
                spans.append((at, at + t.untyped_storage().nbytes()))
        for a in args:
            if isinstance(a, int) and a > 1 << 20:
                seen.append(any(lo <= a < hi for lo, hi in spans))

    monkeypatch.setattr(ss, "_device", lambda t: t.get_device())
    monkeypatch.setattr(ss, "_launch", launch)
    monkeypatch.setattr(ss, "_scratch", lambda ws, nbytes, dev: (None, None, nbytes))
    return seen


def _padded(*shape, dtype=torch.bfloat16):
    """(B, L, ..) of a batch padded to L + 3 rows: no even distance between its tokens."""
    return torch.zeros(shape[0], shape[1] + 3, *shape[2:], dtype=dtype)[:, :shape[1]]


def test_linattn_of_a_padded_batch(launches):
    q, k, v, dy = _padded(2, 70, 4, 64), _padded(2, 70, 2, 64), _padded(2, 70, 2, 128), _padded(2, 70, 4, 128)
    g = torch.zeros(4)
    ss.linattn_fwd(q, k, v, g)
    assert len(launches) >= 5 and all(launches)
    ss.linattn_bwd(q, k, v, g, dy)
    assert len(launches) >= 13 and all(launches)


@pytest.mark.parametrize("make", [_padded, lambda b, l, c: torch.zeros(b, c, l, dtype=torch.bfloat16).transpose(1, 2)])
def test_norm_of_a_padded_and_of_a_transposed_batch(launches, make):
    x, z, dy = make(2, 50, 96), make(2, 50, 96), make(2, 50, 96)
    w, b = torch.ones(96), torch.zeros(96)
    ss.group_norm(x, w, bias=b, z=z, ngroups=3)
    assert len(launches) >= 5 and all(launches)
    ss.group_norm_bwd(x, w, dy, bias=b, z=z, ngroups=3)
    assert len(launches) >= 14 and all(launches)
