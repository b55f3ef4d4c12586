"""Padded and transposed batches, whose tokens lie at no even distance, give what their contiguous copies give."""
import pytest
import torch

from _util import say

pytestmark = pytest.mark.gpu


def _ss():
    from mamba_selective_scan_fwd_amd import ss
    ss.load_library()
    return ss


def _padded(*shape, dtype=torch.bfloat16):
    return torch.randn(shape[0], shape[1] + 3, *shape[2:], device="cuda").to(dtype)[:, :shape[1]]


def _transposed(*shape, dtype=torch.bfloat16):
    return torch.randn(shape[1], shape[0], *shape[2:], device="cuda").to(dtype).transpose(0, 1)


def _equal(a, b):
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("make", [_padded, _transposed])
@pytest.mark.parametrize("L", [50, 700])
def test_linattn(make, L):
    ss = _ss()
    say("linattn %s %d" % (make.__name__, L))
    q, k, v, dy = make(3, L, 4, 64), make(3, L, 2, 64), make(3, L, 2, 64), make(3, L, 4, 64)
    h0, df = (make(3, 4, 64, 64, dtype=torch.float32) for _ in range(2))
    g = torch.tensor([-0.5, -0.1, -0.01, -0.001], device="cuda")

    def work(c):
        q_, k_, v_, dy_, h_, f_ = (c(t).detach() for t in (q, k, v, dy, h0, df))
        y, fin = ss.linattn_fwd(q_, k_, v_, g, h0=h_, return_final_state=True)
        gr = ss.linattn_bwd(q_, k_, v_, g, dy_, h0=h_, dfinal=f_, want_dh0=True)
        leaves = [t.requires_grad_() for t in (q_, k_, v_, h_)]
        z, last = ss.linattn_fn(q_, k_, v_, g, h0=h_, return_final_state=True)
        auto = torch.autograd.grad([z, last], leaves, [dy_, f_])
        return [y, fin, *(gr[n] for n in ("dq", "dk", "dv", "dh0")), z.detach(), *auto]

    want = work(lambda t: t.contiguous())
    _equal(work(lambda t: t), want)
    _equal(want[2:6], want[7:])


@pytest.mark.parametrize("make", [_padded, _transposed])
@pytest.mark.parametrize("C", [96, 75])
@pytest.mark.parametrize("first", [False, True])
def test_norm(make, C, first):
    ss = _ss()
    say("norm %s %d" % (make.__name__, C))
    x, z, dy = make(3, 50, C), make(3, 50, C), make(3, 50, C)
    w, b = torch.randn(C, device="cuda"), torch.randn(C, device="cuda")

    def work(c):
        kw = dict(bias=b, z=c(z), ngroups=3, gate_first=first)
        g = ss.group_norm_bwd(c(x), w, c(dy), **kw)
        return [ss.group_norm(c(x), w, **kw), *(g[n] for n in ("dx", "dweight", "dbias", "dz"))]

    _equal(work(lambda t: t), work(lambda t: t.contiguous()))
