"""Large steps followed by small ones: the decay between two neighbouring small steps is the exponential of a small
difference of large sums of Delta A, and has to keep fp32's accuracy all the same.  The references take every decay by
itself, step by step in 64 bits; bounds as in _layer_ref.py, whose share for the decays knows nothing of the sums."""
import numpy as np
import pytest
import torch

import _layer_ref as ref
import test_layer_grad_gpu as grad
import test_serving_gpu as serving
from _util import f64, say
from test_layer_grad_gpu import DT, _bwd, _check_ssd, _ss, _ssd
from test_serving_gpu import _ssd_check, _ssd_problem, _ssd_run

pytestmark = pytest.mark.gpu


def _check(got, want, mag, name, terms=ref.SUM):
    """_layer_ref.check for values past fp16's range: its largest value is 65504 and the step there is 32, so what
    is 65520 or more rounds to infinity.  An output whose reference is past that by more than its error has to be
    infinite, with the reference's sign; one within its error of it may be."""
    if got.dtype == torch.float16:
        want, mag = np.array(want, dtype=np.float64), np.array(mag, dtype=np.float64)
        past = np.abs(want) + terms * mag >= 65520.0
        must = np.abs(want) - terms * mag >= 65520.0
        g = f64(got)
        assert np.all(np.isinf(g[must]) & (np.sign(g[must]) == np.sign(want[must]))), name
        assert np.all(np.isinf(g[past]) | (np.abs(g[past] - want[past]) <= 2.0 ** -11 * np.abs(want[past])
                                           + terms * mag[past])), name
        got = got.cpu().clone()
        got[torch.from_numpy(past)] = 0.0
        want[past] = mag[past] = 0.0
    ref.check(got, want, mag, name, terms)


@pytest.fixture(autouse=True)
def _past_the_range(monkeypatch):
    monkeypatch.setattr(serving, "check", _check)
    monkeypatch.setattr(grad, "check", _check)


def _steps(T, large, period, first):
    """(T,) values of dt (softplus is near the identity for large ones): `first` of every `period` steps large."""
    t = torch.arange(T)
    return torch.where(t % period < first, torch.full((T,), large), -6.0 + 0.01 * (t % 13))


# stretches of small steps inside a piece of 64 steps, over its end, over two ends
PATTERNS = [(64, 32), (80, 48), (160, 30)]


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("large", [1.0, 8.0, 20.0, 1000.0])
@pytest.mark.parametrize("period,first", PATTERNS)
def test_ssd_prompt(io, large, period, first):
    ss = _ss()
    H, G, N = 2, 1, 32
    say("prompt io=%s large=%g period=%d" % (io, large, period))
    q = _ssd_problem([300, 64, 130], H, G, N, io, seed=int(large) + period, gate=False)
    T = q["dt"].shape[0]
    q["dt"] = _steps(T, large, period, first)[:, None].expand(T, H).contiguous().to(DT[io])
    q["A"], q["bias"] = torch.tensor([-16.0, -3.0]), torch.zeros(H)
    y = torch.zeros(T, H, 64, dtype=DT[io], device="cuda")
    state = _ssd_run(ss, q, H, G, N, y)
    _ssd_check(q, H, G, N, y, state)


@pytest.mark.parametrize("io,gate", [("bf16", False), ("bf16", True), ("f16", False), ("f16", True)])
@pytest.mark.parametrize("large", [1.0, 8.0, 20.0, 1000.0])
@pytest.mark.parametrize("period,first", PATTERNS)
def test_ssd_bwd(io, gate, large, period, first):
    ss = _ss()
    H, L = 2, 300
    say("bwd io=%s gate=%d large=%g period=%d" % (io, gate, large, period))
    q = _ssd(1, L, H, 1, 32, io, seed=int(large) + period, gate=gate, state=True)
    q["dt"] = _steps(L, large, period, first)[None, :, None].expand(1, L, H).contiguous().to(DT[io])
    q["A"], q["dt_bias"] = torch.tensor([-16.0, -3.0]), torch.zeros(H)
    got = _bwd(ss, q, want_dh0=True)
    torch.cuda.synchronize()
    _check_ssd(q, got)
