"""Workspaces that a prepared call owns belong to the stream that its launches go to: the allocator's block is that
stream's, so no other stream's tensor shares its memory while launches are queued, before the call or after it is
dropped."""
import pytest
import torch

from test_serving_gpu import _ss, _step_args, _step_problem

pytestmark = pytest.mark.gpu


def _stream_of(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not an allocation of torch's")


def test_step_call_workspace_is_its_streams():
    ss = _ss()
    q = _step_problem(3, 2, 1, 64, 4, "bf16", seed=61, slots=4)
    _, a = _step_args(q, 2, 1, 64, True)
    y = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    call = ss.SsdStepCall(y=y, stream=side, **a)
    assert _stream_of(call.ws) == side.cuda_stream
    mine = ss.SsdStepCall(y=y, **a)
    assert _stream_of(mine.ws) == torch.cuda.current_stream().cuda_stream
    side.wait_stream(torch.cuda.current_stream())
    call()                                            # and runs there, with what the default stream's gives
    del call
    side.synchronize()
    _, b = _step_args(q, 2, 1, 64, True)
    want = torch.empty_like(y)
    ss.SsdStepCall(y=want, **b)()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(a["state"], b["state"])


def test_forward_call_workspace_is_its_streams():
    ss = _ss()
    t = lambda *s: torch.randn(*s, device="cuda")
    u, delta, B, C, A = t(1, 32, 4096), t(1, 32, 4096), t(1, 16, 4096), t(1, 16, 4096), -torch.rand(32, 16, device="cuda")
    y = torch.zeros_like(u)
    side = torch.cuda.Stream()
    call = ss.FwdCall(u, delta, A, B, C, y=y, stream=side)      # few channels: time is split, over a workspace
    assert _stream_of(call.ws) == side.cuda_stream
    side.wait_stream(torch.cuda.current_stream())
    call()
    del call
    side.synchronize()
    want = torch.empty_like(u)
    ss.FwdCall(u, delta, A, B, C, y=want)()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
