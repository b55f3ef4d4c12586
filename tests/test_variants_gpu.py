"""GPU parity of the kernel variants that many rows, heads or prompts select: several heads per workgroup of the state
kernels (head counts that these divide and do not), several batches of heads in the gradients' pairs, prompts of many
chunks among short ones; dirty workspaces of exactly the stated size.  References and bounds as in test_serving_gpu.py
and test_layer_grad_gpu.py."""
import ctypes

import numpy as np
import pytest
import torch

import _plan
from _layer_ref import ELEMENT, check
from _util import f64, say
from test_layer_grad_gpu import DT, _bwd, _check_ssd, _conv, _ss, _ssd
from test_serving_gpu import _parts, _ssd_check, _ssd_problem, _step_args, _step_problem, _step_ref

pytestmark = pytest.mark.gpu


def _cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


MODES = [("bf16", False), ("bf16", True), ("f16", False), ("f16", True)]


# ---- gradients ------------------------------------------------------------------------


@pytest.mark.parametrize("io,gate", MODES)
@pytest.mark.parametrize("N", [32, 64, 96, 128])
@pytest.mark.parametrize("hb", [2, 3])
def test_ssd_bwd_heads_per_workgroup(io, gate, N, hb):
    """The last row of a batch that takes two or three heads per workgroup (its x and dy end with their allocation):
    16, 17 and 18 heads leave a workgroup none, one or two heads short."""
    ss = _ss()
    H = {32: 17, 64: 16, 96: 18, 128: 17}[N]
    B, L = (18, 70) if hb == 2 else (34, 70)
    assert _plan.bwd_heads(B, L, H, 1, _cus()) == hb
    say("bwd heads io=%s gate=%d N=%d H=%d hb=%d" % (io, gate, N, H, hb))
    q = _ssd(B, L, H, 1, N, io, seed=100 + N + hb, gate=gate, docs=True, state=True)
    got = _bwd(ss, q, want_dh0=True)
    torch.cuda.synchronize()
    rows = ("x", "dt", "Bm", "Cm", "dy", "z", "seq_idx", "h0", "dfinal")
    last = {k: v[-1:] if k in rows else v for k, v in q.items()}
    _check_ssd(last, {k: v[-1:] for k, v in got.items() if k in ("dx", "ddt", "dB", "dC", "dz", "dh0")})


@pytest.mark.parametrize("io,gate,B,L,H,G,hb", [
    ("bf16", False, 34, 70, 17, 1, 3), ("f16", True, 34, 70, 16, 1, 3), ("bf16", False, 9, 300, 17, 1, 2),
    ("bf16", True, 54, 40, 10, 2, 3)])
def test_ssd_bwd_heads_per_workgroup_all_rows(io, gate, B, L, H, G, hb):
    """Every output, the sums over all rows among them."""
    ss = _ss()
    assert _plan.bwd_heads(B, L, H, G, _cus()) == hb
    say("bwd rows io=%s B=%d L=%d H=%d" % (io, B, L, H))
    q = _ssd(B, L, H, G, 32, io, seed=B + L, gate=gate, docs=True, state=True)
    got = _bwd(ss, q, want_dh0=True)
    torch.cuda.synchronize()
    _check_ssd(q, got)


@pytest.mark.parametrize("io,gate", MODES)
@pytest.mark.parametrize("H", [15, 16, 17, 33])
def test_ssd_bwd_many_heads_of_a_group(io, gate, H):
    """More heads in a group than the pairs' kernel takes at once, over pieces on and off the diagonal."""
    ss = _ss()
    say("bwd group io=%s gate=%d H=%d" % (io, gate, H))
    q = _ssd(1, 290, H, 1, 32, io, seed=H, gate=gate, docs=H == 17)
    got = _bwd(ss, q)
    torch.cuda.synchronize()
    _check_ssd(q, got)


# ---- prompts ----------------------------------------------------------------------------


def _prompt(ss, q, H, G, N, own_x, io):
    """y and the pool; x in an allocation of its own (own_x), or a slice of wider rows."""
    g = {k: v.cuda() for k, v in q.items()}
    x, Bm, Cm = _parts(g["row"], H, G, N)
    x = x.contiguous() if own_x else x
    y = torch.zeros(x.shape, dtype=DT[io], device="cuda")
    ss.ssd_prompt(x, g["dt"], g["A"], Bm, Cm, g["cu"], g["state"], D=g.get("D"), z=g.get("z"), dt_bias=g["bias"], y=y,
                  slots=g["slots"], has_state=g["has"])
    torch.cuda.synchronize()
    return y, g["state"]


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("N", [32, 64, 96, 128])
@pytest.mark.parametrize("hb", [2, 3])
def test_ssd_prompt_heads_per_workgroup(io, N, hb):
    ss = _ss()
    H = {32: 17, 64: 16, 96: 18, 128: 17}[N]
    r = np.random.default_rng(N + hb)
    lens = r.integers(0, 50, 34 if hb == 2 else 64).tolist()
    lens[5], lens[-1] = 300, 65                          # two chunks; the last rows are the allocation's last
    T = sum(lens)
    assert _plan.prompt_heads(T, len(lens), H, 1, _cus()) == hb
    say("prompt heads io=%s N=%d H=%d hb=%d" % (io, N, H, hb))
    q = _ssd_problem(lens, H, 1, N, io, seed=N, gate=N != 64)
    y, state = _prompt(ss, q, H, 1, N, True, io)
    _ssd_check(q, H, 1, N, y, state)


@pytest.mark.parametrize("G,H,hb", [(2, 34, 3), (2, 10, 2), (4, 20, 3)])
def test_ssd_prompt_heads_per_workgroup_of_groups(G, H, hb):
    """Strided rows, several groups: a workgroup's heads end with its group's."""
    ss = _ss()
    lens = [20] * {(2, 34): 34, (2, 10): 60, (4, 20): 58}[(G, H)] + [257]
    assert _plan.prompt_heads(sum(lens), len(lens), H, G, _cus()) == hb
    q = _ssd_problem(lens, H, G, 32, "bf16", seed=G * H)
    y, state = _prompt(ss, q, H, G, 32, False, "bf16")
    _ssd_check(q, H, G, 32, y, state)


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("N", [32, 128])
def test_ssd_prompt_many_chunks_among_short_ones(io, N):
    """Prompts of 4 to 13 chunks between short ones: four chunks' states ahead, loaded again and again."""
    ss = _ss()
    H = 3
    lens = [7] * 12 + [1024, 1025, 0, 1500, 2048, 2049, 3300, 1] + [30] * 20
    assert _plan.prompt_ahead(sum(lens), len(lens), H, N, _cus()) == 4
    q = _ssd_problem(lens, H, 1, N, io, seed=N)
    q["A"] = torch.tensor([-0.02, -1.0, -8.0])           # a head that forgets little
    y, state = _prompt(ss, q, H, 1, N, False, io)
    _ssd_check(q, H, 1, N, y, state)


# ---- workspaces ----------------------------------------------------------------------------


def _rooms(need):
    """Workspaces of exactly `need` bytes inside larger buffers, with contents that are NaN, -1 or large numbers."""
    for fill in (0xFF, 0x7E, 0x00):
        room = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        yield room[:need], room[need:], fill


def _same_in_dirty_rooms(need, run, want):
    assert need > 0
    for ws, behind, fill in _rooms(need):
        got = run(ws)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), fill
        assert bool((behind == fill).all())


@pytest.mark.parametrize("io,gate", MODES)
def test_ssd_bwd_workspace_contents_do_not_matter(io, gate):
    ss = _ss()
    q = _ssd(2, 335, 6, 2, 64, io, seed=51, gate=gate, docs=True, state=True)
    pr = ss.ss_ssd_problem(2, 335, 6, 2, 64, 64, ss._IO[DT[io]], 1)
    need = ss.load_library().ss_ssd_bwd_workspace_size(ctypes.byref(pr), int(gate))
    run = lambda ws: list(_bwd(ss, q, want_dh0=True, workspace=ws).values())
    want = run(None)
    torch.cuda.synchronize()
    _same_in_dirty_rooms(need, run, want)


@pytest.mark.parametrize("io", ["bf16", "f16"])
def test_ssd_prompt_workspace_contents_do_not_matter(io):
    ss = _ss()
    H, G, N = 4, 2, 64
    q = _ssd_problem([70, 0, 300, 1, 600], H, G, N, io, seed=52)
    g = {k: v.cuda() for k, v in q.items()}
    x, Bm, Cm = _parts(g["row"], H, G, N)
    T, row = x.shape[0], g["row"].shape[1]

    def run(ws):
        state = g["state"].clone()
        y = torch.zeros(T, H, 64, dtype=DT[io], device="cuda")
        ss.ssd_prompt(x, g["dt"], g["A"], Bm, Cm, g["cu"], state, D=g["D"], z=g["z"], dt_bias=g["bias"], y=y,
                      slots=g["slots"], has_state=g["has"], workspace=ws)
        return y, state

    pr = ss.ss_ssd_prompt_problem(T, 5, g["state"].shape[0], H, G, row, row, row, H * 64, H, 64, N, ss._IO[DT[io]], 1)
    need = ss.load_library().ss_ssd_prompt_workspace_size(ctypes.byref(pr))
    want = run(None)
    torch.cuda.synchronize()
    _same_in_dirty_rooms(need, run, want)


def test_step_and_conv_bwd_workspace_contents_do_not_matter():
    ss = _ss()
    H, G, N = 4, 2, 64
    q = _step_problem(5, H, G, N, 4, "bf16", seed=53, slots=7)
    q["slots"][1] = -1                                    # a row that leaves its part of the workspace alone

    def run(ws):
        g, a = _step_args(q, H, G, N, True)
        y = torch.zeros(5, H, 64, dtype=torch.bfloat16, device="cuda")
        ss.ssd_step(slots=g["slots"], y=y, workspace=ws, **a)
        return y, g["state"], g["conv"]

    want = run(None)
    torch.cuda.synchronize()
    _same_in_dirty_rooms(5 * (H * 64 + 2 * G * N) * 4, run, want)
    g = {k: v.cuda() for k, v in _conv(3, 40, 2100, 4, "bf16", seed=54, docs=True, state=True).items()}
    conv = lambda ws: list(ss.conv1d_bwd(want_dconv_init=True, workspace=ws, **g).values())
    pr = ss.ss_conv_problem(3, 40, 2100, 4, ss.SS_BF16, 1, 0)
    want = conv(None)
    torch.cuda.synchronize()
    _same_in_dirty_rooms(ss.load_library().ss_conv1d_bwd_workspace_size(ctypes.byref(pr)), conv, want)


# ---- the step at width 3 ------------------------------------------------------------------------


@pytest.mark.parametrize("io", ["bf16", "f16"])
def test_ssd_step_width_3(io):
    ss = _ss()
    H, G, N = 4, 2, 64
    q = _step_problem(6, H, G, N, 3, io, seed=55, slots=9)
    q["slots"][4] = -1
    g, a = _step_args(q, H, G, N, True)
    y = torch.full((6, H, 64), 9.0, dtype=DT[io], device="cuda")
    ss.ssd_step(slots=g["slots"], y=y, **a)
    torch.cuda.synchronize()
    yr, ym, conv, state, sm = _step_ref(q, H, G, N, True, q["slots"].tolist())
    yr[4] = 9.0
    # all in fp32: a dozen roundings, and a sum of N
    check(y, yr, ym, "y", terms=2.0 ** -17)
    check(g["state"], state, sm, "state", terms=ELEMENT)
    assert np.array_equal(f64(g["conv"]), conv)
