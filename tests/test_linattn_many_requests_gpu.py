"""Linear attention over the maps of large batches: hundreds of sequences in pieces, most of them empty behind the last row."""
import numpy as np
import pytest
import torch

import test_linattn_gpu as base
from _util import say

pytestmark = pytest.mark.gpu


def _prompts(q):
    H, G, dk, dv = q["dims"]
    g = base._dev(q)
    y = torch.full((q["T"], H, dv), 7.0, dtype=g["q"].dtype, device="cuda")
    base._ss().linattn_prompt(g["q"], g["k"], g["v"], g["g"], g["cu"], g["state"], scale=q["scale"], slots=g["slots"],
                              has_state=g["has"], y=y)
    torch.cuda.synchronize()
    base._check_prompts(q, y, g["state"])


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("lead,tail", [(0, 0), (700, 30)])
def test_empty_sequences_behind_the_last_row(io, lead, tail):
    """Some 500 of them, half with a slot: kept where it is carried, else cleared; rows of no sequence before the first."""
    say("empty sequences %s %d" % (io, lead))
    q = base._problem([300, 0, 1, 900, 64, 77] + [0] * 501, 2, 1, 64, 64, io, seed=100, lead=lead, tail=tail)
    q["slots"][7::2] = -1
    _prompts(q)


@pytest.mark.parametrize("H,lens", [(2, None), (16, None), (16, [900, 0, 2000, 130])])
def test_pieces_over_many_ends(H, lens):
    """Fewer sequences than pieces and more of them; those in several pieces found from either side."""
    r = np.random.default_rng(101)
    lens = lens or r.integers(0, 180, 45).tolist() + [700] + [0] * 9
    _prompts(base._problem(lens, H, H // 2, 64, 64, "bf16", seed=102, lead=3, tail=1))


@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_training_with_empty_documents(io):
    """Their first states are their last ones, and their gradients likewise."""
    q = base._problem([700, 300, 0, 9] + [0] * 130, 2, 1, 64, 128, io, seed=103, lead=1, tail=10)
    base._check_train(q, *base._train(q, 1, 1020, True, True), True)
    q = base._problem([0] * 70, 2, 2, 64, 64, io, seed=104, lead=500, tail=0)      # no rows at all
    base._check_train(q, *base._train(q, 1, 500, True, True), True)


def test_offsets_out_of_order():
    """Calls that end, with more sequences than pieces, and guard rows and slots that stay."""
    ss = base._ss()
    H, T, S = 16, 3000, 200
    q = base._problem([T], H, H, 64, 64, "bf16", seed=105)
    g = base._dev(q)
    r = np.random.default_rng(106)
    for cu in (r.integers(-50, T + 50, S + 1), np.sort(r.integers(0, T, S + 1))[::-1].copy(),
               np.concatenate([np.sort(r.integers(0, T, S)), [5]])):
        bad = torch.from_numpy(cu.astype(np.int32)).cuda()
        guard = torch.full((T + 20, H, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        pool = torch.full((S + 2, H, 64, 64), 3.0, device="cuda")
        ss.linattn_prompt(g["q"], g["k"], g["v"], g["g"], bad, pool[1:-1], y=guard[10:-10])
        a = tuple(g[n].unsqueeze(0) for n in ("q", "k", "v")) + (g["g"],)
        ss.linattn_bwd(*a, g["dy"].unsqueeze(0), cu_seqlens=bad, want_dh0=True)
        torch.cuda.synchronize()
        assert bool((guard[:10] == 7).all()) and bool((guard[-10:] == 7).all())
        assert bool((pool[0] == 3).all()) and bool((pool[-1] == 3).all())


def test_maps_of_a_large_batch():
    """pack_requests' output as it is, thousands of requests: what its prompts alone give."""
    ss = base._ss()
    R, T, H = 40000, 6000, 12
    r = np.random.default_rng(107)
    kind = r.random(R)
    new = np.where(kind < 0.05, 1, np.where(kind < 0.99, 0, r.integers(1, 60, R)))
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()
    m = ss.pack_requests(i32(new), i32(r.permutation(R) % 500), i32(r.integers(0, 9, R)), T)
    n = int((m["prompt_slots"] >= 0).sum())
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    every = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    every[:n] = slots
    torch.manual_seed(108)
    row = torch.randn(T, H, 3, 64, device="cuda").bfloat16()
    q, k, v = (row[:, :, i].contiguous() for i in range(3))
    g = -torch.logspace(-4, -0.2, H, device="cuda")
    out = []
    for cu, s, has in ((m["cu_seqlens"], every, m["has_state"]), (m["cu_seqlens"][:n + 1], slots, m["has_state"][:n])):
        st = torch.ones(n, H, 64, 64, device="cuda")
        y = torch.zeros(T, H, 64, dtype=torch.bfloat16, device="cuda")
        ss.linattn_prompt(q, k, v, g, cu, st, slots=s, has_state=has, y=y)
        out.append((y, st))
    torch.cuda.synchronize()
    assert 0 < n < R and int(m["cu_seqlens"][n]) > 2000
    y, st = out[0]
    z, su = out[1]
    # the pieces' ends lie elsewhere, so that states differ by their roundings
    assert float((y.float() - z.float()).abs().max()) <= 2.0 ** -7 * float(z.float().abs().max())
    assert float((st - su).abs().max()) <= 2.0 ** -18 * float(su.abs().max())


@pytest.mark.parametrize("lens", [[300, 0, 1, 900, 64] + [0] * 300, [900, 300, 5]])
def test_workspaces_of_exactly_their_size(lens):
    """Whatever they hold, and nothing behind them is written."""
    ss = base._ss()
    q = base._problem(lens, 2, 1, 64, 128, "bf16", seed=109, lead=3, tail=2)
    g = base._dev(q)
    a = (g["q"], g["k"], g["v"], g["g"], g["cu"])
    rows = tuple(t.unsqueeze(0) for t in a[:3]) + (g["g"], g["dy"].unsqueeze(0))
    kw = dict(cu_seqlens=g["cu"], h0=g["h0"], dfinal=g["df"], want_dh0=True)

    def sizes():
        pr = ss.ss_linattn_problem(q["T"], len(lens), len(lens) + 2, 2, 1, a[0].stride(0), a[1].stride(0), a[2].stride(0), 64, 128, 2,
                                   1, 0.125, 0)
        lib, p = ss.load_library(), ss.ctypes.byref(pr)
        return lib.ss_linattn_workspace_size(p), lib.ss_linattn_bwd_workspace_size(p)

    outs = []
    for fill in (None, 0xff, 0x7f):
        st = g["state"].clone()
        wide = [None, None] if fill is None else [torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda") for n in sizes()]
        ws = [None if w is None else w[:-512] for w in wide]
        y = torch.zeros(q["T"], 2, 128, dtype=torch.bfloat16, device="cuda")
        ss.linattn_prompt(*a, st, slots=g["slots"], has_state=g["has"], y=y, workspace=ws[0])
        gr = ss.linattn_bwd(*rows, workspace=ws[1], **kw)
        torch.cuda.synchronize()
        outs.append([y, st, *gr.values()])
        for w in wide:
            assert w is None or bool((w[-512:] == fill).all())
    for o in outs[1:]:
        for x, z in zip(o, outs[0]):
            assert torch.equal(x, z)
