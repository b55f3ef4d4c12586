"""Host-side checks of linear attention's, the grouped norm's and the batch maps' C ABI (no GPU): every refusal returns
before any HIP call."""
import ctypes

import pytest
import torch

from mamba_selective_scan_fwd_amd import ss

G = 1 << 34  # far-apart, aligned stand-in addresses; never dereferenced (validation fails first)
R = ctypes.byref


def _lin(**kw):
    d = dict(tokens=700, nseqs=3, nslots=4, nheads=4, kv_heads=2, q_stride=1024, k_stride=1024, v_stride=1024, dk=64, dv=128,
             io_dtype=2, packed=1, scale=0.125, reserved=0)
    d.update(kw)
    return ss.ss_linattn_problem(*(d[n] for n, _ in ss.ss_linattn_problem._fields_))


# q, k and v side by side in rows of 1024: 256, 128 and 256 columns
A = dict(q=G, k=G + 512, v=G + 768, g=2 * G, cu=3 * G, slots=4 * G, has=None, h0=None, state=5 * G, y=6 * G, fin=7 * G, ws=8 * G,
         dy=9 * G, dfinal=None, dq=10 * G, dk=11 * G, dv=12 * G, dh0=None)


def _calls(p, wsz=1 << 40, **kw):
    """The codes of the forward, the prompts, the backward and the step."""
    a, lib = dict(A, **kw), ss.load_library()
    p = R(p) if p is not None else None
    return (lib.ss_linattn_fwd(p, a["q"], a["k"], a["v"], a["g"], a["cu"], a["h0"], a["y"], a["fin"], a["ws"], wsz, None),
            lib.ss_linattn_prompt(p, a["q"], a["k"], a["v"], a["g"], a["cu"], a["slots"], a["has"], a["state"], a["y"],
                                  a["ws"], wsz, None),
            lib.ss_linattn_bwd(p, a["q"], a["k"], a["v"], a["g"], a["cu"], a["h0"], a["dy"], a["dfinal"], a["dq"], a["dk"],
                               a["dv"], a["dh0"], a["ws"], wsz, None),
            lib.ss_linattn_step(p, a["q"], a["k"], a["v"], a["g"], a["slots"], a["state"], a["y"], None))


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), 2), (dict(tokens=(1 << 30) + 1), 2), (dict(nheads=0), 2), (dict(kv_heads=0), 2), (dict(q_stride=255), 2),
    (dict(k_stride=127), 2), (dict(v_stride=255), 2), (dict(v_stride=(1 << 21) + 8), 2), (dict(io_dtype=0), 3),
    (dict(io_dtype=7), 3), (dict(dk=32), 5), (dict(dv=96), 5), (dict(dk=256, q_stride=1024), 5), (dict(kv_heads=3), 5),
    (dict(packed=2), 5), (dict(reserved=1), 5),
    (dict(nheads=1 << 15, kv_heads=1, q_stride=1 << 21, dk=64), 5)])
def test_linattn_rejects_bad_problem(kw, code):
    p = _lin(**kw)
    lib = ss.load_library()
    assert lib.ss_linattn_workspace_size(R(p)) == 0 and lib.ss_linattn_bwd_workspace_size(R(p)) == 0
    assert _calls(p) == (code,) * 4


@pytest.mark.parametrize("kw,code", [
    (dict(nseqs=0), 2), (dict(nseqs=(1 << 20) + 1), 2), (dict(nseqs=1 << 20, nheads=1 << 13, q_stride=1 << 20), 2),
    (dict(q_stride=1028), 4), (dict(k_stride=1028), 4), (dict(v_stride=1028), 4)])
def test_linattn_sequences_reject_bad_problem(kw, code):
    p = _lin(**kw)
    assert ss.load_library().ss_linattn_workspace_size(R(p)) == 0
    assert _calls(p)[:3] == (code,) * 3


def test_linattn_rejects_bad_pointers():
    p = _lin()
    assert _calls(None) == (1,) * 4
    for name, which in (("q", "fpbs"), ("k", "fpbs"), ("v", "fpbs"), ("g", "fpbs"), ("cu", "fpb"), ("y", "fps"), ("state", "ps"),
                        ("dy", "b"), ("dq", "b"), ("dk", "b"), ("dv", "b")):
        got = _calls(p, **{name: None})
        assert all(got["fpbs".index(c)] == 1 for c in which), name
    assert _calls(_lin(packed=0, tokens=699))[0] == 1                                # offsets that the problem does not name
    assert _calls(_lin(packed=0))[0] == 2 and _calls(_lin(packed=0, nseqs=7), cu=None)[1] == 1
    for name, which in (("q", "fpb"), ("k", "fpb"), ("v", "fpb"), ("g", "fpbs"), ("cu", "fpb"), ("slots", "ps"), ("has", "p"),
                        ("h0", "fb"), ("state", "ps"), ("y", "fps"), ("fin", "f"), ("ws", "fpb"), ("dy", "b"), ("dfinal", "b"),
                        ("dq", "b"), ("dk", "b"), ("dv", "b"), ("dh0", "b")):
        got = _calls(p, **{name: 13 * G + 8})
        assert all(got["fpbs".index(c)] == 4 for c in which), name
    assert _calls(p, q=G + 1)[3] == 4                                               # the step takes elements, not bytes
    got = _calls(_lin(nslots=2), slots=None)
    assert got[1] == 5 and got[3] == 5                                              # fewer slots than sequences or rows
    assert _calls(_lin(nslots=0))[1] == 2 and _calls(_lin(nslots=0))[3] == 2


def test_linattn_workspace_and_overlaps():
    lib, p = ss.load_library(), _lin()
    fwd, bwd = lib.ss_linattn_workspace_size(R(p)), lib.ss_linattn_bwd_workspace_size(R(p))
    assert fwd > 0 and bwd >= 3 * fwd // 2
    # shared heads' parts: (tokens, nheads, dk + dv) fp32
    alone = lib.ss_linattn_bwd_workspace_size(R(_lin(kv_heads=4)))
    assert bwd - alone == (700 * 4 * 192 * 4 + 255) // 256 * 256
    # rows enough to fill the GPU are not split: no workspace
    assert lib.ss_linattn_workspace_size(R(_lin(packed=0, tokens=2048 * 64, nseqs=64, nheads=8, q_stride=1024))) == 0
    assert _calls(p, wsz=fwd - 1)[:2] == (5, 5) and _calls(p, wsz=bwd - 1)[2] == 5 and _calls(p, ws=None)[:3] == (5,) * 3
    for k, v in (("y", G), ("y", G + 512), ("ws", 6 * G), ("fin", 6 * G), ("ws", G)):
        assert _calls(p, **{k: v})[0] == 5, k
    for k, v in (("y", G), ("state", G + 768), ("state", 6 * G), ("ws", 5 * G), ("y", 3 * G)):
        assert _calls(p, **{k: v})[1] == 5, k
    for k, v in (("dq", G), ("dk", 10 * G), ("dv", 9 * G), ("dh0", 12 * G), ("ws", 11 * G)):
        assert _calls(p, **{k: v})[2] == 5, k
    assert _calls(p, y=G)[3] == 5 and _calls(p, state=6 * G)[3] == 5


@pytest.mark.parametrize("nseqs,length,packed,pieces", [
    (1, 384, 0, 0), (1, 385, 0, 4), (1, 5000, 0, 40), (4, 4096, 0, 4 * 32), (1, 1 << 20, 0, 128), (64, 4096, 0, 64 * 2),
    (65, 4096, 0, 32), (65, 1536, 0, 12), (65, 1472, 0, 0), (80, 4096, 0, 16 * 4), (81, 4096, 0, 0), (128, 4096, 0, 0),
    (64, 4096, 1, -(-(4096 + 64) // 33)), (3, 130, 1, 5)])
def test_linattn_pieces(nseqs, length, packed, pieces):
    """Short sequences are walked whole; else in pieces of 128 rows or more, two workgroups of the 4 heads to a CU, those of
    packed sequences over their ends.  Where there are more walks than CUs, those beyond the last multiple of these
    are cut if they are a quarter at most: two states of every head each."""
    p = _lin(packed=packed, tokens=nseqs * length, nseqs=nseqs)
    assert ss.load_library().ss_linattn_workspace_size(R(p)) == 2 * pieces * 4 * 64 * 128 * 4


def _norm(**kw):
    d = dict(rows=10, channels=48, ngroups=4, x_stride=96, z_stride=96, y_stride=48, dy_stride=48, eps=1e-5, io_dtype=2, mode=2,
             center=1)
    d.update(kw)
    return ss.ss_norm_problem(*(d[n] for n, _ in ss.ss_norm_problem._fields_))


def _norm_calls(p, wsz=1 << 40, **kw):
    a = dict(x=G, w=2 * G, b=3 * G, z=4 * G, y=5 * G, dy=6 * G, dx=7 * G, dw=8 * G, db=9 * G, dz=10 * G, ws=11 * G)
    a.update(kw)
    lib, p = ss.load_library(), R(p) if p is not None else None
    return (lib.ss_group_norm(p, a["x"], a["w"], a["b"], a["z"], a["y"], None),
            lib.ss_group_norm_bwd(p, a["x"], a["w"], a["b"], a["z"], a["dy"], a["dx"], a["dw"], a["db"], a["dz"], a["ws"], wsz,
                                  None))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), 2), (dict(channels=0), 2), (dict(ngroups=0), 2), (dict(rows=(1 << 30) + 1), 2), (dict(x_stride=47), 2),
    (dict(z_stride=47), 2), (dict(x_stride=(1 << 21) + 1), 2), (dict(io_dtype=3), 3), (dict(ngroups=5), 5), (dict(mode=4), 5),
    (dict(mode=-1), 5), (dict(eps=-1.0), 5), (dict(eps=float("nan")), 5), (dict(mode=0), 1), (dict(mode=1), 1)])
def test_norm_rejects_bad_problem(kw, code):
    assert _norm_calls(_norm(**kw)) == (code, code)


def test_norm_rejects_bad_pointers():
    p = _norm()
    assert _norm_calls(None) == (1, 1)
    for k, i in (("x", (0, 1)), ("z", (0, 1)), ("y", (0,)), ("dy", (1,)), ("dx", (1,)), ("dz", (1,)), ("dw", (1,)), ("db", (1,)),
                 ("w", (1,)), ("b", (1,))):
        assert all(_norm_calls(p, **{k: None})[j] == 1 for j in i), k
    for k, i in (("x", (0, 1)), ("z", (0, 1)), ("y", (0,)), ("dy", (1,)), ("dx", (1,)), ("dz", (1,))):
        assert all(_norm_calls(p, **{k: 20 * G + 1})[j] == 4 for j in i), k
    for k, i in (("w", (0, 1)), ("b", (0, 1)), ("dw", (1,)), ("db", (1,)), ("ws", (1,))):
        assert all(_norm_calls(p, **{k: 20 * G + 4})[j] == 4 for j in i), k
    assert _norm_calls(_norm(y_stride=47))[0] == 2 and _norm_calls(_norm(dy_stride=47))[1] == 2
    need = ss.load_library().ss_group_norm_bwd_workspace_size(R(p))
    assert need == 10 * 48 * 8
    assert _norm_calls(p, wsz=need - 1)[1] == 5 and _norm_calls(p, ws=None)[1] == 5
    assert _norm_calls(p, y=G)[0] == 5 and _norm_calls(p, y=G + 96)[0] == 5          # y between x's rows
    for k, v in (("dx", G), ("dz", 7 * G), ("dw", 9 * G), ("ws", 6 * G), ("db", 2 * G)):
        assert _norm_calls(p, **{k: v})[1] == 5, k


def test_pack_rejects():
    lib = ss.load_library()

    def call(n=10, t=40, **kw):
        at = {i: (i + 1) * G for i in range(11)}
        at.update(kw.get("at", {}))
        return lib.ss_pack_requests(n, t, *(at[i] for i in range(11)), None)

    assert call(n=0) == 2 and call(t=0) == 2 and call(n=(1 << 20) + 1) == 2 and call(t=(1 << 30) + 1) == 2
    for i in range(11):
        assert call(at={i: None}) == 1 and call(at={i: 20 * G + 4}) == 4, i
    assert call(at={3: G}) == 5 and call(at={9: 11 * G}) == 5 and call(at={4: 4 * G + 16}) == 5


def test_python_refuses_host_tensors_and_types():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    g = torch.zeros(4)
    with pytest.raises(ValueError):
        ss.linattn_step(x, x, x, g, torch.zeros(2, 4, 64, 64))
    with pytest.raises(TypeError):
        ss.linattn_fwd(x.float()[None], x.float()[None], x.float()[None], g)
    with pytest.raises(ValueError):
        ss.linattn_fn(x[None], x[None], x[None], g.requires_grad_())
    with pytest.raises(ValueError):
        ss.group_norm(x)
    with pytest.raises(ValueError):
        ss.pack_requests(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 4)
