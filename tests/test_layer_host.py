"""Host-side checks of the layer operators' C ABI (no GPU): every refusal returns before any HIP call."""
import ctypes

import pytest
import torch

from mamba_selective_scan_fwd_amd import ss

G = 1 << 32  # far-apart, aligned stand-in addresses; never dereferenced (validation fails first)
R = ctypes.byref


def _conv(**kw):
    d = dict(tokens=40, nseqs=3, dim=24, nslots=5, x_stride=48, out_stride=24, width=4, io_dtype=2, silu=1, reserved=0)
    d.update(kw)
    return ss.ss_conv_prompt_problem(*(d[n] for n, _ in ss.ss_conv_prompt_problem._fields_))


def _conv_call(p, **kw):
    a = dict(x=G, w=2 * G, bias=None, cu=3 * G, slots=4 * G, has=None, state=5 * G, out=6 * G)
    a.update(kw)
    return ss.load_library().ss_conv1d_prompt(R(p) if p is not None else None, a["x"], a["w"], a["bias"], a["cu"],
                                              a["slots"], a["has"], a["state"], a["out"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), 2), (dict(nseqs=0), 2), (dict(nslots=0), 2), (dict(dim=0), 2), (dict(tokens=(1 << 30) + 1), 2),
    (dict(nseqs=(1 << 20) + 1), 2), (dict(x_stride=23), 2), (dict(out_stride=23), 2), (dict(x_stride=(1 << 21) + 1), 2),
    (dict(tokens=1 << 30, dim=1 << 21, x_stride=1 << 21, out_stride=1 << 21), 2),
    (dict(io_dtype=3), 3), (dict(width=0), 5), (dict(width=5), 5), (dict(reserved=1), 5)])
def test_conv_prompt_rejects_bad_problem(kw, code):
    assert _conv_call(_conv(**kw)) == code


def test_conv_prompt_rejects_bad_pointers():
    p = _conv()
    assert _conv_call(None) == 1
    for k in ("x", "w", "cu", "state", "out"):
        assert _conv_call(p, **{k: None}) == 1
    assert _conv_call(p, x=G + 1) == 4 and _conv_call(p, out=6 * G + 1) == 4     # not aligned to the element
    for k in ("w", "cu", "slots", "state"):
        assert _conv_call(p, **{k: 7 * G + 4}) == 4
    assert _conv_call(_conv(nslots=2), slots=None) == 5                           # fewer slots than sequences
    assert _conv_call(p, out=G + 16) == 5                                         # out inside x's rows
    assert _conv_call(p, state=6 * G) == 5                                        # the pool is out
    assert _conv_call(p, state=G - 16) == 5                                       # the pool runs into x


def _prompt(**kw):
    d = dict(tokens=700, nseqs=3, nslots=4, nheads=4, ngroups=2, x_stride=512, b_stride=512, c_stride=512,
             z_stride=256, dt_stride=4, headdim=64, dstate=64, io_dtype=2, dt_softplus=1)
    d.update(kw)
    return ss.ss_ssd_prompt_problem(*(d[n] for n, _ in ss.ss_ssd_prompt_problem._fields_))


def _prompt_call(p, wsz=1 << 31, **kw):
    a = dict(x=G, dt=2 * G, A=3 * G, Bm=G + 512, Cm=G + 768, D=None, z=None, bias=None, cu=4 * G, slots=5 * G, has=None,
             state=6 * G, y=7 * G, ws=8 * G)
    a.update(kw)
    return ss.load_library().ss_ssd_prompt(R(p) if p is not None else None, a["x"], a["dt"], a["A"], a["Bm"], a["Cm"],
                                           a["D"], a["z"], a["bias"], a["cu"], a["slots"], a["has"], a["state"],
                                           a["y"], a["ws"], wsz, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), 2), (dict(nseqs=0), 2), (dict(nslots=0), 2), (dict(nheads=0), 2), (dict(ngroups=0), 2),
    (dict(x_stride=255), 2), (dict(b_stride=120), 2), (dict(c_stride=127), 2), (dict(dt_stride=3), 2),
    (dict(x_stride=(1 << 21) + 8), 2), (dict(x_stride=516), 4), (dict(b_stride=132), 4), (dict(c_stride=132), 4),
    (dict(io_dtype=0), 3), (dict(headdim=32), 5), (dict(dstate=16), 5), (dict(dstate=80), 5), (dict(ngroups=3), 5),
    (dict(nheads=1 << 16, x_stride=1 << 21, dt_stride=1 << 16), 5),
    (dict(tokens=1 << 30), 2)])
def test_ssd_prompt_rejects_bad_problem(kw, code):
    p = _prompt(**kw)
    assert ss.load_library().ss_ssd_prompt_workspace_size(R(p)) == 0
    assert _prompt_call(p) == code


def test_ssd_prompt_rejects_bad_pointers_and_workspace():
    p = _prompt()
    wsz = ss.load_library().ss_ssd_prompt_workspace_size(R(p))
    places = 700 // 256 + 3
    # a state and a decay per (place, head), C B^T per (place, group)
    assert wsz == places * 4 * 64 * 64 * 4 + 256 + places * 2 * 65536 * 4
    assert _prompt_call(None) == 1
    for k in ("x", "dt", "A", "Bm", "Cm", "cu", "state", "y"):
        assert _prompt_call(p, **{k: None}) == 1
    for k in ("x", "A", "Bm", "Cm", "D", "z", "bias", "cu", "slots", "has", "state", "y", "ws"):
        assert _prompt_call(p, **{k: 9 * G + 2}) == 4
    assert _prompt_call(p, dt=2 * G + 1) == 4
    assert _prompt_call(_prompt(z_stride=255), z=9 * G) == 2 and _prompt_call(_prompt(z_stride=260), z=9 * G) == 4
    assert _prompt_call(p, wsz=wsz - 1) == 5 and _prompt_call(p, ws=None) == 5
    assert _prompt_call(_prompt(nslots=2), slots=None) == 5
    for k, v in (("y", G), ("y", G + 512), ("state", 7 * G), ("ws", 7 * G), ("ws", 6 * G), ("state", G)):
        assert _prompt_call(p, **{k: v}) == 5, (k, v)


def _step(**kw):
    d = dict(rows=3, nslots=4, nheads=4, ngroups=2, xbc_stride=512, z_stride=256, dt_stride=4, headdim=64, dstate=64,
             width=4, io_dtype=2, dt_softplus=1, reserved=0)
    d.update(kw)
    return ss.ss_ssd_step_problem(*(d[n] for n, _ in ss.ss_ssd_step_problem._fields_))


def _step_call(p, wsz=1 << 31, **kw):
    a = dict(xbc=G, dt=2 * G, A=3 * G, w=4 * G, cb=None, D=None, z=None, bias=None, slots=5 * G, cs=6 * G, state=7 * G,
             y=8 * G, ws=9 * G)
    a.update(kw)
    return ss.load_library().ss_ssd_step(R(p) if p is not None else None, a["xbc"], a["dt"], a["A"], a["w"], a["cb"],
                                         a["D"], a["z"], a["bias"], a["slots"], a["cs"], a["state"], a["y"], a["ws"],
                                         wsz, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), 2), (dict(nslots=0), 2), (dict(nheads=0), 2), (dict(ngroups=0), 2), (dict(xbc_stride=511), 2),
    (dict(dt_stride=3), 2), (dict(rows=(1 << 20) + 1), 2), (dict(rows=1 << 20, nheads=16, xbc_stride=2048, dt_stride=16), 2),
    (dict(io_dtype=0), 3), (dict(headdim=128), 5), (dict(dstate=48), 5), (dict(ngroups=3), 5), (dict(width=0), 5),
    (dict(width=5), 5), (dict(reserved=1), 5)])
def test_ssd_step_rejects_bad_problem(kw, code):
    p = _step(**kw)
    assert ss.load_library().ss_ssd_step_workspace_size(R(p)) == 0
    assert _step_call(p) == code


def test_ssd_step_rejects_bad_pointers_and_workspace():
    p = _step()
    wsz = ss.load_library().ss_ssd_step_workspace_size(R(p))
    assert _step_call(None) == 1
    for k in ("xbc", "dt", "A", "w", "cs", "state", "y"):
        assert _step_call(p, **{k: None}) == 1
    for k in ("xbc", "dt", "z"):
        assert _step_call(p, **{k: 11 * G + 1}) == 4
    for k in ("A", "w", "cb", "D", "bias", "slots", "cs", "state", "y", "ws"):
        assert _step_call(p, **{k: 11 * G + 4}) == 4
    assert _step_call(_step(z_stride=255), z=11 * G) == 2
    assert _step_call(p, wsz=wsz - 1) == 5 and _step_call(p, ws=None) == 5
    assert _step_call(_step(nslots=2), slots=None) == 5
    for k, v in (("y", G), ("state", 6 * G), ("cs", G), ("ws", 8 * G), ("ws", 7 * G)):
        assert _step_call(p, **{k: v}) == 5, (k, v)


def _ssd(**kw):
    d = dict(batch=2, seqlen=300, nheads=4, ngroups=2, headdim=64, dstate=64, io_dtype=2, dt_softplus=1)
    d.update(kw)
    return ss.ss_ssd_problem(*(d[n] for n, _ in ss.ss_ssd_problem._fields_))


SSD_ORDER = ("x", "dt", "A", "Bm", "Cm", "D", "z", "bias", "seq", "h0", "dy", "dfinal", "dx", "ddt", "dA", "dB", "dC",
             "dD", "dz", "dbias", "dh0", "ws")


def _ssd_bwd(p, wsz=1 << 40, **kw):
    a = {k: None for k in SSD_ORDER}
    for i, k in enumerate(("x", "dt", "A", "Bm", "Cm", "dy", "dx", "ddt", "dA", "dB", "dC", "ws")):
        a[k] = (i + 1) * G
    a.update(kw)
    return ss.load_library().ss_ssd_bwd(R(p) if p is not None else None, *(a[k] for k in SSD_ORDER), wsz, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 2), (dict(seqlen=0), 2), (dict(io_dtype=0), 3), (dict(headdim=32), 5), (dict(dstate=16), 5),
    (dict(ngroups=3), 5), (dict(batch=1 << 12, seqlen=1 << 14, nheads=16, ngroups=16), 2)])
def test_ssd_bwd_rejects_bad_problem(kw, code):
    p = _ssd(**kw)
    assert ss.load_library().ss_ssd_bwd_workspace_size(R(p), 0) == 0
    assert _ssd_bwd(p) == code


def test_ssd_bwd_rejects_bad_pointers_and_workspace():
    p = _ssd()
    lib = ss.load_library()
    wsz = lib.ss_ssd_bwd_workspace_size(R(p), 0)
    assert lib.ss_ssd_bwd_workspace_size(R(p), 1) > wsz > 0
    assert _ssd_bwd(None) == 1
    for k in ("x", "dt", "A", "Bm", "Cm", "dy", "dx", "ddt", "dA", "dB", "dC"):
        assert _ssd_bwd(p, **{k: None}) == 1
    for a, b in (("z", "dz"), ("D", "dD"), ("bias", "dbias")):       # an input without its gradient, and the reverse
        assert _ssd_bwd(p, **{a: 20 * G}) == 1 and _ssd_bwd(p, **{b: 20 * G}) == 1
    for k in SSD_ORDER:
        both = {"D": "dD", "z": "dz", "bias": "dbias", "dD": "D", "dz": "z", "dbias": "bias"}
        more = {both[k]: 21 * G} if k in both else {}
        assert _ssd_bwd(p, **{k: 20 * G + 4}, **more) == 4, k
    assert _ssd_bwd(p, wsz=wsz - 1) == 5 and _ssd_bwd(p, ws=None) == 5
    assert _ssd_bwd(p, wsz=wsz, z=20 * G, dz=21 * G) == 5             # a gated problem needs more
    for k, v in (("dx", G), ("dB", 4 * G), ("ddt", 2 * G), ("dC", 10 * G), ("ws", 7 * G), ("dh0", 6 * G)):
        assert _ssd_bwd(p, **{k: v}) == 5, (k, v)


CONV_ORDER = ("x", "w", "bias", "seq", "init", "dout", "dfinal", "dx", "dw", "dbias", "dinit", "ws")


def _conv_bwd(wsz=1 << 31, prob=None, **kw):
    p = prob if prob is not None else ss.ss_conv_problem(2, 3, 10, 4, 0, 1, 0)
    a = {k: None for k in CONV_ORDER}
    for i, k in enumerate(("x", "w", "dout", "dx", "dw", "ws")):
        a[k] = (i + 1) * G
    a.update(kw)
    return ss.load_library().ss_conv1d_bwd(R(p), *(a[k] for k in CONV_ORDER), wsz, None)


def test_conv_bwd_rejects():
    lib = ss.load_library()
    for prob, code in ((ss.ss_conv_problem(0, 3, 10, 4, 0, 1, 0), 2), (ss.ss_conv_problem(2, 3, 0, 4, 0, 1, 0), 2),
                       (ss.ss_conv_problem(2, 3, 10, 5, 0, 1, 0), 5), (ss.ss_conv_problem(2, 3, 10, 4, 9, 1, 0), 3),
                       (ss.ss_conv_problem(2, 3, 10, 4, 0, 1, 1), 5), (ss.ss_conv_problem(1, 1 << 24, 1, 4, 0, 1, 0), 2)):
        assert lib.ss_conv1d_bwd_workspace_size(R(prob)) == 0
        assert _conv_bwd(prob=prob) == code
    for k in ("x", "w", "dout", "dx", "dw"):
        assert _conv_bwd(**{k: None}) == 1
    assert _conv_bwd(bias=20 * G) == 1 and _conv_bwd(dbias=20 * G) == 1
    for k in CONV_ORDER:
        more = {"bias": {"dbias": 21 * G}, "dbias": {"bias": 21 * G}}.get(k, {})
        assert _conv_bwd(**{k: 20 * G + 8}, **more) == 4, k
    many = ss.ss_conv_problem(8, 16, 4096, 4, 0, 1, 0)
    need = lib.ss_conv1d_bwd_workspace_size(R(many))
    assert need > 0 and _conv_bwd(prob=many, wsz=need - 1) == 5 and _conv_bwd(prob=many, ws=None) == 5
    for k, v in (("dx", G), ("dx", 3 * G), ("dw", 2 * G), ("dinit", 4 * G)):
        assert _conv_bwd(**{k: v}) == 5, (k, v)


def test_python_calls_refuse_host_tensors_and_wrong_types():
    t = torch.zeros
    with pytest.raises(ValueError):
        ss.conv1d_prompt(t(4, 8), t(8, 4), t(2, dtype=torch.int32), t(1, 8, 3))
    with pytest.raises(TypeError):
        ss.conv1d_prompt(t(4, 8, dtype=torch.float64), t(8, 4), t(2, dtype=torch.int32), t(1, 8, 3))
    with pytest.raises(TypeError):
        ss.ssd_prompt(t(4, 2, 64), t(4, 2), t(2), t(4, 1, 32), t(4, 1, 32), t(2, dtype=torch.int32), t(1, 2, 64, 32))
    with pytest.raises(TypeError):
        ss.ssd_step(t(4, 192), t(4, 2), t(2), t(192, 4), t(4, 192, 3), t(4, 2, 64, 32))
    with pytest.raises(TypeError):
        ss.ssd_bwd(t(1, 4, 2, 64), t(1, 4, 2), t(2), t(1, 4, 1, 32), t(1, 4, 1, 32), t(1, 4, 2, 64))
    with pytest.raises(ValueError):
        ss.conv1d_bwd(t(1, 2, 4), t(2, 4), t(1, 2, 4))
