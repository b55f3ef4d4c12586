"""The sizes that linear attention's calls refuse (CPU): no more than their launches need."""
import ctypes

import pytest

import test_more_host as base
from mamba_selective_scan_fwd_amd import ss

R = ctypes.byref


def _codes(**kw):
    """The codes of the forward, the prompts and the backward of a problem without pointers: 1 if its sizes are taken."""
    none = {n: None for n in base.A}
    return base._calls(base._lin(**kw), **none)[:3]


@pytest.mark.parametrize("kw", [dict(nheads=16, kv_heads=16, dk=64, dv=64), dict(nheads=32, kv_heads=32, dk=128, dv=128),
                                dict(nheads=32, kv_heads=16, dk=64, dv=64), dict(nheads=32, kv_heads=8, dk=64, dv=64)])
def test_gradients_take_what_the_forward_takes(kw):
    """2^22 rows of 16 heads and more: only the sums over shared heads, a thread for 4 channels, have a limit, which
    16 of them with 2^22 * 16 * 128 channels, 2^23 workgroups, are the first to pass."""
    over = kw["kv_heads"] == 16 and kw["nheads"] == 32
    kw = dict(kw, tokens=1 << 22, nseqs=2, packed=0, q_stride=4096, k_stride=4096, v_stride=4096)
    assert _codes(**kw) == (1, 1, 2 if over else 1)
    if over:
        assert _codes(**dict(kw, tokens=(1 << 22) - 2)) == (1, 1, 1)
        return
    lib = ss.load_library()
    size = lib.ss_linattn_bwd_workspace_size(R(base._lin(**kw)))
    if kw["nheads"] != kw["kv_heads"]:
        assert size >= (1 << 22) * kw["nheads"] * (kw["dk"] + kw["dv"]) * 4


def test_sums_over_shared_heads_have_a_limit():
    kw = dict(tokens=1 << 24, nseqs=2, packed=0, dk=64, dv=128, q_stride=4096, k_stride=4096, v_stride=4096)
    assert _codes(**kw, nheads=8, kv_heads=8) == (1, 1, 1)
    assert _codes(**kw, nheads=8, kv_heads=2) == (1, 1, 1)      # 2^24 * 2 * 48 threads, 3 * 2^21 workgroups
    assert _codes(**kw, nheads=8, kv_heads=4) == (1, 1, 2)


def test_packed_sequences_in_pieces_have_no_limit_of_their_own():
    """Pieces go by rows and places, however many sequences there are; whole walks are a workgroup each."""
    kw = dict(tokens=65536, nheads=12, kv_heads=12, dk=128, dv=128, q_stride=4096, k_stride=4096, v_stride=4096)
    assert _codes(**kw, nseqs=1 << 20) == (1, 1, 1)
    whole = dict(kw, tokens=384)
    assert _codes(**whole, nseqs=1 << 18) == (1, 1, 2)          # 12 and 36 walks of each
    assert _codes(**whole, nseqs=1 << 20) == (2, 2, 2)
    assert _codes(**dict(kw, tokens=1 << 20, packed=0), nseqs=1 << 20) == (2, 2, 2)
