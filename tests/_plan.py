"""The rules by which the state and pass kernels choose their variant (csrc/ss_plan.h), compiled for the host."""
import ctypes
import functools
import os
import subprocess
import tempfile

from mamba_selective_scan_fwd_amd import build

_SRC = '''#include "ss_plan.h"
extern "C" int heads(int64_t chunk_groups, int64_t heads_per_group, int64_t cus) {
  return ss::state_heads(chunk_groups, heads_per_group, cus);
}
extern "C" int ahead(int64_t workgroups, int64_t chunks, int64_t nseqs, int64_t cus) {
  return ss::pass_ahead(workgroups, chunks, nseqs, cus);
}
'''


@functools.lru_cache(maxsize=None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(_SRC)
        subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + build.CSRC, src, "-o", lib], check=True)
        so = ctypes.CDLL(lib)
    for fn in (so.heads, so.ahead):
        fn.restype, fn.argtypes = ctypes.c_int, [ctypes.c_int64] * (3 if fn is so.heads else 4)
    return so


def bwd_heads(batch, seqlen, nheads, ngroups, cus=256):
    """Heads per workgroup of the gradients' state kernel."""
    return _lib().heads(2 * batch * ((seqlen + 255) // 256) * ngroups, nheads // ngroups, cus)


def prompt_heads(tokens, nseqs, nheads, ngroups, cus=256):
    """Heads per workgroup of the prompts' state kernel."""
    return _lib().heads((tokens // 256 + nseqs) * ngroups, nheads // ngroups, cus)


def prompt_ahead(tokens, nseqs, nheads, dstate, cus=256):
    """Chunks that the prompts' pass loads ahead."""
    return _lib().ahead(nseqs * nheads * (64 * dstate // 1024), tokens // 256 + nseqs, nseqs, cus)
