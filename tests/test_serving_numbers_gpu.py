"""A serving layer's numbers, link by link: the maps, linear attention over carried states, and the norm of its own outputs."""
import numpy as np
import pytest
import torch

import _linattn_ref as ref
from _layer_ref import check
from _util import f64, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128)])
def test_requests_over_batches(io, dk, dv):
    from mamba_selective_scan_fwd_amd import ss
    R, T, H, G = 7, 600, 2, 1
    say("serving %s %d %d" % (io, dk, dv))
    r = np.random.default_rng(130)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    g, w = torch.tensor([-0.02, -0.4]), torch.from_numpy(1 + 0.2 * r.standard_normal(H * dv)).float()
    slots, state = [3, 0, 8, 1, 5, 2, 6], torch.randn(R + 3, H, dv, dk, device="cuda")
    seen, hist = [0] * R, [[] for _ in range(R)]
    cols = np.cumsum([0, H * dk, G * dk, G * dv, H * dv])
    before = state.clone()
    for new in ([430, 1, 0, 30, 7, 1, 64], [1, 1, 500, 1, 1, 1, 1], [1, 0, 100, 1, 90, 1, 500], [1] * R):
        row = torch.from_numpy(r.standard_normal((T, cols[-1]))).to(io)
        d = row.cuda()
        m = ss.pack_requests(i32(new), i32(slots), i32(seen), T)
        q, k, v = (d[:, cols[i]:cols[i + 1]].unflatten(1, (n, e)) for i, (n, e) in enumerate(((H, dk), (G, dk), (G, dv))))
        y = torch.zeros(T, H, dv, dtype=io, device="cuda")
        ss.linattn_prompt(q, k, v, g.cuda(), m["cu_seqlens"], state, slots=m["prompt_slots"], has_state=m["has_state"], y=y)
        ss.linattn_step(q[:R], k[:R], v[:R], g.cuda(), state, slots=m["step_slots"], y=y[:R])
        out = ss.group_norm(y.flatten(1), w.cuda(), z=d[:, cols[3]:], ngroups=H)
        torch.cuda.synchronize()
        maps = ref.pack(new, slots, seen, T)
        for n, want in maps.items():
            assert np.array_equal(m[n].cpu().numpy(), want), n
        for i in range(R):
            n, at = int(maps["taken"][i]), int(maps["rows"][i])
            if n == 0:
                continue
            x = f64(row[at:at + n])
            hist[i].append(x)
            x = np.concatenate(hist[i])
            a = [x[:, cols[j]:cols[j + 1]].reshape(len(x), c, e) for j, (c, e) in enumerate(((H, dk), (G, dk), (G, dv)))]
            zero = np.zeros((H, dv, dk))
            want, last = ref.linattn_rows(*a, f64(g), dk ** -0.5, zero)
            mag, lm = ref.linattn_rows(*(np.abs(t) for t in a), f64(g), dk ** -0.5, zero)
            check(y[at:at + n], want[-n:], mag[-n:], "y of %d" % i)
            check(state[slots[i]], last, lm, "state")
            # the norm, of the y that it was given
            got = f64(y[at:at + n]).reshape(n, H * dv)
            want, mag = ref.norm(got, f64(w), np.zeros(H * dv), f64(row[at:at + n, cols[3]:]), H, 1e-5, True, "gate")
            check(out[at:at + n], want, mag, "norm", terms=2.0 ** -18)
            seen[i] += n
    for i in set(range(R + 3)) - set(slots):
        assert torch.equal(state[i], before[i])
