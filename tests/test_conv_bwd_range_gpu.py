"""Gradients of the convolution for inputs near fp32's largest value: the steps behind a row's end do not exist, however
large what the weights would make of the row's last inputs there."""
import numpy as np
import pytest
import torch

import _layer_ref as ref
from _util import f64, say
from test_layer_grad_gpu import _conv, _ss

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [1, 2, 3, 8, 13, 16, 23, 2048, 2051])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("docs", [False, True])
def test_rows_that_end_with_large_inputs(L, sign, docs):
    """x[L-1] = 3e38: pre of the last step, 0.1 x, is 3e37, and what the next step's would be, 2 x, is past the type.
    Where |pre| is that large SiLU's slope is 1 or 0 exactly, so dx, dw and dbias are sums of a few finite products,
    held to 2^-20 of the sum of their magnitudes (a dozen roundings of 2^-24 each)."""
    ss = _ss()
    say("large inputs L=%d sign=%g docs=%d" % (L, sign, docs))
    q = _conv(2, 3, L, 4, "f32", seed=L)
    q["w"][1] = torch.tensor([2.0, 2.0, 2.0, 0.1])
    q["x"][1, 1, L - 1] = sign * 3e38
    q["dout"][1, 1, L - 1] = 0.5                          # its product with x stays in range
    if docs:
        q["seq_idx"] = torch.zeros(2, L, dtype=torch.int32)
    got = ss.conv1d_bwd(**{k: v.cuda() for k, v in q.items()})
    torch.cuda.synchronize()
    x, w, dout, bias = (f64(q[k]) for k in ("x", "w", "dout", "bias"))
    with np.errstate(over="ignore"):
        want, _ = ref.conv_grad(x, w, dout, bias)
    # the magnitudes: |dpre| <= 1.1 |dout|, its own error 2^-22 of (1 + |pre|) |dout| where the slope bends at all
    pre = bias[None, :, None] + sum(w[None, :, k, None] * np.concatenate([np.zeros((2, 3, 3)), x], 2)[:, :, k:k + L]
                                    for k in range(4))
    bend = np.where(np.abs(pre) < 100.0, 1.0 + np.abs(pre), 1.0)
    d = np.concatenate([1.2 * np.abs(dout) * bend, np.zeros((2, 3, 3))], 2)
    mag = dict(dx=sum(np.abs(w)[None, :, 3 - m, None] * d[:, :, m:m + L] for m in range(4)),
               dbias=d.sum((0, 2)),
               dw=np.stack([(d[:, :, :L] * np.abs(np.concatenate([np.zeros((2, 3, 3)), x], 2)[:, :, k:k + L])).sum((0, 2))
                            for k in range(4)], 1))
    for k in ("dx", "dw", "dbias"):
        # dw and dbias: fp32 sums of up to 2L terms, 8 a thread and then over 256 threads
        ref.check(got[k], want[k], mag[k], k, terms=2.0 ** -20 if k == "dx" else ref.SUM)
