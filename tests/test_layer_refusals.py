"""Overlaps of strided buffers that the packed calls refuse (CPU): ranges count, not bytes."""
from test_layer_host import G, _conv, _conv_call, _step, _step_call


def test_columns_of_the_same_rows_are_refused():
    """x in the first 24 columns of rows of 48, out in the last 24: no byte is shared, the ranges meet."""
    p = _conv(x_stride=48, out_stride=48)
    assert _conv_call(p, out=G + 24 * 2) == 5 and _conv_call(p, x=G + 24 * 2, out=G) == 5
    last = 39 * 48 * 2 + 24 * 2                       # behind the last row of x's range
    assert _conv_call(p, out=G + last - 2) == 5
    assert _step_call(_step(xbc_stride=1024), y=G + 512 * 2) == 5
