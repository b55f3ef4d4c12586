"""The 64-bit references of linear attention and of the grouped norm, pinned by differences and closed forms (CPU)."""
import numpy as np
import pytest

import _linattn_ref as ref


def _draw(n, H, G, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((n, H, dk)), k=r.standard_normal((n, G, dk)), v=r.standard_normal((n, G, dv)),
                g=-np.exp(r.uniform(-6, 0, H)), scale=0.3, h0=r.standard_normal((H, dv, dk)))


def test_linattn_rows_are_the_weighted_sum():
    p = _draw(9, 2, 1, 3, 4)
    y, H = ref.linattn_rows(**p)
    a = np.exp(p["g"])
    for h in range(2):
        for t in range(9):
            s = a[h] ** (t + 1) * p["h0"][h] @ p["q"][t, h]
            for j in range(t + 1):
                s = s + a[h] ** (t - j) * (p["q"][t, h] @ p["k"][j, 0]) * p["v"][j, 0]
            assert np.allclose(y[t, h], p["scale"] * s, rtol=1e-12)


@pytest.mark.parametrize("G", [1, 2])
def test_linattn_gradients_by_differences(G):
    p = _draw(6, 2, G, 3, 4, seed=G)
    r = np.random.default_rng(7)
    dy, df = r.standard_normal((6, 2, 4)), r.standard_normal((2, 4, 3))

    def loss(**kw):
        y, H = ref.linattn_rows(**dict(p, **kw))
        return (y * dy).sum() + (H * df).sum()

    for name, g in zip(("q", "k", "v", "h0"), ref.linattn_grads(**p, dy=dy, dfinal=df)):
        d = r.standard_normal(p[name].shape)
        e = 1e-6
        num = (loss(**{name: p[name] + e * d}) - loss(**{name: p[name] - e * d})) / (2 * e)
        assert abs(num - (g * d).sum()) <= 1e-7 * (1 + np.abs(g * d).sum()), name


@pytest.mark.parametrize("mode", ["plain", "silu", "gate", "gate_first"])
@pytest.mark.parametrize("center", [False, True])
def test_norm_gradients_by_differences(mode, center):
    r = np.random.default_rng(3)
    x, z, dy = (r.standard_normal((4, 12)) for _ in range(3))
    w, b = r.standard_normal(12), r.standard_normal(12)
    z = z if mode.startswith("gate") else None
    a = dict(x=x, w=w, b=b, z=z)
    g = ref.norm_grads(**a, dy=dy, groups=3, eps=1e-3, center=center, mode=mode)
    for name, key in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("z", "dz")):
        if a[name] is None:
            continue
        d = r.standard_normal(a[name].shape)
        f = lambda s: (ref.norm(**dict(a, **{name: a[name] + s * d}), groups=3, eps=1e-3, center=center, mode=mode)[0] * dy).sum()
        assert abs((f(1e-6) - f(-1e-6)) / 2e-6 - (g[key][0] * d).sum()) <= 1e-6 * (1 + np.abs(g[key][0] * d).sum()), name


def test_norm_of_whole_rows():
    x = np.arange(8.0).reshape(1, 8)
    y, _ = ref.norm(x, np.ones(8), np.zeros(8), None, 1, 0.0, True, "plain")
    assert abs(y.mean()) < 1e-12 and abs((y ** 2).mean() - 1) < 1e-12


def test_pack_by_hand():
    got = ref.pack([1, 5, 0, 1, 1, 4], [3, 2, 1, 0, -1, 7], [9, 0, 5, 0, 4, 6], 8)
    want = dict(rows=[0, 1, -1, 6, -1, 7], taken=[1, 5, 0, 1, 0, 1], step_slots=[3, -1, -1, -1, -1, -1],
                cu_seqlens=[1, 6, 7, 8, 8, 8, 8], prompt_slots=[2, 0, 7, -1, -1, -1], has_state=[0, 0, 1, 0, 0, 0],
                row_request=[0, 1, 1, 1, 1, 1, 3, 5], row_position=[9, 0, 1, 2, 3, 4, 0, 6])
    for k, v in want.items():
        assert got[k].tolist() == v, k
