"""The norm's oracle: gradients against differences of the forward, and its fixed points."""
import numpy as np
import pytest

from oracle import block as ob


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (4, 17)])
def test_norm_gradients_by_differences(rows, cols, kind):
    r = np.random.default_rng(rows * 100 + cols)
    s, w, b, dy, dsum = r.normal(size=(rows, cols)), r.normal(size=cols), r.normal(size=cols), r.normal(size=(rows, cols)), r.normal(size=(rows, cols))
    eps, h = 1e-2, 1e-6
    loss = lambda s_, w_, b_: (dy * ob.norm(s_, w_, b_, eps, kind)).sum() + (dsum * s_).sum()  # noqa: E731
    mean, rstd = ob.norm_stats(s, eps, kind)
    dx, dw, db = ob.norm_backward(dy, s, w, mean, rstd, dsum, kind)

    def differ(name, got, f):
        for i in np.ndindex(got.shape):
            e = np.zeros(got.shape)
            e[i] = h
            d = (f(e) - f(-e)) / (2 * h)
            assert abs(d - got[i]) <= 1e-6 * (1 + abs(got[i])), (name, i)

    differ("dx", dx, lambda e: loss(s + e, w, b))
    differ("dw", dw, lambda e: loss(s, w + e, b))
    differ("db", db, lambda e: loss(s, w, b + e))


def test_norm_fixed_points():
    s = np.array([[1.0, 3.0], [5.0, 5.0]])
    assert np.allclose(ob.norm(s, eps=0.0)[0], [-1.0, 1.0])
    assert np.allclose(ob.norm(s)[1], 0.0)  # a constant row has no deviation
    assert np.allclose(ob.norm(s, eps=0.0, kind="rms")[1], 1.0)
    # a shift of the row leaves the layer norm, a factor the RMS norm
    assert np.allclose(ob.norm(s + 7, eps=0.0)[0], ob.norm(s, eps=0.0)[0])
    assert np.allclose(ob.norm(s * 7, eps=0.0, kind="rms"), ob.norm(s, eps=0.0, kind="rms"))
