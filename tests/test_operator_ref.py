"""The gradients' formulas in tests/operator_ref.py against central differences
in 64 bits (CPU)."""
import numpy as np
import pytest

import operator_ref as R

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _diff(f, a, h=1e-5):
    """Central differences of the scalar f with respect to every entry of a
    (modified in place and put back)."""
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        v = a[i]
        a[i] = v + h
        up = f()
        a[i] = v - h
        dn = f()
        a[i] = v
        g[i] = (up - dn) / (2 * h)
    return g


# second-order differences: error h^2 |f'''| / 6 plus 2^-52 |f| / h, both far below 1e-7 here
TOL = 1e-7


@pytest.mark.parametrize("name", ACTS)
def test_linear_gradients_match_differences(name):
    rng = np.random.default_rng(3)
    x, W, b = rng.normal(size=(3, 4)), rng.normal(size=(5, 4)), rng.normal(size=5)
    dy = rng.normal(size=(3, 5))
    f = lambda: float((R.linear(x, W, b, name, None, "f32", "f32")[0] * dy).sum())
    g = R.linear_backward(dy, x, W, name, x @ W.T + b, "bf16", True)
    for key, a in (("dx", x), ("dW", W), ("db", b)):
        assert np.abs(g[key][0] - _diff(f, a)).max() < TOL, key


@pytest.mark.parametrize("name", ACTS)
def test_activations_at_the_ends(name):
    z = np.array([-60.0, -8.0, -0.0, 0.0, 8.0, 60.0])
    assert np.isfinite(R.act(name, z)).all() and np.isfinite(R.dact(name, z)).all()
    assert np.abs(R.dact(name, np.linspace(-10, 10, 4001))).max() <= R.SLOPE


def test_move_gradients_match_differences():
    rng = np.random.default_rng(4)
    T, k, H = 4, 3, 5
    inv = rng.permutation(T * k).reshape(T, k)
    inv = np.where(inv >= T * k - 2, -1, inv)       # two dropped slots
    x, w, ys = rng.normal(size=(T, H)), rng.normal(size=(T, k)), rng.normal(size=(T * k, H))
    dxs, dy = rng.normal(size=(T * k, H)), rng.normal(size=(T, H))
    live = np.zeros(T * k, bool)
    live[inv[inv >= 0]] = True
    zero = np.zeros((T * k, H))
    f = lambda: float((R.dispatch(x, inv, w, "f32", zero)[0] * dxs).sum())
    assert np.abs(_diff(f, x) - R.combine(dxs, inv, w, None, "f32")[0]).max() < TOL
    assert np.abs(_diff(f, w) - R.slot_dots(x, dxs, inv)[0]).max() < TOL
    f = lambda: float((R.combine(ys, inv, w, x, "f32")[0] * dy).sum())
    assert np.abs(_diff(f, ys) - R.dispatch(dy, inv, w, "f32", zero)[0]).max() < TOL
    assert np.abs(_diff(f, w) - R.slot_dots(dy, ys, inv)[0]).max() < TOL


@pytest.mark.parametrize("renorm", [True, False])
def test_router_gradient_matches_differences(renorm):
    rng = np.random.default_rng(5)
    T, E, k = 3, 6, 2
    l, dw = rng.normal(size=(T, E)), rng.normal(size=(T, k))
    ids = np.argsort(-l, 1)[:, :k]
    f = lambda: float((R.route_weights(l, ids, renorm) * dw).sum())
    w = R.route_weights(l, ids, renorm)
    assert np.abs(_diff(f, l) - R.route_backward(l, ids, w, dw, E, renorm, "f32")[0]).max() < TOL
