"""The oracle of the experts' products against central differences and
hand-worked values, in 64 bits."""
import numpy as np
import pytest

from oracle import expert_oracle as X


@pytest.mark.parametrize("kind,limit", [(k, 0.0) for k in X.GATED + X.SINGLE] + [
    ("silu", 1.0), ("swigluoai", 1.0), ("swiglustep", 0.8)])
def test_activation_slopes(kind, limit):
    rng = np.random.default_rng(3)
    n = 40
    pre = rng.normal(0, 2, (5, n * (2 if kind in X.GATED else 1)))
    h = 1e-6
    f, dg, du = X.activate(kind, pre, limit)
    for j in range(pre.shape[1]):
        up, down = pre.copy(), pre.copy()
        up[:, j] += h
        down[:, j] -= h
        diff = (X.activate(kind, up, limit)[0] - X.activate(kind, down, limit)[0]) / (2 * h)
        want = dg[:, j] if j < n else du[:, j - n]
        assert np.allclose(diff[:, j % n], want, atol=1e-6), (kind, j)


@pytest.mark.parametrize("kind", ["none", "silu", "relu2_no_mul"])
def test_gradients_against_differences(kind):
    rng = np.random.default_rng(5)
    E, K, N = 3, 4, 3
    offsets = [0, 2, 2, 5]
    x = rng.normal(size=(6, K))
    w = rng.normal(size=(E, N * (2 if kind in X.GATED else 1), K))
    gout = rng.normal(size=(6, N))

    def loss(x, w):
        return np.nansum(X.linear(x, w, offsets, kind)["out"][0] * gout)

    pre = X.linear(x, w, offsets, kind)["pre_act"][0]
    got = X.linear_grad(x, w, offsets, gout, pre, kind)
    gx, gw = got["grad_x"][0], got["grad_weight"][0]
    assert np.isnan(gx[5]).all() and (gw[1] == 0).all()
    h = 1e-6
    for t, g in ((x, np.nan_to_num(gx)), (w, gw)):
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + h
            up = loss(x, w)
            t[i] = keep - h
            down = loss(x, w)
            t[i] = keep
            assert abs((up - down) / (2 * h) - g[i]) < 1e-7, i


def test_values_worked_by_hand():
    assert X.activate("silu", np.array([[0.0, 5.0]]))[0][0, 0] == 0.0
    assert X.activate("silu", np.array([[3.0, 2.0]]), 1.0)[0][0, 0] == pytest.approx(
        1.0 / (1.0 + np.exp(-1.0)))
    assert X.activate("swigluoai", np.array([[0.0, 5.0]]))[0][0, 0] == 0.0
    assert X.activate("relu2_no_mul", np.array([[3.0, -2.0]]))[0].tolist() == [[9.0, 0.0]]
    assert X.curve("gelu", np.array([0.0]))[1][0] == 0.5
