"""Pins of the oracle of the operators around the layer (oracle.block_oracle):
its gradients against central differences of its own forward functions in 64
bits, its choices against brute force, and special cases with known values."""
import itertools

import numpy as np
import pytest

from oracle import block_oracle as B


def difference(f, x, step=1e-6):
    """Central differences of the scalar f at x, element by element."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        g[i] = (f(hi) - f(lo)) / (2 * step)
    return g


@pytest.mark.parametrize("score,renormalize", itertools.product(["softmax", "sigmoid"],
                                                                [True, False]))
def test_router_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(3)
    x, k = rng.normal(size=(3, 9)), 4
    x[1, 2] = -np.inf
    x[2, 1:] = -np.inf                        # a single expert left
    gw = rng.normal(size=(3, k))
    kw = dict(score=score, renormalize=renormalize, scale=1.7)
    ids, _ = B.router_topk(x, k, **kw)
    got, _ = B.router_topk_grad(x, ids, gw, **kw)
    want = difference(lambda v: (B.router_topk(v, k, **kw)[1] * gw).sum(), x)
    want[~np.isfinite(x)] = 0.0
    np.testing.assert_allclose(got, want, atol=1e-8)


def test_router_choice_special_cases():
    x = np.array([[1.0, 3.0, 3.0, 2.0], [np.nan, -np.inf, 5.0, np.inf],
                  [-np.inf] * 4, [0.0] * 4])
    ids, w = B.router_topk(x, 3, "softmax")
    assert ids.tolist() == [[1, 2, 3], [3, 2, -1], [-1, -1, -1], [0, 1, 2]]
    np.testing.assert_allclose(w[1], [1, 0, 0], atol=1e-30)
    assert (w[2] == 0).all() and np.allclose(w[3], 1 / 3)
    # the bias moves the choice, not the weights
    ids, w = B.router_topk(x[3:], 2, "sigmoid", bias=[0, 0, 0.1, 0.2], renormalize=False)
    assert ids.tolist() == [[3, 2]] and (w == 0.5).all()
    # groups of two: the best group by its best expert, by its two best
    g = np.array([[3.0, -9.0, 2.0, 2.0]])
    assert B.router_topk(g, 2, "sigmoid", groups=2, topk_groups=1)[0].tolist() == [[0, 1]]
    assert B.router_topk(g, 2, "sigmoid", groups=2, topk_groups=1,
                         group_top=2)[0].tolist() == [[2, 3]]
    # a group whose second expert is masked counts its first alone
    g[0, 1] = -np.inf
    assert B.router_topk(g[:, :2], 1, "sigmoid", groups=1, group_top=2)[0].tolist() == [[0]]


def test_sorted_slots_and_sums():
    ids = np.array([[1, 0], [0, -1], [5, 1], [1, 1]])
    off, slot_row, row_slot = B.sort_slots(ids, 2, pad=[0, 0, 0, 0])
    assert off.tolist() == [0, 2, 6] and row_slot.tolist() == [1, 2, 0, 5, 6, 7]
    assert slot_row.tolist() == [[2, 0], [1, -1], [-1, 3], [4, 5]]
    rng = np.random.default_rng(5)
    rows, w, g = rng.normal(size=(8, 3)), rng.normal(size=(4, 2)), rng.normal(size=(4, 3))
    grad_rows, gw, _ = B.combine_grad(g, rows, slot_row, w)
    f = lambda r, v: (B.combine(r, slot_row, v)[0] * g).sum()          # noqa: E731
    np.testing.assert_allclose(gw, difference(lambda v: f(rows, v), w), atol=1e-8)
    want = difference(lambda r: f(r, w), rows)
    for r in range(8):
        np.testing.assert_allclose(grad_rows.get(r, np.zeros(3)), want[r], atol=1e-8)


@pytest.mark.parametrize("kind,sigmoid,post", [("none", False, True), ("token", True, True),
                                               ("channel", False, False), ("full", True, True),
                                               ("channel", True, True)])
def test_norm_gradients_against_differences(kind, sigmoid, post):
    rng = np.random.default_rng(7)
    T, H = 3, 5
    r, y = rng.normal(size=(T, H)), rng.normal(size=(T, H))
    w_pre, w_post = rng.normal(size=H), rng.normal(size=H)
    gate = {"none": None, "token": rng.normal(size=T), "channel": rng.normal(size=H),
            "full": rng.normal(size=(T, H))}[kind]
    dh, dr = rng.normal(size=(T, H)), rng.normal(size=(T, H))
    kw = dict(post_norm=post, kind=kind, sigmoid=sigmoid, eps=1e-3, scale=0.7, offset=0.4)

    def loss(r=r, y=y, w_pre=w_pre, w_post=w_post, gate=gate):
        o = B.block_norm(r, y, w_post=w_post if post else None, gate=gate, w_pre=w_pre, **kw)
        return (o["normed"][0] * dh).sum() + (o["residual_out"][0] * dr).sum()

    x = B.block_norm(r, y, w_post=w_post if post else None, gate=gate, w_pre=w_pre,
                     **kw)["residual_out"][0]
    got = B.block_norm_grad(x, dh, dr, y, w_post=w_post if post else None, gate=gate,
                            w_pre=w_pre, **kw)
    close = lambda n, want: np.testing.assert_allclose(got[n][0], want, atol=2e-8)  # noqa: E731
    close("grad_residual", difference(lambda v: loss(r=v), r))
    close("grad_y", difference(lambda v: loss(y=v), y))
    close("grad_pre_weight", difference(lambda v: loss(w_pre=v), w_pre))
    if post:
        close("grad_post_weight", difference(lambda v: loss(w_post=v), w_post))
    if gate is not None:
        close("grad_gate", difference(lambda v: loss(gate=v), gate))
