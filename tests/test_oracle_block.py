"""Pins of oracle/block.py: closed forms, small cases by hand, and gradients against differences."""
import numpy as np
import pytest

from oracle import block as B


def test_scores_closed_forms():
    assert np.allclose(B.scores([[0.0, np.log(3.0), -np.inf, 800.0]], True), [[0.5, 0.75, 0.0, 1.0]])
    assert np.allclose(B.scores([[0.0, np.log(3.0), -np.inf]], False), [[0.25, 0.75, 0.0]])
    assert (B.scores(np.full((1, 3), -np.inf), False) == 0).all()


def test_route_by_hand():
    l = np.array([[0.0, 2.0, 2.0, 1.0, -1.0, 3.0]])
    ids, w = B.route_scored(l, 3, renorm=False)
    assert ids.tolist() == [[5, 1, 2]] and np.allclose(w, 1 / (1 + np.exp(-l[0, ids])))
    # the bias moves the selection, not the weights
    ids, w = B.route_scored(l, 2, bias=[1.0, 0, 0, 0, 0, 0], scale=2.0)
    s = B.scores(l, True)[0]
    assert ids.tolist() == [[0, 5]] and np.allclose(w, 2 * s[[0, 5]] / s[[0, 5]].sum())
    # two groups of three: the second has the largest expert, the first the larger pair
    a = dict(k=2, groups=2, top_groups=1)
    assert B.route_scored(l, group_top=1, **a)[0].tolist() == [[5, 3]]
    assert B.route_scored(l, group_top=2, **a)[0].tolist() == [[1, 2]]
    # masked experts come last, with weight 0
    ids, w = B.route_scored([[-np.inf, 1.0, -np.inf, -np.inf]], 3, bias=[9.0, 0, 0, 0])
    assert ids.tolist() == [[1, 0, 2]] and w.tolist() == [[1.0, 0.0, 0.0]]


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_is_the_derivative(sigmoid, renorm):
    rng = np.random.default_rng(1)
    l, dw = rng.normal(size=(3, 7)), rng.normal(size=(3, 2))
    kw = dict(sigmoid=sigmoid, renorm=renorm, scale=2.5)

    def f(l):
        return (B.route_scored(l, 2, **kw)[1] * dw).sum()

    ids, w = B.route_scored(l, 2, **kw)
    got, _ = B.route_scored_grad(l, ids, w, dw, **kw)
    for i in np.ndindex(l.shape):
        d = np.zeros_like(l)
        d[i] = 1e-6
        assert abs((f(l + d) - f(l - d)) / 2e-6 - got[i]) < 1e-8


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_block_grad_is_the_derivative(post, gate):
    rng = np.random.default_rng(2)
    T, d, eps = 3, 8, 1e-3
    x, r, dy, dh = (rng.normal(size=(T, d)) for _ in range(4))
    a = dict(x=x, r=r, post=rng.normal(size=d) if post else None, pre=rng.normal(size=d),
             gate={None: None, "channel": rng.normal(size=d), "token": rng.normal(size=(T, d))}[gate])

    def f(a):
        h, _, y = B.block_norm(a["x"], a["r"], a["post"], a["gate"], a["pre"], 0.7, 0.3, eps)
        return (y(h) * dy).sum() + (h * dh).sum()

    h = B.block_norm(x, r, a["post"], a["gate"], a["pre"], 0.7, 0.3, eps)[0]
    g = B.block_norm_grad(dy, dh, x, h, a["post"], a["gate"], a["pre"], 0.7, 0.3, eps)
    for name, key in (("x", "dx"), ("r", "dres"), ("pre", "dpre"), ("post", "dpost"), ("gate", "dgate")):
        if a[name] is None:
            continue
        for i in np.ndindex(a[name].shape):
            e = np.zeros_like(a[name])
            e[i] = 1e-6
            diff = (f(dict(a, **{name: a[name] + e})) - f(dict(a, **{name: a[name] - e}))) / 2e-6
            assert abs(diff - g[key][i]) < 1e-7, (name, i)


def test_w4_values_by_hand():
    codes = np.array([[0x21, 0xF0]], np.uint8)  # 1, 2, 0, 15
    assert B.w4_values(codes, [[2.0, 0.5]], None, 2).tolist() == [[-14.0, -12.0, -4.0, 3.5]]
    assert B.w4_values(codes, [[2.0, 0.5]], [[1, 15]], 2).tolist() == [[0.0, 2.0, -7.5, 0.0]]
    w = np.array([[1.0, -2.0]])
    assert B.gemm_w4([[3.0, 1.0]], w)[0].tolist() == [[1.0]]
    y, _ = B.gemm_w4([[3.0, 1.0]], w, 2 * w)
    assert np.allclose(y, 1 / (1 + np.exp(-1.0)) * 2)


def test_block_norm_by_hand():
    # mean squares of 1 and 4: x / 1 * post, then the gate, both scales and the residual; h / 2 * pre
    x, r = [[1.0, -1.0]], [[6.0, 4.0]]
    h, mag, y = B.block_norm(x, r, [2.0, 4.0], [0.5, -1.0], [3.0, 10.0], 0.5, -1.0, 0.0)
    assert h.tolist() == [[2.0, -2.0]] and mag.tolist() == [[4.0, 6.0]] and y(h).tolist() == [[3.0, -10.0]]
    h, _, y = B.block_norm(x, r, None, None, [1.0, 1.0], 1.0, 1.0, 2.0)
    assert h.tolist() == [[7.0, 3.0]] and np.allclose(y(h), h / np.sqrt(31.0))
