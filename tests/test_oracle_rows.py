"""CPU pins of oracle/rows.py: gradients against central differences in float64, int8 rows against
hand values."""
import numpy as np
import pytest

from oracle import rows as R


def _diff(f, x, dir_, step=1e-5):
    return (f(x + step * dir_) - f(x - step * dir_)) / (2 * step)


@pytest.mark.parametrize("T,d", [(1, 8), (3, 40)])
def test_rmsnorm_grad_against_differences(T, d):
    r = np.random.default_rng(T * 100 + d)
    h, w, dy = r.normal(size=(T, d)), r.normal(size=d), r.normal(size=(T, d))
    dx, dw = R.rmsnorm_grad(dy, h, w, 1e-3)
    vh, vw = r.normal(size=(T, d)), r.normal(size=d)
    # central differences of a smooth function of order 1: error step^2 = 1e-10, rounding 1e-11
    assert _diff(lambda a: (dy * R.rmsnorm(a, w, 1e-3)).sum(), h, vh) == pytest.approx((dx * vh).sum(), abs=1e-7)
    assert _diff(lambda a: (dy * R.rmsnorm(h, a, 1e-3)).sum(), w, vw) == pytest.approx((dw * vw).sum(), abs=1e-7)


def test_sort_grads_against_differences():
    r = np.random.default_rng(5)
    T, E, k, d = 6, 5, 3, 16
    logits = r.normal(size=(T, E))
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    slot = r.permutation(T * k)
    y, dout, x = r.normal(size=(T * k, d)), r.normal(size=(T, d)), r.normal(size=(T, d))

    def weights(lg):
        v = np.exp(np.take_along_axis(lg, ids, 1))
        return v / v.sum(1, keepdims=True)

    def combine(yp, w):
        return (w[:, :, None] * yp[slot].reshape(T, k, d)).sum(1)

    w = weights(logits)
    dy, dw = R.combine_grad(dout, y, slot, w)
    v = r.normal(size=y.shape)
    assert _diff(lambda a: (dout * combine(a, w)).sum(), y, v) == pytest.approx((dy * v).sum(), abs=1e-7)
    dl = R.route_grad(ids, w, dw, E)
    v = r.normal(size=logits.shape)
    assert _diff(lambda a: (dout * combine(y, weights(a))).sum(), logits, v) == pytest.approx((dl * v).sum(), abs=1e-7)
    g = r.normal(size=(T * k, d))  # arrives at x_perm[slot[t*k+j]] = x[t]

    def gather(a):
        xp = np.zeros((T * k, d))
        xp[slot] = np.repeat(a, k, axis=0)
        return xp

    v = r.normal(size=x.shape)
    assert _diff(lambda a: (g * gather(a)).sum(), x, v) == pytest.approx((R.permute_grad(g, slot, k) * v).sum(), abs=1e-7)


def test_int8_rows_by_hand():
    q, s = R.quant_i8([[254.0, -127.0, 1.0, 3.0, -255.0], [0, 0, 0, 0, 0]])
    assert s[0] == np.float32(255 / 127) and s[1] == 1.0
    assert q[0].tolist() == [127, -63, 0, 1, -127]  # v * 127 / 255: 126.502, -63.25, 0.498, 1.494, -127
    assert q[1].tolist() == [0] * 5
    assert R.gemm_i8([[1, -2]], [0.5], [[3, 4], [-128, 127]], [2.0, 1.0]).tolist() == [[-5.0, -191.0]]
