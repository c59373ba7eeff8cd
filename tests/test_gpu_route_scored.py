"""GPU: routing by scores and its gradient, against float64.

Ids are equal.  Weights, u = 2^-24: a score's exponential and its argument 6 u, 1 + e and the quotient 3 u,
a softmax's sum over E / 64 and then 6 steps, the sum of up to 8 scores 7 u, quotient and scale 3 u: within
2^-19.  Gradients: each of the terms that are summed within 2^-18 of its magnitude."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_top_amd import moe as _moe
from oracle import block as B

pytestmark = pytest.mark.gpu
W, G = 2.0 ** -19, 2.0 ** -18


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _moe.lib()
    return _moe


def _logits(T, E, seed=0, std=1.5):
    return (torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * std)


def _bias(E, seed=0, std=0.05):
    return torch.randn(E, generator=torch.Generator().manual_seed(1000 + seed)) * std


def f64(t):
    return t.double().cpu().numpy()


SCORE = {True: 1, False: 0}  # moe.SCORE_SIGMOID, SCORE_SOFTMAX


def check(moe, l, k, bias=None, sigmoid=True, tiny=0.0, **kw):
    ids, w = moe.route_scored(l.cuda(), k, None if bias is None else bias.cuda(), score=SCORE[sigmoid], **kw)
    want, ww = B.route_scored(f64(l), k, None if bias is None else f64(bias), sigmoid, **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want)
    assert (np.abs(f64(w) - ww) <= W * np.abs(ww) + tiny).all()
    return ids, w


SHAPES = [  # T, E, k, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 8, 2, 1, 1, 1), (5, 60, 4, 6, 3, 1), (7, 60, 4, 1, 1, 1), (77, 64, 8, 8, 3, 2),
    (130, 65, 5, 13, 7, 2), (64, 128, 8, 4, 1, 1), (33, 160, 6, 8, 3, 1), (300, 256, 8, 8, 4, 2),
    (257, 384, 8, 1, 1, 1), (9, 512, 8, 64, 8, 2), (11, 512, 8, 2, 2, 1), (4, 512, 1, 1, 1, 1), (6, 16, 8, 8, 4, 2),
    (4, 7, 7, 7, 7, 1), (5, 320, 3, 5, 1, 2), (70, 96, 8, 12, 5, 2), (70, 192, 6, 3, 2, 2), (3, 511, 8, 1, 1, 2)]


@pytest.mark.parametrize("T,E,k,groups,top,gt", SHAPES)
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_route_scored(moe, T, E, k, groups, top, gt, sigmoid, bias):
    b = _bias(E, E, 0.05 if sigmoid else 1.0 / E) if bias else None
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        check(moe, _logits(T, E, T + E), k, b, sigmoid, groups=groups, top_groups=top, group_top=gt,
              renorm=renorm, scale=scale)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("groups,top,gt", [(1, 1, 1), (8, 4, 2)])
def test_route_scored_many_tokens(moe, sigmoid, groups, top, gt):
    """Enough rows that some hold scores within fp32's roundings of each other."""
    check(moe, _logits(20000, 256, 5), 8, _bias(256, 5, 0.05 if sigmoid else 0.004), sigmoid, groups=groups,
          top_groups=top, group_top=gt)


def test_route_scored_near_ties(moe):
    """Biases that put pairs of scores some fp32 steps, or a fraction of one, apart: the order is that of 64
    bits; equal pairs go to the lower id."""
    rng = np.random.default_rng(3)
    T, E = 400, 64
    l = rng.normal(size=(1, E)).astype(np.float32).repeat(T, 0)
    l[:, 1::2] += rng.normal(size=(T, E // 2)).astype(np.float32) * 1e-7
    s = 1 / (1 + np.exp(-l[0].astype(np.float64)))
    bias = (2.0 - np.round(s * 16) / 16 - s + np.round(s * 16) / 16).astype(np.float32)  # c near 2 for all
    check(moe, torch.from_numpy(l), 8, torch.from_numpy(bias))
    check(moe, torch.from_numpy(l), 8, torch.from_numpy(bias), groups=8, top_groups=3, group_top=2)
    check(moe, torch.zeros(5, 96), 8, torch.full((96,), 0.3), groups=4, top_groups=2, group_top=2)
    check(moe, torch.zeros(5, 96), 8, sigmoid=False)
    check(moe, torch.zeros(5, 96), 8, groups=4, top_groups=2, group_top=2)
    l = torch.zeros(4, 64)
    l[:, ::2] = -0.0
    check(moe, l, 8)


@pytest.mark.parametrize("E,k,groups,top", [(64, 8, 1, 1), (256, 8, 8, 2), (60, 4, 6, 2)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("value", [-np.inf, float(np.finfo(np.float32).min)])
def test_route_scored_masked(moe, E, k, groups, top, sigmoid, bias, value):
    """Experts masked in whole, in part, all but one; rows masked whole; by -inf and by the lowest float."""
    l = _logits(8, E, 3)
    l[0] = value
    l[1, 1:] = value
    l[2, ::2] = value
    l[3, : E - 3] = value
    l[4, 5:] = value
    l[5, E // 2:] = value
    b = _bias(E, 2, 0.3 if sigmoid else 0.01) if bias else None
    for renorm in (True, False):
        for gt in (1, 2):
            ids, w = check(moe, l, k, b, sigmoid, groups=groups, top_groups=top, group_top=gt, renorm=renorm)
            assert all(len(set(r)) == k for r in ids.cpu().tolist())


def test_route_scored_bias_masks(moe):
    """-inf and the lowest float as a bias mask an expert in all rows, +inf selects it first."""
    E, l = 40, _logits(9, 40, 1)
    b = _bias(E, 1)
    b[3], b[17], b[20:36] = np.inf, -np.inf, float(np.finfo(np.float32).min)
    ids, _ = check(moe, l, 8, b)
    assert (ids[:, 0] == 3).all()
    check(moe, l, 8, b, sigmoid=False, groups=4, top_groups=4, group_top=1)
    check(moe, l, 8, torch.full((E,), -np.inf))


def test_route_scored_extreme_logits(moe):
    """Scores that leave fp32's range keep their ratio; +inf is a sigmoid's 1."""
    l = _logits(6, 32, 2)
    l[0] -= 100
    l[1] -= 500
    l[2] += 60
    l[3] = torch.linspace(-90, 90, 32)
    l[4, 7] = np.inf
    check(moe, l, 4, tiny=2.0 ** -149)
    check(moe, l, 4, renorm=False, tiny=2.0 ** -149)
    check(moe, l, 4, _bias(32, 1), tiny=2.0 ** -149)
    check(moe, l[:4], 4, sigmoid=False, tiny=2.0 ** -149)
    check(moe, l[:4], 4, sigmoid=False, renorm=False, tiny=2.0 ** -149)
    check(moe, l[:4], 4, _bias(32, 1, 1.0), sigmoid=False, tiny=2.0 ** -149)  # (scores of 1e-30 selected)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_scored_scores_near_fp32s_smallest(moe, sigmoid, renorm):
    """Selected experts far below the first, whose scores fp32 holds in a few bits or none: a renormalisation or a
    factor brings them back, with all their bits.  (2^-149: what a weight itself may be off by)"""
    l = torch.full((6, 64), -200.0)
    for i, low in enumerate((-60.0, -75.0, -88.0, -95.0, -100.0, -103.0)):
        l[i, 3:9] = low - torch.arange(6) / 7.0
        if not sigmoid:
            l[i, 20] = 0.0  # (the softmax's largest)
    check(moe, l, 6, sigmoid=sigmoid, renorm=renorm, scale=2.0 ** 100, tiny=2.0 ** -149)
    check(moe, l, 6, sigmoid=sigmoid, renorm=renorm, scale=1.0, tiny=2.0 ** -149)


@pytest.mark.parametrize("E,k,groups,top", [(256, 8, 8, 4), (256, 8, 1, 1), (64, 6, 1, 1), (384, 8, 1, 1)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_scored_of_any_address(moe, E, k, groups, top, sigmoid):
    """Logits, bias and gradients that start at a multiple of 4 bytes, not of 16."""
    T = 37
    l, b = _logits(T, E, 3), _bias(E, 2, 0.05 if sigmoid else 0.004)

    def moved(t):
        return torch.cat([torch.zeros(1), t.flatten()]).cuda()[1:].view(t.shape)

    for bias in (b, None):
        kw = dict(groups=groups, top_groups=top, group_top=2, renorm=False)
        want, ww = B.route_scored(f64(l), k, None if bias is None else f64(bias), sigmoid, **kw)
        for ml in (moved, torch.Tensor.cuda):
            for mb in (moved, torch.Tensor.cuda):
                ids, w = moe.route_scored(ml(l), k, None if bias is None else mb(bias), score=SCORE[sigmoid], **kw)
                assert np.array_equal(ids.cpu().numpy(), want) and (np.abs(f64(w) - ww) <= W * ww).all()
        dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).cuda()
        got = [moe.route_scored_grad(m(l), ids, w, dw, SCORE[sigmoid], False) for m in (moved, torch.Tensor.cuda)]
        ref, mag = B.route_scored_grad(f64(l), want, f64(w), f64(dw), sigmoid, renorm=False)
        assert all((np.abs(f64(g) - ref) <= G * mag).all() for g in got)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_scored_non_finite_rows(moe, sigmoid):
    """Whatever a row holds its ids are different experts, and the other rows are left."""
    l = _logits(8, 48, 4)
    kw = dict(score=SCORE[sigmoid], groups=4, top_groups=2, group_top=2)
    for b in (None, _bias(48, 1).cuda()):
        ids0, w0 = moe.route_scored(l.cuda(), 8, b, **kw)
        bad = l.clone()
        bad[1], bad[2, 5], bad[4, 3], bad[4, 30], bad[6] = np.nan, np.nan, np.inf, np.inf, np.inf
        ids, w = moe.route_scored(bad.cuda(), 8, b, **kw)
        assert all(len(set(r)) == 8 and 0 <= min(r) and max(r) < 48 for r in ids.cpu().tolist())
        rest = [0, 3, 5, 7]
        assert torch.equal(ids[rest], ids0[rest]) and torch.equal(w[rest], w0[rest])


def test_route_scored_neighbours_and_zero_tokens(moe):
    T, E, k = 5, 256, 6
    l = _logits(T, E, 1).cuda()
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    dl = torch.full((T + 1, E), -7.0, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    sc = moe.Scoring(1, 1, 1, 1, 1, 1.0)
    L = moe.lib()
    assert L.moe_route_scored(l.data_ptr(), None, T, E, k, sc, ids.data_ptr(), w.data_ptr(), st) == 0
    for score, renorm in ((1, 1), (0, 0)):
        sc = moe.Scoring(score, 1, 1, 1, renorm, 1.0)
        assert L.moe_route_scored_grad(l.data_ptr(), ids.data_ptr(), w.data_ptr(), w.data_ptr(), T, E, k, sc,
                                       dl.data_ptr(), st) == 0
        assert (dl[T] == -7).all() and not (dl[:T] == -7).any()
    assert (ids[T] == -7).all() and (w[T] == -7).all()
    i0, w0 = moe.route_scored(l[:0], k)
    assert i0.shape == w0.shape == (0, k) and moe.route_scored_grad(l[:0], i0, w0, w0).shape == (0, E)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129])
def test_route_scored_row_counts(moe, T):
    check(moe, _logits(T, 96, T), 8, _bias(96, T), groups=6, top_groups=3, group_top=2)
    check(moe, _logits(T, 384, T), 8)


def check_grad(moe, l, k, sigmoid, renorm, scale, ids=None, w=None, dw=None):
    T, E = l.shape
    kw = dict(renorm=renorm, scale=scale)
    if ids is None:
        ids, w = moe.route_scored(l.cuda(), k, score=SCORE[sigmoid], **kw)
    if dw is None:
        dw = torch.randn(T, k, generator=torch.Generator().manual_seed(9))
    dl = moe.route_scored_grad(l.cuda(), ids, w, dw.cuda(), score=SCORE[sigmoid], **kw)
    ref, mag = B.route_scored_grad(f64(l), ids.cpu().numpy(), f64(w), f64(dw), sigmoid, **kw)
    assert dl.shape == l.shape and (np.abs(f64(dl) - ref) <= G * mag + 2.0 ** -140).all()
    return dl


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 8, 2), (7, 60, 4), (130, 65, 5), (300, 256, 8), (9, 512, 8),
                                   (5, 511, 1), (2000, 384, 8), (77, 130, 3)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm,scale", [(True, 2.5), (False, 1.0), (False, 0.5)])
def test_route_scored_grad(moe, T, E, k, sigmoid, renorm, scale):
    dl = check_grad(moe, _logits(T, E, T + E), k, sigmoid, renorm, scale)
    assert torch.equal(dl, check_grad(moe, _logits(T, E, T + E), k, sigmoid, renorm, scale))


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_scored_grad_edges(moe, sigmoid, renorm):
    """Masked rows, far logits, an expert named twice, ids outside the experts, weights of 0."""
    l = _logits(7, 20, 3)
    l[0] = -np.inf
    l[1, 2:] = -np.inf
    l[2] += 90
    l[3] -= 90
    l[4] = torch.linspace(-200, 200, 20)
    check_grad(moe, l, 4, sigmoid, renorm, 1.0)
    ids = torch.tensor([[1, 1, 5], [0, 19, 0], [-1, 3, 20], [2 ** 30, -2 ** 31, 4]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 0.25], [0, 0, 0], [0.3, 0.3, 0.4], [0.1, 0.2, 0.7]], device="cuda")
    check_grad(moe, _logits(4, 20, 1), 3, sigmoid, renorm, 1.0, ids, w)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_scored_grad_against_differences(moe, sigmoid, renorm):
    """Along one direction, the float64 weights' central differences: the gradient's fp32 errors, summed with
    the direction's magnitudes, bound the gap (and the differences' own 1e-9)."""
    T, E, k = 4, 24, 3
    l, dw = _logits(T, E, 2), _logits(T, k, 3)
    kw = dict(renorm=renorm, scale=1.5)
    ids, w = moe.route_scored(l.cuda(), k, score=SCORE[sigmoid], **kw)
    dl = f64(moe.route_scored_grad(l.cuda(), ids, w, dw.cuda(), score=SCORE[sigmoid], **kw))
    v, e = f64(_logits(T, E, 4)), 1e-5
    f = lambda a: (B.route_scored(a, k, None, sigmoid, **kw)[1] * f64(dw)).sum()  # noqa: E731
    num = (f(f64(l) + e * v) - f(f64(l) - e * v)) / (2 * e)
    _, mag = B.route_scored_grad(f64(l), ids.cpu().numpy(), f64(w), f64(dw), sigmoid, **kw)
    assert abs(num - (dl * v).sum()) <= (mag * np.abs(v)).sum() * (G + W) + 1e-8


SIZES = [(64, 8, 4, 2), (128, 4, 2, 1), (256, 8, 4, 2), (384, 16, 5, 2), (512, 2, 1, 2), (8, 2, 1, 1), (60, 6, 2, 2),
         (320, 4, 2, 2), (511, 7, 3, 1)]  # E, groups, top_groups, group_top


def _places(E):
    """Experts at the ends of the row, of its sixteenths and of its middle."""
    v = (E + 15) // 16
    return sorted({e for e in (0, 1, v - 1, v, 2 * v - 1, E // 2 - 1, E // 2, E - v, E - 2, E - 1) if 0 <= e < E})


@pytest.mark.parametrize("E,groups,top,gt", SIZES)
@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_scored_every_expert_first_in_far_rows(moe, E, groups, top, gt, sigmoid):
    """Rows of neighbouring logits that lie far from 0, each expert of interest the largest of its row: without a
    bias the order is the logits', wherever they lie."""
    down = torch.stack([(torch.arange(E) - e) % E for e in _places(E)]).float()
    k = min(8, E // groups * top)
    for step in (1.0 / 8, 1.0):
        rows = [off - step * down for off in (0.0, 20.0, 255.0, 272.5, 300.0, 500.0, 600.0, 1e3, 5e3, 1e4, 2.0 ** 20)]
        l = torch.cat(rows + [r - 2 * r[:, :1].max() for r in rows])
        for kw in (dict(), dict(groups=groups, top_groups=top, group_top=gt)):
            check(moe, l, k, sigmoid=sigmoid, tiny=2.0 ** -149, **kw)


@pytest.mark.parametrize("E,groups,top,gt", SIZES)
@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_scored_every_expert_first_by_far_biases(moe, E, groups, top, gt, sigmoid):
    """The same of biases, which order the experts and lie far from 0."""
    k = min(8, E // groups * top)
    l = _logits(3, E, 7, 0.01)
    for off in (0.0, 20.0, 33.0, 34.0, 40.0, 64.0, 100.0, 1e3, -31.0, -40.0, -100.0, -1e3):
        for e in _places(E):
            bias = off - ((torch.arange(E) - e) % E).float() / 16
            for kw in (dict(), dict(groups=groups, top_groups=top, group_top=gt)):
                ids, _ = check(moe, l, k, bias, sigmoid, **kw)
                assert (ids[:, 0] == e).all() or kw


def _at_a_border(rng, T, E, c, step):
    """Logits [T, E] and biases [E], on fp32's grid of width `step` there, whose sums all lie within some 2^-24 of
    c + step / 2, half a step: fp32's scores, off by less, put them a whole step apart."""
    m = rng.integers(int(0.1 / step), int(0.9 / step) + 1, E)
    s = step / 2 + step * m
    l = np.log(s / (1 - s)).astype(np.float32)
    l = l + rng.integers(-1, 2, (T, E)) * np.spacing(l)
    return torch.from_numpy(l.astype(np.float32)), torch.from_numpy((c - step * m).astype(np.float32))


@pytest.mark.parametrize("E,k", [(8, 4), (16, 8), (14, 6), (64, 8), (60, 8)])
@pytest.mark.parametrize("c", [2.0 ** 6, 2.0 ** 16, 2.0 ** 20, 2.0 ** 21, 2.0 ** 22, 3.0 * 2 ** 20])
def test_route_scored_at_a_border_of_far_sums(moe, E, k, c):
    """Scores and biases whose sums fp32 rounds to either side, far from 0: compared in 64 bits."""
    l, b = _at_a_border(np.random.default_rng(E), 200, E, c, float(np.spacing(np.float32(c))))
    b[16:] -= 4.0  # (16 or fewer are near: in some rows as many are above the border as are selected)
    check(moe, l, k, b)
    if E % 4 == 0:
        check(moe, l, 4, b, groups=4, top_groups=2, group_top=2 if E > 4 else 1)


@pytest.mark.parametrize("E,k", [(8, 2), (16, 4), (14, 3), (64, 2), (60, 6)])
@pytest.mark.parametrize("top", [100.0, 50.0, 1000.0, -100.0])
def test_route_scored_at_the_end_of_the_span(moe, E, k, top):
    """One expert as far above the others as the fast comparison reaches, and the others at a border of fp32 there:
    its nearest places, and what lies below them."""
    step = float(np.spacing(np.float32(abs(top) + 1.0)))
    for off in range(-2, 3):
        l, b = _at_a_border(np.random.default_rng(E + off), 200, E, top - 2.0 + off * step, step)
        l[:, E // 2], b[E // 2] = 0.0, top - 0.5
        b[16:] -= 4.0
        check(moe, l, k, b)


@pytest.mark.parametrize("E,k,groups,top", [(256, 8, 8, 4), (384, 8, 1, 1), (60, 4, 6, 3), (100, 1, 1, 1)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm,scale", [(True, 2.5), (False, 1.0)])
def test_route_scored_weights_are_rounded_once(moe, E, k, groups, top, sigmoid, renorm, scale):
    """Scores, their sum, quotient and scale in 64 bits: with an exponential of 2 u64, E additions and 4 more
    roundings, u64 = 2^-53, an fp32 weight is within half a step, 2^-24, and 2^-42 of it more."""
    l = _logits(1500, E, E)
    l[::7] *= 20.0  # (scores near 0 and 1 too)
    kw = dict(groups=groups, top_groups=top, group_top=2, renorm=renorm, scale=scale)
    for bias in (None, _bias(E, E, 0.05 if sigmoid else 1.0 / E)):
        ids, w = check(moe, l, k, bias, sigmoid, tiny=2.0 ** -149, **kw)
        ww = B.route_scored(f64(l), k, None if bias is None else f64(bias), sigmoid, **kw)[1]
        assert (np.abs(f64(w) - ww) <= (2.0 ** -24 + 2.0 ** -42) * np.abs(ww) + 2.0 ** -150).all()


@pytest.mark.parametrize("E", [64 * i for i in range(1, 9)])
def test_route_scored_of_whole_vectors_and_not(moe, E):
    """Every E of whole 16-byte vectors per lane, and the same rows at an address that allows none (a softmax's sum
    then has another order: a last bit)."""
    T = 70
    l, b = _logits(T, E, E).cuda(), _bias(E, E).cuda()
    moved = torch.cat([torch.zeros(1, device="cuda"), l.flatten()])[1:].view(T, E)
    for kw in (dict(), dict(groups=8, top_groups=4, group_top=2), dict(score=0, renorm=False)):
        for bias in (b, None):
            (i0, w0), (i1, w1) = moe.route_scored(l, 8, bias, **kw), moe.route_scored(moved, 8, bias, **kw)
            assert torch.equal(i0, i1) and (w0 - w1).abs().max() <= 2.0 ** -24
    check(moe, l.cpu(), 8, b.cpu(), groups=8, top_groups=4, group_top=2)


def test_route_scored_past_32_bit_offsets(moe):
    """More than 2^32 bytes of logits: every fourth row is the same row."""
    E, k = 512, 8
    T = 2 ** 30 // E + 400
    l, b = _logits(4, E, 1).cuda(), _bias(E, 1).cuda()
    big = l.repeat(T // 4, 1)
    ids0, w0 = moe.route_scored(l, k, b, groups=8, top_groups=4, group_top=2)
    ids, w = moe.route_scored(big, k, b, groups=8, top_groups=4, group_top=2)
    assert torch.equal(ids.view(-1, 4, k), ids0.expand(T // 4, 4, k))
    assert torch.equal(w.view(-1, 4, k), w0.expand(T // 4, 4, k))
    for score, renorm in ((1, True), (0, False)):
        d0 = moe.route_scored_grad(l, ids0, w0, w0, score=score, renorm=renorm)
        d = moe.route_scored_grad(big, ids, w, w, score=score, renorm=renorm)
        assert torch.equal(d.view(-1, 4, E), d0.expand(T // 4, 4, E))
        del d
