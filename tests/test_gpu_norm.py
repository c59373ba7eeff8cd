"""GPU: RMS norm with its 8-bit outputs, and its gradient, against float64.

Tolerances count roundings.  u = 2^-24.  The sum of squares: eight fp32 FMAs of positive terms, then
fp64 (8 u), halved by the root; mean, eps, root, quotient and the two products: 6 u more; so y before
its output rounding is within 12 u < 2^-20 of the exact value.  bf16 adds 2^-8, e4m3 2^-4 (2^-10 of the
scale below its normal range), int8 half a scale."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_top_amd import moe as _moe
from oracle import fp8_e4m3
from oracle import rows as R

pytestmark = pytest.mark.gpu
EPS = 1e-6
Y = 2.0 ** -20


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _moe.lib()
    return _moe


def _bf16(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def values(moe, act, q, qs, d):
    """(codes' values times scales, scales spread over the columns) as float64."""
    if act == moe.DTYPE_INT8:
        s = np.repeat(f64(qs)[:, None], d, 1)
        return f64(q) * s, s
    code = fp8_e4m3.decode(q.cpu().numpy()).astype(np.float64)
    if act == moe.DTYPE_FP8:
        s = np.repeat(f64(qs), 128, 1)
    else:
        s = np.repeat(np.exp2(qs.cpu().numpy().astype(np.float64) - 127), 32, 1)
    return code * s, s


ACTS = {"bf16": 0, "fp8": 1, "mxfp8": 3, "int8": 4}
SHAPES = [(1, 128), (3, 128), (1, 7168), (5, 512), (77, 4096), (130, 640), (2, 4224), (9, 8192), (3, 12288),
          (2, 32768)]


def check_forward(moe, act, x, w, res, h, y, q, qs):
    d = x.shape[1]
    want_h = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(h.view(torch.int16), want_h.view(torch.int16))
    ref = R.rmsnorm(f64(want_h), f64(w), EPS)
    if y is not None:
        assert (np.abs(f64(y) - ref) <= np.abs(ref) * (2.0 ** -8 + Y)).all()
    if act == moe.DTYPE_BF16:
        assert q is None and qs is None
        return
    v, s = values(moe, act, q, qs, d)
    group = {moe.DTYPE_FP8: 128, moe.DTYPE_MXFP4_A8: 32, moe.DTYPE_INT8: d}[act]
    amax = np.repeat(np.abs(ref).reshape(-1, d // group, group).max(-1), group, 1)
    if act == moe.DTYPE_INT8:
        assert (np.abs(s - amax / 127) <= amax / 127 * 2 * Y).all()
        tol = s / 2 + np.abs(ref) * 2 * Y
    else:
        if act == moe.DTYPE_FP8:
            assert (np.abs(s - amax / 448) <= amax / 448 * 2 * Y).all()
        else:  # the smallest power of two that holds amax
            assert (amax <= 448 * s * (1 + Y)).all() and (amax > 224 * s * (1 - Y)).all()
        tol = np.maximum(np.abs(ref) * 2.0 ** -4, s * 2.0 ** -10) + np.abs(ref) * 2 * Y
    assert (np.abs(v - ref) <= tol).all()


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("fmt", ACTS)
def test_rmsnorm(moe, fmt, T, d):
    act = ACTS[fmt]
    x, w = _bf16(T, d, seed=T + d), _bf16(d, seed=d)
    res = _bf16(T, d, seed=T + d + 1, std=3.0) if (T + d // 128) % 2 else None
    h, y, q, qs = moe.rmsnorm(x, w, res, EPS, act)
    check_forward(moe, act, x, w, res, h, y, q, qs)
    assert h is x if res is None else h is not x
    if fmt != "bf16":
        assert moe.rmsnorm(x, w, res, EPS, act, want_y=False)[1] is None


@pytest.mark.parametrize("fmt,d", [("bf16", 8), ("bf16", 200), ("bf16", 4104), ("mxfp8", 32), ("mxfp8", 4128),
                                   ("int8", 16), ("int8", 4112)])
def test_rmsnorm_odd_rows(moe, fmt, d):
    """Rows that end inside a wavefront, of the fewest channels each format takes."""
    x, w, res = _bf16(7, d, seed=d), _bf16(d, seed=1), _bf16(7, d, seed=2)
    check_forward(moe, ACTS[fmt], x, w, res, *moe.rmsnorm(x, w, res, EPS, ACTS[fmt]))


def test_rmsnorm_int16_bits_and_zero_tokens(moe):
    x, w = _bf16(4, 256, seed=1), _bf16(256, seed=2)
    h, y, _, _ = moe.rmsnorm(x.view(torch.int16), w.view(torch.int16))
    assert y.dtype == torch.int16 and torch.equal(y, moe.rmsnorm(x, w)[1].view(torch.int16))
    h, y, q, qs = moe.rmsnorm(x[:0], w, x[:0], EPS, moe.DTYPE_INT8)
    assert h.shape == y.shape == q.shape == (0, 256) and qs.shape == (0,)
    dx, dw = moe.rmsnorm_grad(x[:0], x[:0], w)
    assert dx.shape == (0, 256) and torch.equal(dw, torch.zeros_like(dw))


def test_rmsnorm_in_place_and_neighbours(moe):
    """h_out may be the residual itself; rows behind the last one stay as they were."""
    T, d = 5, 4224
    x, res, w = _bf16(T + 2, d, seed=1), _bf16(T + 2, d, seed=2), _bf16(d, seed=3)
    want = (x.float() + res.float()).to(torch.bfloat16)
    for inplace in ("residual", "x"):
        a, b = x.clone(), res.clone()
        out = b if inplace == "residual" else a
        keep = out[T:].clone()
        y = torch.full_like(x, 7.0)
        q = torch.full((T + 2, d), 77, dtype=torch.uint8, device="cuda")
        qs = torch.full((T + 2, d // 128), 7.0, device="cuda")
        st = torch.cuda.current_stream().cuda_stream
        assert moe.lib().moe_rmsnorm(a.data_ptr(), b.data_ptr(), w.data_ptr(), EPS, T, d, moe.DTYPE_FP8,
                                     out.data_ptr(), y.data_ptr(), q.data_ptr(), qs.data_ptr(), st) == 0
        torch.cuda.synchronize()
        assert torch.equal(out[:T], want[:T]) and torch.equal(out[T:], keep)
        assert (y[T:] == 7).all() and (q[T:] == 77).all() and (qs[T:] == 7).all()
        check_forward(moe, moe.DTYPE_FP8, x[:T], w, res[:T], out[:T], y[:T], q[:T], qs[:T])


@pytest.mark.parametrize("fmt", ACTS)
def test_rmsnorm_zero_and_non_finite_rows(moe, fmt):
    """A zero row is zero with scale 1; an infinity or NaN makes its own row NaN and no other."""
    act, T, d = ACTS[fmt], 6, 384
    x, w = _bf16(T, d, seed=9), _bf16(d, seed=3)
    clean = moe.rmsnorm(x, w, None, EPS, act)
    bad = x.clone()
    bad[1] = 0
    bad[2, 5], bad[3, 383], bad[4, 0] = float("inf"), float("nan"), float("-inf")
    h, y, q, qs = moe.rmsnorm(bad, w, None, EPS, act)
    assert torch.equal(y[[0, 5]], clean[1][[0, 5]])
    assert (y[1] == 0).all() and y[2:5].isnan().all()
    if act == moe.DTYPE_BF16:
        return
    v, s = values(moe, act, q, qs, d)
    vc, _ = values(moe, act, clean[2], clean[3], d)
    assert (v[[0, 5]] == vc[[0, 5]]).all() and (v[1] == 0).all() and (s[1] == 1).all()
    assert np.isnan(v[2:5]).all()


def test_rmsnorm_small_and_large_values(moe):
    """Rows far below and above one: eps leads, or the squares stay inside fp32."""
    d = 512
    x, w = _bf16(4, d, seed=4), _bf16(d, seed=5)
    for scale in (1e-20, 1e-4, 1e4, 1e17):
        xs = (x.float() * scale).to(torch.bfloat16)
        for act in ACTS.values():
            check_forward(moe, act, xs, w, None, *moe.rmsnorm(xs, w, None, EPS, act))


def check_grad(dy, h, w, dh, dx, dw):
    """dx: bf16's 2^-8, and 2^-20 of each term that is added (mean(g n) by its terms' magnitudes).
    dw: fp32 sums over T / 512 rows, 16 and 32 partials, each product rounded a few times."""
    T, d = dy.shape
    dy64, h64, w64 = f64(dy), f64(h), f64(w)
    ref, refw = R.rmsnorm_grad(dy64, h64, w64, EPS)
    r = 1 / np.sqrt((h64 ** 2).mean(-1, keepdims=True) + EPS)
    g, n = dy64 * w64, h64 * r
    add = 0 if dh is None else f64(dh)
    terms = r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(-1, keepdims=True)) + np.abs(add)
    ref = ref + add
    assert (np.abs(f64(dx) - ref) <= np.abs(ref) * 2.0 ** -8 + terms * 2 * Y).all()
    if dw is not None:
        depth = -(-T // 512) + 16 + 32 + 14
        assert (np.abs(f64(dw) - refw) <= depth * 2.0 ** -24 * np.abs(dy64 * n).sum(0)).all()


@pytest.mark.parametrize("T,d", [(1, 8), (1, 7168), (3, 128), (5, 520), (77, 1024), (200, 4104), (600, 256),
                                 (1030, 2048), (33, 8192), (7, 12288), (3, 16384)])
def test_rmsnorm_grad(moe, T, d):
    h, dy, w = _bf16(T, d, seed=T, std=2.0), _bf16(T, d, seed=T + 1, std=0.1), _bf16(d, seed=d)
    for dh in (None, _bf16(T, d, seed=3, std=0.1)):
        dx, dw = moe.rmsnorm_grad(dy, h, w, dh, EPS)
        check_grad(dy, h, w, dh, dx, dw)
        again, dw2 = moe.rmsnorm_grad(dy, h, w, dh, EPS)
        assert torch.equal(dx, again) and torch.equal(dw, dw2)  # fixed order
    dx2, none = moe.rmsnorm_grad(dy, h, w, dh, EPS, want_dweight=False)
    assert none is None and torch.equal(dx, dx2)


def test_rmsnorm_grad_in_place(moe):
    T, d = 6, 4104
    h, dy, w, dh = _bf16(T, d, seed=1), _bf16(T, d, seed=2), _bf16(d, seed=3), _bf16(T, d, seed=4)
    want, _ = moe.rmsnorm_grad(dy, h, w, dh, EPS)
    for which in ("dy", "dh"):
        a, b = dy.clone(), dh.clone()
        out = a if which == "dy" else b
        st = torch.cuda.current_stream().cuda_stream
        assert moe.lib().moe_rmsnorm_grad(a.data_ptr(), b.data_ptr(), h.data_ptr(), w.data_ptr(), EPS, T, d,
                                          out.data_ptr(), None, None, 0, st) == 0
        assert torch.equal(out, want)


def test_rmsnorm_grad_against_differences(moe):
    """The kernel's dx and dw against central differences of the float64 norm, along one direction:
    the gradients' bf16 and fp32 errors, summed with the direction's magnitudes, bound the gap."""
    T, d = 3, 256
    h, dy, w = _bf16(T, d, seed=1), _bf16(T, d, seed=2), _bf16(d, seed=3)
    dx, dw = moe.rmsnorm_grad(dy, h, w, None, EPS)
    v, vw = f64(_bf16(T, d, seed=4)), f64(_bf16(d, seed=5))
    f = lambda a, b: (f64(dy) * R.rmsnorm(a, b, EPS)).sum()  # noqa: E731
    e = 1e-5
    num = (f(f64(h) + e * v, f64(w)) - f(f64(h) - e * v, f64(w))) / (2 * e)
    assert abs(num - (f64(dx) * v).sum()) <= (np.abs(f64(dx) * v)).sum() * 2.0 ** -8 + 1e-6
    num = (f(f64(h), f64(w) + e * vw) - f(f64(h), f64(w) - e * vw)) / (2 * e)
    assert abs(num - (f64(dw) * vw).sum()) <= (np.abs(f64(dw) * vw)).sum() * 2.0 ** -18 + 1e-6


def test_rmsnorm_past_32_bit_offsets(moe):
    """More than 2^32 bytes per tensor: every fourth row is the same row."""
    d = 7168
    T = 2 ** 31 // d // 4 * 4 + 400
    x, res, w = _bf16(4, d, seed=1), _bf16(4, d, seed=2), _bf16(d, seed=3)
    big = [t.repeat(T // 4, 1) for t in (x, res)]
    few = moe.rmsnorm(x, w, res, EPS, moe.DTYPE_INT8)
    got = moe.rmsnorm(big[0], w, big[1], EPS, moe.DTYPE_INT8)
    for a, b in zip(got, few):
        assert torch.equal(a.view(T // 4, 4, -1), b.view(1, 4, -1).expand(T // 4, 4, -1))
    del got
    dy, dh, h = _bf16(4, d, seed=4), _bf16(4, d, seed=5), few[0]
    dx0, _ = moe.rmsnorm_grad(dy, h, w, dh, EPS)
    dx, dw = moe.rmsnorm_grad(dy.repeat(T // 4, 1), h.repeat(T // 4, 1), w, dh.repeat(T // 4, 1), EPS)
    assert torch.equal(dx.view(T // 4, 4, d), dx0.expand(T // 4, 4, d))
    # dw: a workgroup adds T / 512 rows one after another, the sum over workgroups 16 and then 32 more;
    # each term is within 12 u
    n = h.double() / (h.double().square().mean(1, keepdim=True) + EPS).sqrt()
    terms = dy.double() * n
    room = (T / 512 + 1 + 48 + 12) * 2.0 ** -24 * terms.abs().sum(0) * (T // 4)
    assert ((dw.double() - terms.sum(0) * (T // 4)).abs() <= room).all()


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 191, 193, 1535, 1536, 1537])
def test_rmsnorm_grad_weight_by_rows(moe, T):
    """Row counts around those at which workgroups take one, some and many rows."""
    d = 136
    h, dy, w = _bf16(T, d, seed=T), _bf16(T, d, seed=T + 1), _bf16(d, seed=3)
    dx, dw = moe.rmsnorm_grad(dy, h, w, None, EPS)
    hd = h.double()
    rstd = (hd.square().mean(1, keepdim=True) + EPS).rsqrt()
    g = dy.double() * w.double()
    want = rstd * (g - hd * rstd * rstd * (g * hd).mean(1, keepdim=True))
    # (g - n mean(g n)) / rms: both products and their sums within 2^-20 of their magnitudes, then bf16
    mag = rstd * (g.abs() + (hd * rstd).abs() * rstd * (g * hd).abs().mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= want.abs() * 2.0 ** -8 + mag * 2.0 ** -19).all()
    terms = dy.double() * hd * rstd
    assert ((dw.double() - terms.sum(0)).abs() <= (T + 60) * 2.0 ** -24 * terms.abs().sum(0)).all()


def test_rmsnorm_of_the_most_rows(moe):
    """2^25 - 1 rows, forward and backward: the first and the last are those of a small call."""
    T = 2 ** 25 - 1
    few, g, w = _bf16(7, 8, seed=9), _bf16(7, 8, seed=10), _bf16(8, seed=11)
    x = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    x[:7], x[-7:], dy[:7], dy[-7:] = few, few, g, g
    y = moe.rmsnorm(x, w, None, EPS)[1]
    dx, dw = moe.rmsnorm_grad(dy, x, w, None, EPS)
    want, (wdx, wdw) = moe.rmsnorm(few, w, None, EPS)[1], moe.rmsnorm_grad(g, few, w, None, EPS)
    for part in (slice(0, 7), slice(T - 7, T)):
        assert torch.equal(y[part], want) and torch.equal(dx[part], wdx)
    assert not y[7:-7].any() and not dx[7:-7].any()
    # (14 rows that are not zero, in some order: twice the small sum within their roundings)
    n = few.double() * (few.double().square().mean(1, keepdim=True) + EPS).rsqrt()
    assert ((dw.double() - 2 * wdw.double()).abs() <= 2 * 30 * 2.0 ** -24 * (g.double() * n).abs().sum(0) * 2).all()


def test_rmsnorm_e4m3_groups_of_subnormal_scale(moe):
    """fp32(amax / 448) of a few bits: quotients up to 1.5 * 448 saturate and stay finite.  h is 2^-133 in
    every column and w whole multiples of 2^-17 * 2^-9, so y is a whole multiple n of 2^-149 (rstd is
    1000 (1 + 2^-23) at most off, n below 2^11 and away from half steps)."""
    d = 2048
    n = np.array([464, 625, 1000, 448, 1100, 300, 671, 1119, 480, 1561, 500, 667, 1343, 2000, 230, 5])
    unit = 65536 * 1000.0  # y / 2^-149 of w = 1
    w = torch.from_numpy(n / unit).to(torch.bfloat16).repeat_interleave(128).cuda()
    x = torch.full((3, d), 2.0 ** -133, dtype=torch.bfloat16, device="cuda")
    x[1] *= -1
    exact = np.outer([1, -1, 1], f64(w) * unit)  # (w is rounded: n is only near it)
    keep = np.abs(np.abs(exact) % 1 - 0.5) > 2.0 ** -10
    got = np.rint(exact)
    s = np.repeat(np.rint(np.abs(got).reshape(3, -1, 128).max(-1) / 448.0), 128, 1)
    s = np.where(s == 0, 2.0 ** 149, s)  # the scale 1, in units
    _, _, q, qs = moe.rmsnorm(x, w, None, EPS, moe.DTYPE_FP8)
    assert np.array_equal(np.repeat(f64(qs), 128, 1)[keep], (s * 2.0 ** -149)[keep])
    want = fp8_e4m3.encode(np.clip(got / s, -448, 448))
    assert ((q.cpu().numpy() & 0x7F) != 0x7F).all()
    assert np.array_equal(q.cpu().numpy()[keep], want[keep])
    assert (want & 0x7F == 0x7E).any()


def test_rmsnorm_int8_rows_of_subnormal_scale(moe):
    """y of n 2^-149, n up to 150: fp32(amax / 127) is 2^-149, codes would pass 127, and the scale is
    2^-148."""
    n = np.array([150, -150, 128, -140, 127, -120, 3, 0] * 32)
    x = torch.from_numpy(np.stack([np.sign(n), -np.sign(n)]) * 2.0 ** -133).to(torch.bfloat16).cuda()
    # (rstd is 1000 to within 2^-23; a step of w is 1/256, so y is near n, away from half steps)
    w = torch.from_numpy(np.abs(n) / 65536e3).to(torch.bfloat16).cuda()
    y = np.stack([np.sign(n), -np.sign(n)]) * f64(w) * 65536e3
    assert (np.abs(np.abs(y) % 1 - 0.5) > 2.0 ** -10).all() and np.rint(np.abs(y)).max() == 150
    _, _, q, qs = moe.rmsnorm(x, w, None, EPS, moe.DTYPE_INT8)
    assert (f64(qs) == 2.0 ** -148).all()
    assert np.array_equal(f64(q), np.rint(np.rint(y) / 2))


def test_rmsnorm_int8_half_steps(moe):
    """Exact half steps of a scale that is no power of two: 16384 values whose squares sum to 16384 and
    w = 255 / 128 make y = h w and s = 255 / 128 exactly; h = n + 1/2 rounds to the even side."""
    d = 16384
    row = np.zeros(d)
    row[0] = 127  # 16129; the half steps below bring 203.5, ones and two halves the other 51.5
    row[1:12] = [0.5, -0.5, 1.5, -1.5, 2.5, -2.5, 3.5, -3.5, 4.5, -4.5, 11.0]
    left = d - (row ** 2).sum()
    ones = int(left)
    row[20:20 + ones] = 1
    row[4000:4000 + int((left - ones) * 4)] = 0.5
    assert (row ** 2).sum() == d
    x = torch.from_numpy(np.stack([row, -row])).to(torch.bfloat16).cuda()
    w = torch.full((d,), 255 / 128, dtype=torch.bfloat16, device="cuda")
    _, _, q, qs = moe.rmsnorm(x, w, None, 0.0, moe.DTYPE_INT8)
    assert (qs == 255 / 128).all()
    want = np.rint(np.stack([row, -row]))  # (numpy rounds halves to even)
    assert np.array_equal(f64(q), want)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8"])
def test_rmsnorm_codes_are_the_quantisers(moe, fmt):
    """h = +-1 and eps = 0 make rstd exactly 1 and y = +-w in full: the rows and scales of the quantisers on
    y, bit for bit, for groups of every magnitude that bf16 has."""
    d = 8192
    g = torch.Generator().manual_seed(3)
    mag = torch.linspace(-132, 120, d // 32).repeat_interleave(32)
    w = (torch.randn(d, generator=g) * torch.exp2(mag)).to(torch.bfloat16).cuda()
    w[64:96] = 0
    sign = torch.randint(0, 2, (5, d), generator=g).mul_(2).sub_(1).to(torch.bfloat16).cuda()
    y = sign * w
    _, got, q, qs = moe.rmsnorm(sign, w, None, 0.0, ACTS[fmt])
    assert torch.equal(got, y)
    quant = moe.quant_act if fmt == "fp8" else moe.quant_act_mx
    wq, ws = quant(y.view(torch.int16))
    assert torch.equal(qs, ws) and torch.equal(q, wq)


RANGE = [(2.0 ** -133, 0.0), (1e-38, 0.0), (1e-30, 0.0), (1e-23, 0.0), (1e-20, 1e-44), (1e-19, 1e-38), (1e-12, 0.0),
         (1e18, EPS), (1e20, EPS), (1e30, 0.0), (5e37, EPS)]


@pytest.mark.parametrize("scale,eps", RANGE, ids=str)
@pytest.mark.parametrize("d", [256, 4224, 16384])
def test_rmsnorm_of_every_magnitude(moe, d, scale, eps):
    """Squares below and above fp32's range, without eps or with one as small: y is still h / rms * w to
    within 2^-20, or half a step of the smallest float, before it is rounded."""
    x64 = np.random.default_rng(d).normal(size=(5, d)) * scale
    x = torch.from_numpy(x64).to(torch.bfloat16).cuda()
    x[3, 5:] = x[1, 5:]  # (a row that shares most of another's values)
    x[4] = 1  # an ordinary row beside them
    w = _bf16(d, seed=d)
    ref = R.rmsnorm(f64(x), f64(w), float(np.float32(eps)))
    for act in ACTS.values():
        h, y, q, qs = moe.rmsnorm(x, w, None, eps, act)
        assert torch.equal(h, x)
        assert (np.abs(f64(y) - ref) <= np.abs(ref) * (2.0 ** -8 + Y) + 2.0 ** -134).all()
        if act != moe.DTYPE_BF16:
            v, s = values(moe, act, q, qs, d)
            step = s / 2 if act == moe.DTYPE_INT8 else np.maximum(np.abs(ref) * 2.0 ** -4, s * 2.0 ** -10)
            assert (np.abs(v - ref) <= step + np.abs(ref) * 2 * Y).all()


def test_rmsnorm_zero_row_without_eps(moe):
    """0 / 0, in that row alone."""
    x, w = _bf16(3, 384, seed=1), _bf16(384, seed=2)
    clean = moe.rmsnorm(x, w, None, 0.0)[1]
    x[1] = 0
    y = moe.rmsnorm(x, w, None, 0.0)[1]
    assert y[1].isnan().all() and torch.equal(y[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("scale,eps", RANGE, ids=str)
@pytest.mark.parametrize("d", [256, 4104, 16384])
def test_rmsnorm_grad_of_every_magnitude(moe, d, scale, eps):
    """The gradient of such rows: the tolerances of ordinary ones, and half a step of bf16's smallest value
    (and of fp32's, times n's magnitude, inside)."""
    T = 5
    x64 = np.random.default_rng(d).normal(size=(T, d)) * scale
    h = torch.from_numpy(x64).to(torch.bfloat16).cuda()
    h[4] = _bf16(d, seed=7)  # an ordinary row beside them
    w = _bf16(d, seed=d)
    # (so that dx is a bf16 number: dy / scale)
    dy, dh = _bf16(T, d, seed=1, std=1e-3 if scale < 1 else 1e3), _bf16(T, d, seed=2, std=1e-3)
    eps = float(np.float32(eps))
    dx, dw = moe.rmsnorm_grad(dy, h, w, dh, eps)
    dy64, h64, w64 = f64(dy), f64(h), f64(w)
    ref, refw = R.rmsnorm_grad(dy64, h64, w64, eps)
    r = 1 / np.sqrt((h64 ** 2).mean(-1, keepdims=True) + eps)
    g, n = dy64 * w64, h64 * r
    terms = r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(-1, keepdims=True)) + np.abs(f64(dh))
    ref = ref + f64(dh)
    assert (np.abs(f64(dx) - ref) <= np.abs(ref) * 2.0 ** -8 + terms * 2 * Y + 2.0 ** -133).all()
    assert (np.abs(f64(dw) - refw) <= (1 + 16 + 32 + 14) * 2.0 ** -24 * np.abs(dy64 * n).sum(0)).all()


def test_rmsnorm_grad_of_non_finite_rows(moe):
    """An infinity or NaN in h makes its row of dx NaN; an infinite dy makes mean(g n) infinite and so its
    row of dx, g - n mean(g n), infinite or (at its own place) NaN.  The other rows are left."""
    T, d = 6, 4104
    h, dy, w = _bf16(T, d, seed=1), _bf16(T, d, seed=2), _bf16(d, seed=3)
    want, _ = moe.rmsnorm_grad(dy, h, w, None, EPS)
    h[1, 5], h[3, 4103], dy[4, 0] = float("inf"), float("nan"), float("-inf")
    dx, dw = moe.rmsnorm_grad(dy, h, w, None, EPS)
    assert dx[[1, 3]].isnan().all() and dx[4].isfinite().logical_not().all() and dx[4, 0].isnan()
    assert torch.equal(dx[[0, 2, 5]], want[[0, 2, 5]])
    assert dw[5].isnan() and dw[4103].isnan()


@pytest.mark.parametrize("size", [0.9, 6.0])
@pytest.mark.parametrize("d", [64, 256, 1024, 8192])
def test_rmsnorm_grad_of_products_past_fp32(moe, d, size):
    """Ordinary rows whose dy * weight * h passes fp32's range in the sum, with a dx that does not: rows of
    mean square below and above one."""
    g = torch.Generator().manual_seed(d)
    h = (torch.randint(0, 2, (2, d), generator=g) * 2 - 1).to(torch.bfloat16).mul_(size).cuda()
    dy = (torch.rand(2, d, generator=g) + 1).mul_(8e37 if size < 1 else 5e37).to(torch.bfloat16).cuda()
    w = (torch.rand(d, generator=g) * 0.5 + 0.5).to(torch.bfloat16).cuda()
    dx, dw = moe.rmsnorm_grad(dy, h, w, None, EPS)
    dy64, h64, w64 = f64(dy), f64(h), f64(w)
    chains = (dy64 * w64 * h64).reshape(2, -1, 8).cumsum(-1)
    assert np.abs(chains).max() > 3.5e38
    ref, refw = R.rmsnorm_grad(dy64, h64, w64, EPS)
    r = 1 / np.sqrt((h64 ** 2).mean(-1, keepdims=True) + EPS)
    gg, n = dy64 * w64, h64 * r
    terms = r * (np.abs(gg) + np.abs(n) * np.abs(gg * n).mean(-1, keepdims=True))
    assert np.abs(ref).max() < 3e38
    assert (np.abs(f64(dx) - ref) <= np.abs(ref) * 2.0 ** -8 + terms * 2 * Y).all()
    if np.abs(refw).max() < 3e38:
        assert (np.abs(f64(dw) - refw) <= (1 + 16 + 32 + 14) * 2.0 ** -24 * np.abs(dy64 * n).sum(0)).all()


@pytest.mark.parametrize("dy_size,h_size", [(1e-30, 1e-9), (1e-36, 1e-4), (1e-28, 1e-14), (1e-38, 1e-6)])
@pytest.mark.parametrize("d", [256, 8192])
def test_rmsnorm_grad_of_products_below_fp32(moe, d, dy_size, h_size):
    """dy * weight * h below the smallest normal float, of rows in fp32's range: mean(g n) keeps its bits."""
    h, dy, w = _bf16(3, d, seed=1, std=h_size), _bf16(3, d, seed=2, std=dy_size), _bf16(d, seed=3)
    dy = (dy.float() + 3 * h.float() * (dy_size / h_size)).to(torch.bfloat16)  # (a mean(g n) that counts)
    dy[1] = 0
    dx, _ = moe.rmsnorm_grad(dy, h, w, None, 0.0)
    dy64, h64, w64 = f64(dy), f64(h), f64(w)
    ref, _ = R.rmsnorm_grad(dy64, h64, w64, 0.0)
    r = 1 / np.sqrt((h64 ** 2).mean(-1, keepdims=True))
    g, n = dy64 * w64, h64 * r
    terms = r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(-1, keepdims=True) + 2.0 ** -149)
    assert (np.abs(f64(dx) - ref) <= np.abs(ref) * 2.0 ** -8 + terms * 2 * Y + r * 2.0 ** -148).all()
    assert not dx[1].any()


@pytest.mark.parametrize("T", [8192, 65536, 65537, 300000, 2 ** 21 + 5, 2 ** 25 - 1])
def test_rmsnorm_grad_sums_over_long_columns(moe, T):
    """Equal rows of whole numbers, without eps: a column is T times one fp32 product, whose additions a chain of
    fp32 would round the same way each.  At most 128 rows of a workgroup one behind another, 16 and then 32 sums."""
    d, v = 8, np.array([[3.0, 7.0, -11.0, 13.0, 1.0, -5.0, 2.0, 9.0]], np.float32)
    n = (v * (np.float32(1) / np.sqrt(np.float32((v.astype(np.float64) ** 2).sum() / d)))).astype(np.float64)[0]
    row = torch.from_numpy(v).to(torch.bfloat16).cuda()
    one = torch.ones_like(row)
    dw = moe.rmsnorm_grad(one.expand(T, d).contiguous(), row.expand(T, d).contiguous(), one[0], None, 0.0)[1]
    assert (np.abs(f64(dw) - T * n) <= (128 + 16 + 32 + 2) * 2.0 ** -24 * T * np.abs(n)).all()
