"""GPU: the norms around a block and their gradient, against float64.

Tolerances count roundings, u = 2^-24.  A norm's value is within 12 u of the exact one (test_gpu_norm.py);
gate, scale and the residual's product and sum add 5 u: h before its rounding is within 2^-19 of the magnitude
of its two terms, and bf16 adds 2^-8.  Gradients: two norms' backward passes one behind the other, each
within 2^-19 of the magnitudes it adds: 2^-17 over both, and the output's 2^-8 for bf16; sums over rows
add one u per row of a workgroup and of the sum of workgroups."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_top_amd import moe as _moe
from oracle import block as B
from oracle import rows as R

from test_gpu_norm import ACTS, RANGE, Y, check_forward, f64, values

pytestmark = pytest.mark.gpu
EPS = 1e-6
H, G, BF = 2.0 ** -19, 2.0 ** -17, 2.0 ** -8


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _moe.lib()
    return _moe


def _bf16(*shape, seed=0, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(torch.bfloat16).cuda()


def _gate(kind, T, d):
    return {"none": None, "channel": _bf16(d, seed=7, std=0.3), "token": _bf16(T, d, seed=8, std=0.3)}[kind]


def n64(t):
    return None if t is None else f64(t)


def check_block(moe, act, x, r, pre, post, gate, rs, bs, out, eps=EPS):
    h, y, q, qs = out
    ref, mag, _ = B.block_norm(f64(x), f64(r), n64(post), n64(gate), f64(pre), rs, bs, eps)
    assert h.dtype == x.dtype and (np.abs(f64(h) - ref) <= np.abs(ref) * BF + mag * H + 2.0 ** -133).all()
    if eps == EPS:
        check_forward(moe, act, h, pre, None, h, y, q, qs)  # the rest of the way, from the h that was kept
    elif y is not None:
        want = R.rmsnorm(f64(h), f64(pre), eps)
        assert (np.abs(f64(y) - want) <= np.abs(want) * (BF + Y) + 2.0 ** -133).all()


SHAPES = [(1, 128), (3, 128), (1, 7168), (5, 512), (77, 4096), (130, 640), (2, 4224), (9, 8192), (3, 12288),
          (2, 32768), (1100, 256), (1030, 2176)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("fmt", ACTS)
def test_block_norm(moe, fmt, T, d):
    x, r, pre = _bf16(T, d, seed=T + d), _bf16(T, d, seed=T + d + 1, std=2.0), _bf16(d, seed=d)
    i = T + d // 128
    post = _bf16(d, seed=d + 1) if i % 4 else None
    gate = _gate(("none", "channel", "token")[i % 3], T, d)
    rs, bs = ((1.0, 1.0), (0.5, 0.22))[i % 2]
    rs, bs = float(np.float32(rs)), float(np.float32(bs))
    out = moe.block_norm(x, r, pre, post, gate, rs, bs, EPS, ACTS[fmt])
    check_block(moe, ACTS[fmt], x, r, pre, post, gate, rs, bs, out)
    if fmt != "bf16":
        o2 = moe.block_norm(x, r, pre, post, gate, rs, bs, EPS, ACTS[fmt], want_y=False)
        assert o2[1] is None and torch.equal(o2[0], out[0]) and torch.equal(o2[2], out[2])


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("T,d", [(4, 8), (7, 200), (6, 4104), (1025, 72)])
def test_block_norm_odd_rows(moe, post, gate, T, d):
    x, r, pre = _bf16(T, d, seed=1), _bf16(T, d, seed=2), _bf16(d, seed=3)
    post, gate = _bf16(d, seed=4) if post else None, _gate(gate, T, d)
    check_block(moe, 0, x, r, pre, post, gate, -1.5, 0.75, moe.block_norm(x, r, pre, post, gate, -1.5, 0.75))


def test_block_norm_without_a_step_is_rmsnorm(moe):
    """No norm behind the block, no gate, scales of 1: rmsnorm with a residual, bit for bit."""
    x, r, pre = _bf16(9, 1024, seed=1), _bf16(9, 1024, seed=2), _bf16(1024, seed=3)
    for act in ACTS.values():
        for a, b in zip(moe.block_norm(x, r, pre, act_dtype=act), moe.rmsnorm(x, pre, r, EPS, act)):
            assert (a is None and b is None) or torch.equal(a, b)


def test_block_norm_int16_bits_and_zero_tokens(moe):
    x, r, w = _bf16(4, 256, seed=1), _bf16(4, 256, seed=2), _bf16(256, seed=3)
    i16 = lambda t: t.view(torch.int16)  # noqa: E731
    a = moe.block_norm(x, r, w, w, x)
    b = moe.block_norm(i16(x), i16(r), i16(w), i16(w), i16(x))
    assert all(q.dtype == torch.int16 and torch.equal(i16(p), q) for p, q in zip(a[:2], b[:2]))
    h, y, q, qs = moe.block_norm(x[:0], r[:0], w, w, x[:0], act_dtype=moe.DTYPE_INT8)
    assert h.shape == y.shape == q.shape == (0, 256) and qs.shape == (0,)
    dx, dr, dp, dq, dg = moe.block_norm_grad(x[:0], x[:0], x[:0], w, post_weight=w, gate=w)
    assert dx.shape == dr.shape == (0, 256) and not dp.any() and not dq.any() and not dg.any()


def test_block_norm_in_place_and_neighbours(moe):
    """h_out may be x or the residual; rows behind the last one stay as they were."""
    T, d = 5, 4224
    x, r, pre, post = _bf16(T + 2, d, seed=1), _bf16(T + 2, d, seed=2), _bf16(d, seed=3), _bf16(d, seed=4)
    gate = _bf16(d, seed=5)
    want = moe.block_norm(x[:T], r[:T], pre, post, gate, 0.5, 2.0, EPS, moe.DTYPE_FP8)
    for inplace in ("residual", "x"):
        a, b = x.clone(), r.clone()
        out = b if inplace == "residual" else a
        keep = out[T:].clone()
        y = torch.full_like(x, 7.0)
        q = torch.full((T + 2, d), 77, dtype=torch.uint8, device="cuda")
        qs = torch.full((T + 2, d // 128), 7.0, device="cuda")
        blk = moe.Block(post.data_ptr(), gate.data_ptr(), pre.data_ptr(), 0, 0.5, 2.0, EPS)
        st = torch.cuda.current_stream().cuda_stream
        assert moe.lib().moe_block_norm(blk, a.data_ptr(), b.data_ptr(), T, d, moe.DTYPE_FP8, out.data_ptr(),
                                        y.data_ptr(), q.data_ptr(), qs.data_ptr(), st) == 0
        for got, w in zip((out, y, q, qs), want):
            assert torch.equal(got[:T], w)
        assert torch.equal(out[T:], keep) and (y[T:] == 7).all() and (q[T:] == 77).all() and (qs[T:] == 7).all()


@pytest.mark.parametrize("fmt", ACTS)
def test_block_norm_zero_and_non_finite_rows(moe, fmt):
    """A zero branch leaves the residual; an infinity or NaN makes its own row NaN and no other."""
    act, T, d = ACTS[fmt], 7, 384
    x, r, pre, post = _bf16(T, d, seed=9), _bf16(T, d, seed=8), _bf16(d, seed=3), _bf16(d, seed=4)
    clean = moe.block_norm(x, r, pre, post, act_dtype=act)
    bx, br = x.clone(), r.clone()
    bx[1] = 0
    bx[2, 5], bx[3, 383], br[4, 0] = float("inf"), float("nan"), float("-inf")
    bx[5], br[5] = 0, 0
    h, y, q, qs = moe.block_norm(bx, br, pre, post, act_dtype=act)
    assert torch.equal(y[[0, 6]], clean[1][[0, 6]]) and torch.equal(h[1], r[1])
    assert (y[5] == 0).all() and y[2:5].isnan().all() and h[2:4].isnan().all()
    if act != moe.DTYPE_BF16:
        v, _ = values(moe, act, q, qs, d)
        assert np.isnan(v[2:5]).all() and (v[5] == 0).all() and np.isfinite(v[[0, 1, 6]]).all()


@pytest.mark.parametrize("scale,eps", RANGE, ids=str)
@pytest.mark.parametrize("d", [256, 4224, 16384])
def test_block_norm_of_every_magnitude(moe, d, scale, eps):
    """Block outputs whose squares leave fp32's range beside an ordinary row: the norm brings them to one."""
    x = torch.from_numpy(np.random.default_rng(d).normal(size=(5, d)) * scale).to(torch.bfloat16).cuda()
    x[4] = 1
    r, pre, post = _bf16(5, d, seed=2), _bf16(d, seed=3), _bf16(d, seed=4)
    eps = float(np.float32(eps))
    out = moe.block_norm(x, r, pre, post, None, 1.0, 0.5, eps)
    check_block(moe, 0, x, r, pre, post, None, 1.0, 0.5, out, eps)


def check_grad(dy, dh, x, h, pre, post, gate, rs, bs, out, eps=EPS, tiny=2.0 ** -133):
    T, d = dy.shape
    ref = B.block_norm_grad(f64(dy), n64(dh), f64(x), f64(h), n64(post), n64(gate), f64(pre), rs, bs, eps)
    depth = (-(-T // 512) + 16 + 32) * 2.0 ** -24
    for name, got in zip(("dx", "dres", "dpre", "dpost", "dgate"), out):
        if name not in ref:
            assert got is None
            continue
        if got is None:
            continue
        rows = ref[name].ndim == 2
        assert got.dtype == (dy.dtype if rows else torch.float32) and got.shape == ref[name].shape
        tol = ref["e_" + name] * (G + (0 if rows else depth)) + (np.abs(ref[name]) * BF + tiny if rows else 0)
        assert (np.abs(f64(got) - ref[name]) <= tol).all(), name


GRAD_SHAPES = [(1, 8), (1, 7168), (3, 128), (5, 520), (77, 1024), (200, 4104), (600, 256), (1030, 2048), (1600, 136),
               (33, 8192), (7, 12288), (3, 16384), (70, 4096)]


@pytest.mark.parametrize("T,d", GRAD_SHAPES)
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_grad(moe, T, d, gate, post):
    x, r, pre = _bf16(T, d, seed=T), _bf16(T, d, seed=T + 1, std=2.0), _bf16(d, seed=d)
    post, gate = _bf16(d, seed=d + 1) if post else None, _gate(gate, T, d)
    h = moe.block_norm(x, r, pre, post, gate, 0.5, 0.25)[0]
    dy = _bf16(T, d, seed=T + 2, std=0.1)
    for dh in (None, _bf16(T, d, seed=3, std=0.1)):
        a = (dy, x, h, pre, dh, post, gate, 0.5, 0.25)
        out = moe.block_norm_grad(*a)
        check_grad(dy, dh, x, h, pre, post, gate, 0.5, 0.25, out)
        for p, q in zip(out, moe.block_norm_grad(*a)):  # fixed order
            assert (p is None and q is None) or torch.equal(p, q)
    few = moe.block_norm_grad(*a, want_sums=False)
    assert few[2] is None and few[3] is None and torch.equal(few[0], out[0]) and torch.equal(few[1], out[1])
    if gate is not None and gate.dim() == 2:
        assert torch.equal(few[4], out[4])
    else:
        assert few[4] is None


def test_block_norm_grad_is_rmsnorm_grads(moe):
    """Without gate, scales and a norm behind the block: dx and dresidual are rmsnorm_grad's dx."""
    T, d = 40, 1024
    x, h, pre, dy, dh = (_bf16(T, d, seed=i) if i != 2 else _bf16(d, seed=2) for i in range(5))
    dx, dr, dp, _, _ = moe.block_norm_grad(dy, x, h, pre, dh)
    want, dw = moe.rmsnorm_grad(dy, h, pre, dh)
    assert torch.equal(dx, dr)
    near = lambda a, b, t: ((a.double() - b.double()).abs() <= t * (a.double().abs() + b.double().abs()) + 1e-4 * t).all()  # noqa: E731,E501
    assert near(dx, want, 2 * BF) and near(dp, dw, 2.0 ** -12)


def test_block_norm_grad_in_place_and_neighbours(moe):
    T, d = 6, 4104
    dy, dh, x, h = (_bf16(T + 2, d, seed=i) for i in range(4))
    pre, post, gate = _bf16(d, seed=5), _bf16(d, seed=6), _bf16(T + 2, d, seed=7)
    want = moe.block_norm_grad(dy[:T], x[:T], h[:T], pre, dh[:T], post, gate[:T])
    blk = moe.Block(post.data_ptr(), gate.data_ptr(), pre.data_ptr(), 1, 1.0, 1.0, EPS)
    st = torch.cuda.current_stream().cuda_stream
    for i, j in ((0, 1), (2, 0), (1, 3), (0, 3), (2, 1)):
        a = [t.clone() for t in (dy, dh, x, h)]
        dg = torch.full_like(gate, 7.0)
        keep = a[i][T:].clone(), a[j][T:].clone()
        assert moe.lib().moe_block_norm_grad(blk, a[0].data_ptr(), a[1].data_ptr(), a[2].data_ptr(), a[3].data_ptr(),
                                             T, d, a[i].data_ptr(), a[j].data_ptr(), None, None, dg.data_ptr(), None,
                                             0, st) == 0
        assert torch.equal(a[i][:T], want[0]) and torch.equal(a[j][:T], want[1]) and torch.equal(dg[:T], want[4])
        assert torch.equal(a[i][T:], keep[0]) and torch.equal(a[j][T:], keep[1]) and (dg[T:] == 7).all()


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_block_norm_grad_against_differences(moe, gate):
    """All gradients against central differences of the float64 block, along one direction each: their bf16
    and fp32 errors, summed with the direction's magnitudes, bound the gap."""
    T, d, rs, bs = 3, 256, 0.5, 0.75
    x, r, pre, post, gate = _bf16(T, d, seed=1), _bf16(T, d, seed=2), _bf16(d, seed=3), _bf16(d, seed=4), _gate(gate, T, d)
    dy, dh = _bf16(T, d, seed=5), _bf16(T, d, seed=6)
    # (the backward pass at the rounded h: the same h is the block's at a residual moved by the rounding)
    h = moe.block_norm(x, r, pre, post, gate, rs, bs)[0]
    exact = B.block_norm(f64(x), f64(r), f64(post), n64(gate), f64(pre), rs, bs, EPS)[0]
    r64 = f64(r) + (f64(h) - exact) / rs
    got = dict(zip(("x", "r", "pre", "post", "gate"), moe.block_norm_grad(dy, x, h, pre, dh, post, gate, rs, bs)))
    at = dict(x=f64(x), r=r64, pre=f64(pre), post=f64(post), gate=n64(gate))

    def f(a):
        h, _, y = B.block_norm(a["x"], a["r"], a["post"], a["gate"], a["pre"], rs, bs, EPS)
        return (y(h) * f64(dy)).sum() + (h * f64(dh)).sum()

    ref = B.block_norm_grad(f64(dy), f64(dh), f64(x), f64(h), f64(post), n64(gate), f64(pre), rs, bs, EPS)
    for name, key in (("x", "dx"), ("r", "dres"), ("pre", "dpre"), ("post", "dpost"), ("gate", "dgate")):
        if at[name] is None:
            continue
        v = np.random.default_rng(1).normal(size=at[name].shape)
        e = 1e-5
        num = (f(dict(at, **{name: at[name] + e * v})) - f(dict(at, **{name: at[name] - e * v}))) / (2 * e)
        g = f64(got[name])
        rows = g.ndim == 2
        room = ((np.abs(g) * (BF if rows else 0) + 2 * G * ref["e_" + key]) * np.abs(v)).sum()
        assert abs(num - (g * v).sum()) <= room + 1e-5, name


@pytest.mark.parametrize("scale,eps", RANGE, ids=str)
@pytest.mark.parametrize("which", ["x", "h"])
@pytest.mark.parametrize("d", [256, 4104, 16384])
def test_block_norm_grad_of_every_magnitude(moe, d, which, scale, eps):
    """Rows of x or of h whose squares leave fp32's range, beside an ordinary one."""
    T = 5
    big = torch.from_numpy(np.random.default_rng(d).normal(size=(T, d)) * scale).to(torch.bfloat16).cuda()
    big[4] = _bf16(d, seed=7)
    x, h = (big, _bf16(T, d, seed=1)) if which == "x" else (_bf16(T, d, seed=1), big)
    pre, post = _bf16(d, seed=3), _bf16(d, seed=4)
    std = 1e-3 if scale < 1 else 1e3
    dy, dh = _bf16(T, d, seed=5, std=std), _bf16(T, d, seed=6, std=1e-3)
    gate = _bf16(d, seed=8, mean=1.0, std=0.1)
    eps = float(np.float32(eps))
    ref = B.block_norm_grad(f64(dy), f64(dh), f64(x), f64(h), f64(post), f64(gate), f64(pre), 1.0, 0.5, eps)
    if max(np.abs(ref[n]).max() for n in ("e_dx", "e_dres", "e_dpost", "e_dgate")) > 1e38:
        dy = (dy.float() * min(1.0, scale)).to(torch.bfloat16)  # (so that the gradients are bf16 numbers)
    out = moe.block_norm_grad(dy, x, h, pre, dh, post, gate, 1.0, 0.5, eps)
    # (half a step of the smallest float inside, times what the last root multiplies it by)
    r = (1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + eps)).max()
    check_grad(dy, dh, x, h, pre, post, gate, 1.0, 0.5, out, eps, 2.0 ** -133 + r * 2.0 ** -147)


def test_block_norm_grad_of_non_finite_rows(moe):
    T, d = 6, 4104
    x, h, dy = _bf16(T, d, seed=1), _bf16(T, d, seed=2), _bf16(T, d, seed=3)
    pre, post = _bf16(d, seed=4), _bf16(d, seed=5)
    want = moe.block_norm_grad(dy, x, h, pre, None, post)
    x[1, 5], h[3, 4103], dy[4, 0] = float("inf"), float("nan"), float("-inf")
    dx, dr, dp, dq, _ = moe.block_norm_grad(dy, x, h, pre, None, post)
    assert dx[[1, 3]].isnan().all() and dr[3].isnan().all() and not dr[4].isfinite().any() and not dx[4].isfinite().any()
    assert torch.equal(dx[[0, 2, 5]], want[0][[0, 2, 5]]) and torch.equal(dr[[0, 1, 2, 5]], want[1][[0, 1, 2, 5]])
    assert dp[4103].isnan() and dq[5].isnan()


@pytest.mark.parametrize("d", [512, 1024, 2048, 4096, 8192, 16384])
def test_block_norm_grad_row_sums_past_24_bits(moe, d):
    """Whole numbers, whose squares sum to more than fp32 holds: eight at a time they are exact in fp32, and a
    row's are in fp64, so that both roots are those of the exact mean, bit for bit."""
    rng = np.random.default_rng(d)
    one, zero = torch.ones(1, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, d, dtype=torch.bfloat16, device="cuda")
    for _ in range(24):
        v = rng.integers(-256, 257, (1, d)).astype(np.float32)
        t = torch.from_numpy(v).to(torch.bfloat16).cuda()
        n = v * (np.float32(1) / np.sqrt(np.float32((v.astype(np.float64) ** 2).sum() / d)))
        # dpre = dy n2; with dy = 0 H is dh, and dpost = H n1
        dpre = moe.block_norm_grad(one, one, t, one[0], eps=0.0)[2]
        dpost = moe.block_norm_grad(zero, t, one, one[0], one, one[0], eps=0.0)[3]
        assert np.array_equal(dpre.cpu().numpy(), n[0]) and np.array_equal(dpost.cpu().numpy(), n[0])


@pytest.mark.parametrize("T", [63, 64, 65, 127, 128, 129, 130, 1023, 1024, 1025, 1026])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_block_norm_grad_row_shares(moe, T, gate):
    """As many workgroups as rows, one with two, and full ones beside one that is not."""
    d = 72
    x, h, dy, dh = (_bf16(T, d, seed=i) for i in range(4))
    pre, post, gate = _bf16(d, seed=5), _bf16(d, seed=6), _gate(gate, T, d)
    a = (dy, x, h, pre, dh, post, gate, 0.5, 0.25)
    out = moe.block_norm_grad(*a)
    check_grad(dy, dh, x, h, pre, post, gate, 0.5, 0.25, out)
    assert moe.lib().moe_block_norm_grad_workspace_bytes(T, d) >= 8 * d * min(T, 64)


@pytest.mark.parametrize("T", [8192, 65536, 65537, 300000, 2 ** 21 + 5, 2 ** 25 - 1])
@pytest.mark.parametrize("token", [False, True])
def test_block_norm_grad_sums_over_long_columns(moe, T, token):
    """Equal rows: a column is T times one fp32 product (whole numbers, eps 0: test_..._past_24_bits), whose
    additions a chain of fp32 would round the same way each.  At most 128 rows of a workgroup one behind another, 16
    and then 32 sums: 176 u, and a gate's and the output's roundings."""
    d, v = 8, np.array([[3.0, 7.0, -11.0, 13.0, 1.0, -5.0, 2.0, 9.0]], np.float32)
    row = torch.from_numpy(v).to(torch.bfloat16).cuda()
    n = (v * (np.float32(1) / np.sqrt(np.float32((v.astype(np.float64) ** 2).sum() / d)))).astype(np.float64)[0]
    one, pre = torch.ones(1, d, dtype=torch.bfloat16, device="cuda").expand(T, d).contiguous(), row.new_ones(d)
    rows = row.expand(T, d).contiguous()
    gate = 2 * one if token else 2 * pre
    _, _, dpre, _, _ = moe.block_norm_grad(one, one, rows, pre, eps=0.0)
    _, _, _, dpost, dgate = moe.block_norm_grad(torch.zeros_like(one), rows, one, pre, one, pre, gate, eps=0.0)
    got = [(dpre, 1), (dpost, 2)] + ([] if token else [(dgate, 1)])
    for g, f in got:
        assert (np.abs(f64(g) - f * T * n) <= (128 + 16 + 32 + 2) * 2.0 ** -24 * f * T * np.abs(n)).all()


@pytest.mark.parametrize("T,d", [(8192, 264), (70001, 40), (300000, 16)])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_block_norm_grad_of_many_rows(moe, T, d, gate):
    """Products of one sign, so that nothing cancels on the way."""
    x, h, dy, dh = (_bf16(T, d, seed=i, mean=2.0, std=0.3) for i in range(4))
    pre, post, gate = _bf16(d, seed=5, mean=1.0, std=0.1), _bf16(d, seed=6, mean=1.0, std=0.1), _gate(gate, T, d)
    out = moe.block_norm_grad(dy, x, h, pre, dh, post, gate, 0.5, 0.25)
    ref = B.block_norm_grad(f64(dy), f64(dh), f64(x), f64(h), f64(post), f64(gate), f64(pre), 0.5, 0.25, EPS)
    for name, g in zip(("dpre", "dpost", "dgate"), out[2:]):
        if ref[name].ndim == 1:
            assert (np.abs(f64(g) - ref[name]) <= ref["e_" + name] * (G + 178 * 2.0 ** -24)).all(), name


@pytest.mark.parametrize("T,d", [(1000, 256), (30000, 64), (1100, 7168)])
def test_block_norm_root_is_rounded_once(moe, T, d):
    """Whole numbers without eps, whose mean squares are exact where d is a power of two: h = bf16(fp32(x root)), bit
    for bit, with the one fp32 number that is nearest to the root (rows where that is a close call, 2^-40, aside)."""
    rng = np.random.default_rng(d)
    v = rng.integers(-200, 201, (T, d))
    x = torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).cuda()
    one, zero = torch.ones(d, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(x)
    h = moe.block_norm(x, zero, one, one, None, 0.0, 1.0, 0.0)[0]
    root = 1 / np.sqrt((v ** 2).sum(1, keepdims=True) / np.float64(d))
    near = root.astype(np.float32)
    gap = np.abs(np.abs(root - near) / np.spacing(near) - 0.5)  # (from a half step)
    sure = (gap > 2.0 ** -16)[:, 0]
    want = torch.from_numpy(v.astype(np.float32) * near).to(torch.bfloat16)
    assert sure.mean() > 0.99 and torch.equal(h.cpu()[sure], want[sure])


def test_block_norm_past_32_bit_offsets(moe):
    """More than 2^32 bytes per tensor: every fourth row is the same row."""
    d = 7168
    T = 2 ** 31 // d // 4 * 4 + 400
    x, r, gate = _bf16(4, d, seed=1), _bf16(4, d, seed=2), _bf16(4, d, seed=3)
    pre, post = _bf16(d, seed=4), _bf16(d, seed=5)
    many = lambda t: t.repeat(T // 4, 1)  # noqa: E731
    few = moe.block_norm(x, r, pre, post, gate, act_dtype=moe.DTYPE_INT8)
    got = moe.block_norm(many(x), many(r), pre, post, many(gate), act_dtype=moe.DTYPE_INT8)
    for a, b in zip(got, few):
        assert torch.equal(a.view(T // 4, 4, -1), b.view(1, 4, -1).expand(T // 4, 4, -1))
    del got
    dy, dh, h = _bf16(4, d, seed=6), _bf16(4, d, seed=7), few[0]
    w = moe.block_norm_grad(dy, x, h, pre, dh, post, gate)
    g = moe.block_norm_grad(many(dy), many(x), many(h), pre, many(dh), post, many(gate))
    for i in (0, 1, 4):
        assert torch.equal(g[i].view(T // 4, 4, d), w[i].expand(T // 4, 4, d))


def test_block_norm_of_the_most_rows(moe):
    """2^25 - 1 rows, forward and backward: the first and the last are those of a small call."""
    T = 2 ** 25 - 1
    x, r, g = _bf16(7, 8, seed=9), _bf16(7, 8, seed=10), _bf16(7, 8, seed=11)
    pre, post = _bf16(8, seed=12), _bf16(8, seed=13)

    def spread(t):
        o = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
        o[:7], o[-7:] = t, t
        return o

    h, y = moe.block_norm(x, r, pre, post)[:2]
    H_, Y_ = moe.block_norm(spread(x), spread(r), pre, post)[:2]
    w = moe.block_norm_grad(g, x, h, pre, None, post)
    W_ = moe.block_norm_grad(spread(g), spread(x), H_, pre, None, post)
    for big, small in ((H_, h), (Y_, y), (W_[0], w[0]), (W_[1], w[1])):
        assert torch.equal(big[:7], small) and torch.equal(big[-7:], small) and not big[7:-7].any()
