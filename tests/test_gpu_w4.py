"""GPU: products with 4-bit weights, and what surrounds a block run together, against float64.

A product's terms are exact; a group's fp32 sum makes at most `group` roundings, its scaling one, the sum over
groups and over the wavefronts' shares K / group + 4 more: within (group + K / group + 8) 2^-24 of the
terms' magnitudes, then bf16's 2^-8.  SwiGLU: that of its two sums, and (|g| + 16) 2^-22 for the
exponential's argument and the products."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_top_amd import moe as _moe
from oracle import block as B

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


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


def _w(N, K, group, zeros, seed=0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = (torch.rand(N, K // group, generator=g) * 0.02 + 0.001).to(dtype)
    z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zeros else None
    return codes.cuda(), s.cuda(), None if z is None else z.cuda()


def values(w, group):
    return B.w4_values(w[0].cpu().numpy(), f64(w[1]), None if w[2] is None else w[2].cpu().numpy(), group)


def check(x, y, w, up, group):
    K = x.shape[1]
    a = values(w, group)
    ref, mag = B.gemm_w4(f64(x), a, None if up is None else values(up, group))
    tol = np.abs(ref) * BF + mag * (group + K / group + 8) * 2.0 ** -24
    if up is not None:
        tol += np.abs(ref) * (np.abs(f64(x) @ a.T) + 16) * 2.0 ** -22
    assert y.dtype == torch.bfloat16 and y.shape == ref.shape
    assert (np.abs(f64(y) - ref) <= tol).all()


SHAPES = [(1, 16, 128), (1, 2048, 7168), (2, 48, 256), (3, 16, 384), (5, 208, 640), (8, 512, 1024), (15, 32, 128),
          (16, 1024, 4096), (17, 64, 512), (31, 80, 896), (33, 272, 1152), (47, 144, 256), (64, 640, 2048), (65, 528, 384),
          (100, 256, 256), (128, 2048, 512), (129, 272, 128), (200, 1024, 640), (257, 1040, 1024), (300, 16, 256),
          (513, 4096, 256), (1000, 1424, 1024)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("pair", [False, True])
def test_gemm_w4(moe, M, N, K, group, zeros, pair):
    x = _bf16(M, K, seed=M)
    dtype = torch.float16 if (M + N // 16) % 2 else torch.bfloat16
    w = _w(N, K, group, zeros, N, dtype)
    up = _w(N, K, group, zeros, N + 1, dtype) if pair else None
    t = moe.w4_tile(*w)
    y = moe.gemm_w4(x, t, moe.w4_tile(*up) if pair else None)
    check(x, y, w, up, group)


def test_gemm_w4_one_matrix_with_zeros(moe):
    """The gate with zero points and the up matrix without, and the other way round."""
    x = _bf16(20, 512, seed=1)
    a, b = _w(96, 512, 64, True, 1), _w(96, 512, 64, False, 2)
    check(x, moe.gemm_w4(x, moe.w4_tile(*a), moe.w4_tile(*b)), a, b, 64)
    check(x, moe.gemm_w4(x, moe.w4_tile(*b), moe.w4_tile(*a)), b, a, 64)
    x = x[:3].contiguous()
    check(x, moe.gemm_w4(x, moe.w4_tile(*a), moe.w4_tile(*b)), a, b, 64)
    check(x, moe.gemm_w4(x, moe.w4_tile(*b), moe.w4_tile(*a)), b, a, 64)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemm_w4_every_code(moe, M, group):
    """One value of x at a time picks out single weights: code, zero point and scale are exact, so the product
    is the exact weight rounded once."""
    N, K = 64, 256
    codes, s, _ = _w(N, K, group, False, 3)
    codes[:, :128] = torch.arange(N * 128, device="cuda").reshape(N, 128).to(torch.uint8)
    z = torch.randint(0, 128, (N, K // group), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).cuda()
    for zeros in (None, z):
        w = (codes, s, zeros)
        t = moe.w4_tile(*w)
        want = torch.from_numpy(values(w, group)).to(torch.bfloat16).cuda()
        for k0 in range(0, K, M):
            x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
            n = min(M, K - k0)
            x[torch.arange(n), k0 + torch.arange(n)] = 1
            assert torch.equal(moe.gemm_w4(x, t)[:n], want[:, k0:k0 + n].t())
            if M == 1 and k0 > 40:
                break


@pytest.mark.parametrize("M", [1, 16, 33, 128, 300])
def test_gemm_w4_large_and_non_finite_values(moe, M):
    """x near bf16's largest value with scales that bring it back; an infinity, a NaN reach their row alone."""
    N, K = 128, 512
    codes, s, z = _w(N, K, 128, True, 5)
    w = (codes, (s.float() * 1e-30).to(torch.bfloat16), z)
    t = moe.w4_tile(*w)
    x = (_bf16(M, K, seed=1).float() * 1e34).to(torch.bfloat16)
    check(x, moe.gemm_w4(x, t), w, None, 128)
    t = moe.w4_tile(codes, s, z)
    x = _bf16(M, K, seed=2)
    clean = moe.gemm_w4(x, t)
    x[M // 2, 7] = float("nan")
    x[M - 1, 300] = float("inf")
    y = moe.gemm_w4(x, t)
    bad = sorted({M // 2, M - 1})
    assert not y[bad].isfinite().any()
    rest = [i for i in range(M) if i not in bad]
    assert torch.equal(y[rest], clean[rest])
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    assert not moe.gemm_w4(x, t).any()


@pytest.mark.parametrize("M", [1, 16, 33, 64, 128, 300])
@pytest.mark.parametrize("N", [128, 4096])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [None, 8, 127])
def test_gemm_w4_of_the_largest_x(moe, M, N, group, zero):
    """x just below 2^114, of one sign, by codes of 0: the largest sums of a group that are promised, 2^14 times x
    at most, are finite, and its scale brings them back."""
    K = 256
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.full((N, K // group), 2.0 ** -115, dtype=torch.bfloat16, device="cuda")
    w = (codes, s, None if zero is None else torch.full((N, K // group), zero, dtype=torch.uint8, device="cuda"))
    x = torch.full((M, K), 2.0 ** 114 * (1 - 2.0 ** -8), dtype=torch.bfloat16, device="cuda")
    check(x, moe.gemm_w4(x, moe.w4_tile(*w)), w, None, group)


@pytest.mark.parametrize("M", [1, 5, 16, 40, 70, 150, 300])
@pytest.mark.parametrize("pair", [False, True])
def test_gemm_w4_neighbours_and_repeat(moe, M, pair):
    """Rows behind the last stay as they were, x of other rows has no part, and a second call gives the same bits."""
    N, K = 208, 640
    w, up = moe.w4_tile(*_w(N, K, 32, True, 1)), moe.w4_tile(*_w(N, K, 32, True, 2)) if pair else None
    x = _bf16(M + 3, K, seed=3)
    x[M:] = float("nan")
    y = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert moe.lib().moe_gemm_w4(x.data_ptr(), M, w.struct(), up.struct() if pair else None, y.data_ptr(), st) == 0
    assert torch.equal(y[:M], moe.gemm_w4(x[:M].contiguous(), w, up)) and (y[M:] == 7).all()


def test_gemm_w4_zero_tokens_and_bits(moe):
    w = moe.w4_tile(*_w(32, 256, 64, False, 1))
    x = _bf16(3, 256, seed=1)
    assert moe.gemm_w4(x[:0], w).shape == (0, 32)
    y = moe.gemm_w4(x.view(torch.int16), w)
    assert y.dtype == torch.int16 and torch.equal(y, moe.gemm_w4(x, w).view(torch.int16))


def test_gemm_w4_past_32_bit_offsets(moe):
    """An output of more than 2^32 bytes, an x just below that, and codes of 2^31 values: every 64th row is the
    same row."""
    N, K, M = 4096 + 16, 128, 2 ** 20
    w = moe.w4_tile(*_w(N, K, 128, True, 1))
    x = _bf16(64, K, seed=1)
    few = moe.gemm_w4(x, w)
    y = moe.gemm_w4(x.repeat(M // 64, 1), w)
    # (a row's sums do not depend on how many rows there are only within one choice of tiles)
    assert ((y.view(-1, 64, N).float() - few.float()).abs() <= few.float().abs() * 2 * BF + 1e-2).all()
    del y
    K, M = 7168, 2 ** 31 // 7168 - 1
    w = moe.w4_tile(*_w(16, K, 32, False, 2))
    x = _bf16(3, K, seed=2)
    big = x.repeat(M // 3, 1)
    y, few = moe.gemm_w4(big, w), moe.gemm_w4(x, w)
    assert ((y.view(-1, 3, 16).float() - few.float()).abs() <= few.float().abs() * 2 * BF + 1e-1).all()
    del big, y
    N, K = 2 ** 17 - 16, 2 ** 14
    codes = torch.randint(0, 256, (64, K // 2), dtype=torch.uint8).cuda()
    s = torch.rand(64, K // 128).to(torch.bfloat16).cuda()
    few = moe.w4_tile(codes, s)
    big = moe.w4_tile(codes.repeat(2 ** 11, 1)[:N].contiguous(), s.repeat(2 ** 11, 1)[:N].contiguous())
    for M in (1, 200):
        x = _bf16(M, K, seed=3)
        y, want = moe.gemm_w4(x, big), moe.gemm_w4(x, few)
        want = want.repeat(1, 2 ** 11)[:, :N].float()
        assert ((y.float() - want).abs() <= want.abs() * 2 * BF + 1).all()


# Of a matrix of few columns so many weight rows (or rows of x) that the middling or the MFMA tiles take it: tiles of 128
# weight rows by 64 rows of x (more than half of 256 CUs), by 128 rows of x, and of 256 by 128 rows.
TILES = [(999, 3216, 256), (1000, 4096, 128), (97, 24592, 128), (33, 49168, 128), (1025, 2992, 1152), (6145 * 32, 16, 128),
         (250, 4224, 128), (130, 5520, 256), (70, 8336, 384), (64, 16400, 640), (33, 17000 // 16 * 16, 1152), (2000, 528, 512),
         (999, 8208, 256), (129, 22288, 128), (65, 33360, 384), (2100, 2080, 1280), (5000, 1040, 128), (300, 7152, 384), (120, 18416, 256),
         (8321, 128, 256), (17000, 48, 384), (9000, 144, 128)]


@pytest.mark.parametrize("M,N,K", TILES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("pair", [False, True])
def test_gemm_w4_many_tiles(moe, M, N, K, group, zeros, pair):
    assert (M + 63) // 64 * ((N + 127) // 128) > 128
    test_gemm_w4(moe, M, N, K, group, zeros, pair)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gemm_w4_many_tiles_of_a_pair(moe, zeros, dtype):
    """So few weight rows that only both matrices together are many tiles, the last of 16 or 80 rows; matrices with
    and without zero points."""
    for M, N, K, group in ((999, 1616, 256, 64), (600, 1040, 384, 32), (2100, 1168, 128, 128)):
        x, w, up = _bf16(M, K, seed=1), _w(N, K, group, zeros, 1, dtype), _w(N, K, group, True, 2, dtype)
        check(x, moe.gemm_w4(x, moe.w4_tile(*w), moe.w4_tile(*up)), w, up, group)


@pytest.mark.parametrize("N", [8976, 24592, 33360, 65552])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_gemm_w4_many_tiles_every_code(moe, N, group, zeros):
    """x a unit matrix: the product is the exact weights, rounded once."""
    K = 128
    codes, s, _ = _w(N, K, group, False, 3)
    codes[:, :64] = torch.arange(N * 64, device="cuda").reshape(N, 64).to(torch.uint8)
    z = torch.randint(0, 128, (N, K // group), generator=torch.Generator().manual_seed(1), dtype=torch.uint8)
    w = (codes, s, z.cuda() if zeros else None)
    want = torch.from_numpy(values(w, group)).to(torch.bfloat16).cuda()
    y = moe.gemm_w4(torch.eye(K, dtype=torch.bfloat16, device="cuda"), moe.w4_tile(*w))
    assert torch.equal(y, want.t())


@pytest.mark.parametrize("N", [1616, 3216, 8208])
def test_gemm_w4_many_tiles_neighbours_and_non_finite_values(moe, N):
    M, K = 999, 256
    w = moe.w4_tile(*_w(N, K, 32, True, 1))
    x = _bf16(M + 3, K, seed=3)
    x[M:] = float("nan")
    y = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert moe.lib().moe_gemm_w4(x.data_ptr(), M, w.struct(), None, y.data_ptr(), st) == 0
    x = x[:M].contiguous()
    clean = moe.gemm_w4(x, w)
    assert torch.equal(y[:M], clean) and (y[M:] == 7).all()
    x[500, 7], x[M - 1, 200] = float("nan"), float("inf")
    y = moe.gemm_w4(x, w)
    rest = [i for i in range(M) if i not in (500, M - 1)]
    assert not y[[500, M - 1]].isfinite().any() and torch.equal(y[rest], clean[rest])
    codes, s, z = _w(N, K, 128, True, 5)
    w = (codes, (s.float() * 1e-30).to(torch.bfloat16), z)
    x = (_bf16(M, K, seed=1).float() * 1e34).to(torch.bfloat16)
    check(x, moe.gemm_w4(x, moe.w4_tile(*w)), w, None, 128)


@pytest.mark.parametrize("N", [1616, 3216, 8208])
def test_gemm_w4_many_tiles_captured_and_on_two_streams(moe, N):
    """A captured call replayed with new inputs, and two at once, give the eager call's bits."""
    M, K = 999, 640
    w, up = moe.w4_tile(*_w(N, K, 64, True, 1)), moe.w4_tile(*_w(N, K, 64, False, 2))
    x, other = _bf16(M, K, seed=3), _bf16(M, K, seed=4)
    want = {0: moe.gemm_w4(x, w, up), 1: moe.gemm_w4(other, w, up)}
    a = x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = moe.gemm_w4(a, w, up)
    for i in (0, 1, 0, 1):
        a.copy_(other if i else x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((i, moe.gemm_w4(other if i else x, w, up)))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[i]) for i, v in got)


@pytest.mark.parametrize("M,N,K", [(1, 2064, 512), (1, 2032, 512), (7, 2064, 1152), (16, 2064, 4096), (16, 2048, 4096)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("pair", [False, True])
def test_gemm_w4_few_rows_by_more_or_fewer_weight_rows_than_cus_take(moe, M, N, K, group, zeros, pair):
    """Either side of 16 weight rows per CU (of a pair in sum), with x on chip and not."""
    test_gemm_w4(moe, M, N, K, group, zeros, pair)


@pytest.mark.parametrize("M,K", [(9, 4096), (16, 2048), (16, 7168)])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("pair", [False, True])
def test_gemm_w4_a_workgroup_per_cu_and_one_more(moe, M, K, group, zeros, pair):
    """As many blocks of 16 weight rows as there are CUs, of both matrices in sum, and more: x beside 16 and 32 weight
    rows gives the same bits."""
    N = 16 * torch.cuda.get_device_properties(0).multi_processor_count // (2 if pair else 1)
    big = [_w(N + 16, K, group, zeros, i) for i in range(2 if pair else 1)]
    few = [tuple(None if t is None else t[:N].contiguous() for t in w) for w in big]
    x = _bf16(M, K, seed=M)
    y = moe.gemm_w4(x, *(moe.w4_tile(*w) for w in big))
    check(x, y, big[0], big[1] if pair else None, group)
    assert torch.equal(moe.gemm_w4(x, *(moe.w4_tile(*w) for w in few)), y[:, :N])


@pytest.mark.parametrize("M,K", [(16, 1920), (16, 2048), (4, 7936), (4, 8192), (1, 32640), (1, 32768)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("pair", [False, True])
def test_gemm_w4_as_long_as_lds_holds(moe, M, K, zeros, pair):
    """Few rows that just fit on chip beside the weights, and that just do not."""
    test_gemm_w4(moe, M, 48, K, 128, zeros, pair)


def test_gemm_w4_of_the_longest_rows(moe):
    """16 rows of 2^26 columns, 2^31 bytes: one value of each picks out a column of exact weights."""
    N, K, M = 16, 2 ** 26, 16
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    s = (torch.rand(N, K // 128, device="cuda") * 0.02 + 0.001).to(torch.bfloat16)
    at = torch.randint(0, K, (M,), generator=torch.Generator().manual_seed(1)).cuda()
    at[0], at[1] = 0, K - 1
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(M), at] = 1
    y = moe.gemm_w4(x, moe.w4_tile(codes, s))
    c = codes[:, at // 2].int()
    want = (torch.where(at % 2 == 1, c >> 4, c & 15) - 8).double() * s[:, at // 128].double()
    assert torch.equal(y, want.t().to(torch.bfloat16))


# ------------------------------------------------------------------------------------------------
# a block's surroundings, run together
# ------------------------------------------------------------------------------------------------

def _block_step(moe, s):
    """From an attention block's output to the next block's input: norms and gate, routing by scores, int8
    experts, a 4-bit shared expert, combine, norms; then the way back through routing and norms."""
    T, E, k, d, f = s["T"], s["E"], s["k"], s["d"], s["f"]
    h, y, q, qs = moe.block_norm(s["attn"], s["stream"], s["w"][0], s["w"][1], s["gate"], 1.0, 0.5, 1e-6, moe.DTYPE_INT8)
    ids, w = moe.route_scored(s["logits"], k, s["bias"], groups=4, top_groups=2, group_top=2, scale=2.5)
    counts, offsets, _, slot, xp, xps = moe.permute(ids, E, q, qs)
    yp = moe.grouped_ffn(xp, xps, counts, offsets, s["experts"], T, k)
    shared = moe.gemm_w4(moe.gemm_w4(y, s["sh_gate"], s["sh_up"]), s["sh_down"])
    out = moe.combine(yp, slot, w, shared).view(torch.bfloat16)
    h2, y2, _, _ = moe.block_norm(out, h, s["w"][2], s["w"][3], None, 1.0, 0.5)
    dout, dh, dp2, dq2, _ = moe.block_norm_grad(s["dy"], out, h2, s["w"][2], s["dh"], s["w"][3], None, 1.0, 0.5)
    dyp, dw = moe.combine_grad(dout, yp.view(torch.bfloat16), slot, w)
    dl = moe.route_scored_grad(s["logits"], ids, w, dw, scale=2.5)
    da, ds, dp, dq, dg = moe.block_norm_grad(dout, s["attn"], h, s["w"][0], dh, s["w"][1], s["gate"], 1.0, 0.5)
    return [h, y, q, qs, ids, w, yp, shared, out, h2, y2, dout, dh, dp2, dq2, dyp, dw, dl, da, ds, dp, dq, dg]


def _state(moe, T, seed):
    E, k, d, f = 16, 4, 256, 384
    g = torch.Generator().manual_seed(seed)
    s = dict(T=T, E=E, k=k, d=d, f=f, attn=_bf16(T, d, seed=seed), stream=_bf16(T, d, seed=seed + 1),
             w=[_bf16(d, seed=seed + 2 + i) for i in range(4)], gate=_bf16(T, d, seed=seed + 6),
             dy=_bf16(T, d, seed=seed + 7), dh=_bf16(T, d, seed=seed + 8),
             logits=torch.randn(T, E, generator=g).cuda(), bias=(torch.randn(E, generator=g) * 0.1).cuda())
    ew = {}
    for n, shape in (("gate", (E, f, d)), ("up", (E, f, d)), ("down", (E, d, f))):
        ew[n] = moe.int8_tile(torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).cuda())
        ew["s_" + n] = (torch.rand(*shape[:2], generator=g) * 1e-3).cuda()
    s["experts"] = moe.ExpertWeights(**ew)
    for n, (a, b) in dict(sh_gate=(f, d), sh_up=(f, d), sh_down=(d, f)).items():
        s["raw_" + n] = _w(a, b, 32, True, a + b)
        s[n] = moe.w4_tile(*s["raw_" + n])
    return s


@pytest.mark.parametrize("T", [1, 37, 300])
def test_block_run_together(moe, T):
    """Every step against float64 from the step's own inputs."""
    from oracle import rows as R
    s = _state(moe, T, 5)
    (h, y, q, qs, ids, w, yp, shared, out, h2, y2, dout, dh, dp2, dq2, dyp, dw, dl, da, ds, dp, dq, dg) = \
        _block_step(moe, s)
    W = [f64(t) for t in s["w"]]
    ref, mag, _ = B.block_norm(f64(s["attn"]), f64(s["stream"]), W[1], f64(s["gate"]), W[0], 1.0, 0.5, 1e-6)
    assert (np.abs(f64(h) - ref) <= np.abs(ref) * BF + mag * 2.0 ** -19).all()
    want, ww = B.route_scored(f64(s["logits"]), 4, f64(s["bias"]), groups=4, top_groups=2, group_top=2, scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), want) and (np.abs(f64(w) - ww) <= ww * 2.0 ** -19).all()
    sh = moe.gemm_w4(y, s["sh_gate"], s["sh_up"])
    check(y, sh, s["raw_sh_gate"], s["raw_sh_up"], 32)
    check(sh, shared, s["raw_sh_down"], None, 32)
    ref, mag, _ = B.block_norm(f64(out), f64(h), W[3], None, W[2], 1.0, 0.5, 1e-6)
    assert (np.abs(f64(h2) - ref) <= np.abs(ref) * BF + mag * 2.0 ** -19).all()
    g = B.block_norm_grad(f64(s["dy"]), f64(s["dh"]), f64(out), f64(h2), W[3], None, W[2], 1.0, 0.5, 1e-6)
    for name, got in (("dx", dout), ("dres", dh), ("dpre", dp2), ("dpost", dq2)):
        assert (np.abs(f64(got) - g[name]) <= np.abs(g[name]) * BF + g["e_" + name] * 2.0 ** -16).all()
    ref, mag = B.route_scored_grad(f64(s["logits"]), want, f64(w), f64(dw), scale=2.5)
    assert (np.abs(f64(dl) - ref) <= mag * 2.0 ** -18).all()
    g = B.block_norm_grad(f64(dout), f64(dh), f64(s["attn"]), f64(h), W[1], f64(s["gate"]), W[0], 1.0, 0.5, 1e-6)
    for name, got in (("dx", da), ("dres", ds), ("dpre", dp), ("dpost", dq), ("dgate", dg)):
        assert (np.abs(f64(got) - g[name]) <= np.abs(g[name]) * BF + g["e_" + name] * 2.0 ** -16).all()


@pytest.mark.parametrize("T", [1, 37, 300])
def test_block_captured_and_replayed(moe, T):
    """The whole run in a HIP graph: every replay gives the eager call's bits, with eager work and new inputs
    between the replays."""
    s, other = _state(moe, T, 5), _state(moe, T, 50)
    _block_step(moe, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _block_step(moe, s)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _block_step(moe, s)
    for i in range(4):
        want = _block_step(moe, s)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        _block_step(moe, other)
        for n in ("attn", "stream", "gate", "dy", "dh", "logits", "bias"):
            s[n].copy_(other[n] * (0.5 + i))


def test_two_streams_at_once(moe):
    """Calls on two streams at a time, with their own tensors, give what they give alone."""
    a, b = _state(moe, 64, 5), _state(moe, 300, 50)
    want = _block_step(moe, a), _block_step(moe, b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = _block_step(moe, s)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for p, q in zip(g, w):
            assert torch.equal(p, q)
