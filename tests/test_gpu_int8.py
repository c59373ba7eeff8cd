"""GPU: int8 rows and products, alone, as experts and in the whole layer.

Sums are exact integers, so a product's value differs from the exact one by the fp32 scaling (the sum's
conversion and two products: 2^-22) and bf16's rounding (2^-8), and every tile family gives the same
bits.  For the experts, codes of h that lie within fp32 error of a half step may go either way; the
oracle says what those can do to y."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_top_amd import inputs as I
from mixture_experts_layer_top_amd import moe as _moe
from oracle import moe_oracle as O
from oracle import rows as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _moe.lib()
    return _moe


def f64(t):
    return t.double().cpu().numpy()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf16(*shape, seed=0, std=1.0):
    return (torch.randn(*shape, generator=_gen(seed)) * std).to(torch.bfloat16).cuda()


def _codes(*shape, seed=0):
    return torch.randint(-128, 128, shape, generator=_gen(seed), dtype=torch.int16).to(torch.int8).cuda()


def _scales(*shape, seed=0, mid=1e-3):
    return ((torch.rand(*shape, generator=_gen(seed)) + 0.5) * mid).cuda()


@pytest.mark.parametrize("T,d", [(1, 16), (1, 7168), (3, 128), (77, 4096), (5, 4112), (9, 8192), (2, 32768)])
def test_quant_act_i8(moe, T, d):
    x = _bf16(T, d, seed=T + d)
    if T > 2:
        x[1] = 0
        x[2, 0] = -300.0
    q, s = moe.quant_act_i8(x)
    want_q, want_s = R.quant_i8(f64(x))
    assert np.array_equal(f64(s), want_s)
    # float64 quotient by the reciprocal: off by 2^-52 of it, so only exact half steps could differ,
    # and those are exact in both
    assert np.array_equal(f64(q), want_q)


def test_quant_act_i8_non_finite_rows(moe):
    x = _bf16(4, 256, seed=1)
    x[1, 3], x[2, 255] = float("inf"), float("nan")
    q, s = moe.quant_act_i8(x)
    ref, sr = moe.quant_act_i8(_bf16(4, 256, seed=1))
    assert s[1:3].isnan().all() and (q[1:3] == 0).all()
    assert torch.equal(q[[0, 3]], ref[[0, 3]]) and torch.equal(s[[0, 3]], sr[[0, 3]])
    assert moe.quant_act_i8(x[:0])[0].shape == (0, 256)


GEMMS = [(1, 16, 128), (1, 2048, 7168), (16, 48, 256), (17, 256, 384), (33, 272, 128), (64, 512, 4224),
         (65, 256, 128), (100, 528, 640), (130, 1040, 256), (257, 256, 1152), (300, 4096, 512), (1030, 2064, 384),
         (2100, 7168, 256)]


@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm_i8(moe, M, N, K):
    xq, w = _codes(M, K, seed=M), _codes(N, K, seed=N + 1)
    xs, ws = _scales(M, seed=K), _scales(N, seed=K + 1)
    y = moe.gemm_i8(xq, xs, moe.int8_tile(w), ws)
    ref = R.gemm_i8(f64(xq), f64(xs), f64(w), f64(ws))
    assert (np.abs(f64(y) - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -21)).all()


def test_gemm_i8_extremes(moe):
    """The longest K at the largest codes: the sum reaches 2^29 and stays exact; M = 0; rows behind the
    last one stay as they were."""
    K, N = 32768, 32
    xq = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(N, device="cuda")
    t = moe.int8_tile(w)
    for M in (3, 80):
        x = xq[:1].expand(M, K).contiguous()
        y = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
        xs = torch.ones(M, device="cuda")
        assert moe.lib().moe_gemm_i8(x.data_ptr(), xs.data_ptr(), M, t.data_ptr(), one.data_ptr(), N, K,
                                     y.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert (y[:M] == 2.0 ** 29).all() and (y[M:] == 7).all()
    assert moe.gemm_i8(xq[:0], one[:0], t, one).shape == (0, N)
    with pytest.raises(moe.MoEError, match="int8_tile"):
        moe.gemm_i8(xq, one[:3], w, one)


def test_gemm_i8_passes_non_finite_rows_on(moe):
    x = _bf16(70, 256, seed=1)
    x[5, 7] = float("nan")
    w, ws = _codes(256, 256, seed=2), _scales(256, seed=3)
    q, s = moe.quant_act_i8(x)
    y = moe.gemm_i8(q, s, moe.int8_tile(w), ws)
    assert y[5].isnan().all() and y[:5].isfinite().all() and y[6:].isfinite().all()


# ------------------------------------------------------------------------------------------------
# experts
# ------------------------------------------------------------------------------------------------

class Experts:
    def __init__(self, moe, E, d, f, seed, shared_f=0):
        def w(n, k, i, lead=()):
            m = torch.randn(*lead, n, k, generator=_gen(seed + i)).mul_(32).round_().clamp_(-127, 127)
            return m.to(torch.int8).cuda(), _scales(*lead, n, seed=seed + 50 + i, mid=0.02 / 32)

        self.c, self.s = {}, {}
        for i, (name, n, k) in enumerate((("gate", f, d), ("up", f, d), ("down", d, f))):
            self.c[name], self.s["s_" + name] = w(n, k, i, (E,))
        if shared_f:
            for i, (name, n, k) in enumerate((("gate", shared_f, d), ("up", shared_f, d), ("down", d, shared_f))):
                self.c["sh_" + name], self.s["s_sh_" + name] = w(n, k, 10 + i)
        self.ew = moe.ExpertWeights(**{n: moe.int8_tile(t) for n, t in self.c.items()}, **self.s)
        self.shared = bool(shared_f)

    def get(self, e):
        r = {n: f64(self.c[n][e]) for n in ("gate", "up", "down")}
        r.update({"s_" + n: f64(self.s["s_" + n][e]) for n in ("gate", "up", "down")})
        return r

    def get_shared(self):
        r = {n: f64(self.c["sh_" + n]) for n in ("gate", "up", "down")}
        r.update({"s_" + n: f64(self.s["s_sh_" + n]) for n in ("gate", "up", "down")})
        return r


def _rows(counts, d, seed):
    counts = torch.tensor(counts, dtype=torch.int32)
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = counts.cumsum(0)
    n = int(off[-1])
    q = torch.randn(n, d, generator=_gen(seed)).mul_(32).round_().clamp_(-127, 127).to(torch.int8)
    return q.cuda(), _scales(n, seed=seed + 1, mid=1.0 / 32), counts.cuda(), off.cuda()


FFN = [  # counts per expert, d, f: one row; empty experts; short and tall tiles; odd K-step counts; tails
    ([0, 1, 0], 128, 128), ([8] * 4, 256, 512), ([1, 0, 33, 5, 0, 17], 384, 640), ([70, 2, 0, 200], 512, 256),
    ([300, 1, 64], 640, 384), ([16, 129, 257, 40], 4224, 256), ([3, 0, 2], 256, 4224), ([700], 256, 1152),
]


@pytest.mark.parametrize("counts,d,f", FFN, ids=lambda v: str(v).replace(" ", ""))
def test_grouped_ffn(moe, counts, d, f):
    xq, xs, cnt, off = _rows(counts, d, seed=d + f)
    W = Experts(moe, len(counts), d, f, seed=3)
    n = xq.shape[0]
    out = {}
    for name, cfg in (("auto", moe.CONFIG_AUTO), ("stream", moe.CONFIG_STREAM), ("mfma", moe.CONFIG_MFMA)):
        out[name] = moe.grouped_ffn(xq, xs, cnt, off, W.ew, n, 1, cfg).view(torch.bfloat16)
    assert torch.equal(out["stream"], out["mfma"]) and torch.equal(out["auto"], out["mfma"])
    y = f64(out["auto"])
    for e, c in enumerate(counts):
        if c:
            a = int(off[e])
            ref, slack = R.expert_i8(f64(xq[a:a + c]), f64(xs[a:a + c]), W.get(e))
            assert (np.abs(y[a:a + c] - ref) <= slack * (1 + 2.0 ** -7) + np.abs(ref) * (2.0 ** -8 + 2.0 ** -20)).all(), e


def test_grouped_ffn_many_tiles(moe):
    """Several rounds of tiles, full heights with tails, and the two-class order (long K)."""
    counts = [520, 300, 0, 40, 1, 260, 128, 5]
    xq, xs, cnt, off = _rows(counts, 4096, seed=1)
    W = Experts(moe, len(counts), 4096, 8192, seed=5)
    n = xq.shape[0]
    a = moe.grouped_ffn(xq, xs, cnt, off, W.ew, n, 1, moe.CONFIG_MFMA)
    assert torch.equal(a, moe.grouped_ffn(xq, xs, cnt, off, W.ew, n, 1, moe.CONFIG_STREAM))
    assert torch.equal(a, moe.grouped_ffn(xq, xs, cnt, off, W.ew, n, 1))
    y = f64(a.view(torch.bfloat16))
    for e in (1, 4, 7):
        s = slice(int(off[e]), int(off[e + 1]))
        ref, slack = R.expert_i8(f64(xq[s]), f64(xs[s]), W.get(e))
        assert (np.abs(y[s] - ref) <= slack * (1 + 2.0 ** -7) + np.abs(ref) * (2.0 ** -8 + 2.0 ** -20)).all(), e


def test_grouped_ffn_leaves_other_rows(moe):
    """Fewer rows than T * k: rows past offsets[E] are not written, and a NaN row stays alone."""
    xq, xs, cnt, off = _rows([5, 0, 90], 256, seed=2)
    W = Experts(moe, 3, 256, 256, seed=9)
    base = moe.grouped_ffn(xq, xs, cnt, off, W.ew, 95, 1)
    bad = xs.clone()
    bad[7] = float("nan")
    got = moe.grouped_ffn(xq, bad, cnt, off, W.ew, 95, 1)
    keep = torch.arange(95, device="cuda") != 7
    assert torch.equal(got[keep], base[keep]) and got[7].view(torch.bfloat16).isnan().all()
    import ctypes
    p = moe.problem(100, 256, 256, 3, 1, wdtype=moe.DTYPE_INT8)
    ws = torch.empty(moe.lib().moe_grouped_ffn_workspace_bytes(ctypes.byref(p)), dtype=torch.uint8, device="cuda")
    y = torch.full((100, 256), 7, dtype=torch.int16, device="cuda")
    w = W.ew.struct()
    assert moe.lib().moe_grouped_ffn(ctypes.byref(p), xq.data_ptr(), xs.data_ptr(), cnt.data_ptr(), off.data_ptr(),
                                     ctypes.byref(w), y.data_ptr(), ws.data_ptr(), ws.numel(),
                                     torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y[:95], base) and (y[95:] == 7).all()


LAYERS = [(1, 256, 256, 8, 2, 0), (3, 384, 128, 16, 8, 256), (33, 256, 512, 4, 2, 0), (150, 512, 256, 6, 3, 384),
          (600, 256, 256, 2, 1, 0)]


@pytest.mark.parametrize("T,d,f,E,k,sf", LAYERS)
def test_layer(moe, T, d, f, E, k, sf):
    """moe_layer on int8 experts: the steps one by one give the same bits, and the oracle's layer on the
    quantised rows the same values."""
    x, logits = _bf16(T, d, seed=T), torch.randn(T, E, generator=_gen(T + 1)).cuda()
    W = Experts(moe, E, d, f, seed=11, shared_f=sf)
    out, keep = moe.layer(logits, x.view(torch.int16), W.ew, k, keep_routing=True)
    xq, xs = moe.quant_act_i8(x)
    ids, w = moe.route(logits, k)
    cnt, off, perm, slot, xp, xps = moe.permute(ids, E, xq, xs)
    assert torch.equal(xp, xq[perm.long() // k]) and torch.equal(xps, xs[perm.long() // k])
    y = moe.grouped_ffn(xp, xps, cnt, off, W.ew, T, k)
    ysh = None
    if sf:  # the shared expert as a one-expert grouped FFN of all tokens
        one = moe.ExpertWeights(**{n: getattr(W.ew, "sh_" + n).unsqueeze(0) for n in ("gate", "up", "down")},
                                **{"s_" + n: getattr(W.ew, "s_sh_" + n).unsqueeze(0) for n in ("gate", "up", "down")})
        for n in ("gate", "up", "down"):
            getattr(one, n)._moe_tiled = True
        c = torch.tensor([T], dtype=torch.int32, device="cuda")
        ysh = moe.grouped_ffn(xq, xs, c, torch.tensor([0, T], dtype=torch.int32, device="cuda"), one, T, 1)
    assert torch.equal(out, moe.combine(y, slot, w, ysh))
    ref, slack = np.zeros((T * k, d)), np.zeros((T * k, d))
    o = off.tolist()
    for e in range(E):
        if o[e] < o[e + 1]:
            s = slice(o[e], o[e + 1])
            ref[s], slack[s] = R.expert_i8(f64(xp[s]), f64(xps[s]), W.get(e))
    tol = slack + np.abs(ref) * 2.0 ** -7  # y is held in bf16 between the products and the combine
    wk, sl = f64(w), slot.cpu().numpy()
    want = (wk[..., None] * ref[sl].reshape(T, k, d)).sum(1)
    room = (wk[..., None] * tol[sl].reshape(T, k, d)).sum(1)
    if sf:
        r, sk = R.expert_i8(f64(xq), f64(xs), W.get_shared())
        want, room = want + r, room + sk + np.abs(r) * 2.0 ** -7
    assert (np.abs(f64(out.view(torch.bfloat16)) - want) <= room * 1.01 + np.abs(want) * 2.0 ** -8).all()
    noal = moe.layer_noalloc(logits, x.view(torch.int16), W.ew, k) if T * k < 400 else out
    assert torch.equal(noal, out)


def test_norm_sort_experts_together_in_a_graph(moe):
    """The serving path: norm (bf16 and int8 rows) -> route -> permute -> int8 experts -> combine -> the
    next norm; eager, on another stream, and captured and replayed on new inputs."""
    T, d, f, E, k = 40, 512, 256, 8, 2
    W = Experts(moe, E, d, f, seed=21)
    nw, router = _bf16(d, seed=1), torch.randn(d, E, generator=_gen(2)).cuda()
    x, res = _bf16(T, d, seed=3), _bf16(T, d, seed=4)

    def step(x, res):
        h, y, q, qs = moe.rmsnorm(x, nw, res, 1e-6, moe.DTYPE_INT8)
        ids, w = moe.route(y.float() @ router, k)
        cnt, off, _, slot, xp, xps = moe.permute(ids, E, q, qs)
        o = moe.combine(moe.grouped_ffn(xp, xps, cnt, off, W.ew, T, k), slot, w).view(torch.bfloat16)
        return moe.rmsnorm(o, nw, h)[:2]

    h0, y0 = (t.clone() for t in step(x, res))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h1, y1 = step(x, res)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(h0, h1) and torch.equal(y0, y1)
    sx, sr = x.clone(), res.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gh, gy = step(sx, sr)
    for seed in (0, 30, 40):
        if seed:
            sx.copy_(_bf16(T, d, seed=seed))
            sr.copy_(_bf16(T, d, seed=seed + 1))
        g.replay()
        torch.cuda.synchronize()
        h, y = step(sx, sr)  # eager work between the replays
        torch.cuda.synchronize()
        assert torch.equal(gh, h) and torch.equal(gy, y)
    # against the oracle: routing from the library's bf16 y, everything behind it in float64
    hh, yy, q, qs = moe.rmsnorm(sx, nw, sr, 1e-6, moe.DTYPE_INT8)
    ids, w = moe.route(yy.float() @ router, k)
    qn, qsn, idn, wn = f64(q), f64(qs), ids.cpu().numpy(), f64(w)
    o = np.zeros((T, d))
    room = np.zeros((T, d))
    for e in range(E):
        for j in range(k):
            r = np.nonzero(idn[:, j] == e)[0]
            if len(r):
                v, sl = R.expert_i8(qn[r], qsn[r], W.get(e))
                o[r] += wn[r, j, None] * v
                room[r] += wn[r, j, None] * (sl + np.abs(v) * 2.0 ** -7)
    want = f64(hh) + o
    assert (np.abs(f64(gh) - want) <= 1.01 * room + (np.abs(o) + np.abs(want)) * 2.0 ** -8).all()


# ------------------------------------------------------------------------------------------------
# the tile choices
# ------------------------------------------------------------------------------------------------

# Dense products by the tile they take on 256 CUs (16 token rows x 16 weight rows): 4x4, 2x4, 1x2, 2x2 and
# 1x1, with ragged last blocks and, for two m-tiles or more, a grid that is no multiple of 8; then MFMA
# pieces only (32, 64, 128 and 256 rows), whole tiles with 1, 2, 4 and 8 pieces per tile behind them, and
# with none.
TILES = [(64, 12352, 128), (100, 6160, 256), (33, 6208, 128), (160, 2064, 128), (20, 3120, 384), (16, 6160, 256),
         (33, 3120, 128), (30, 6160, 128), (7, 2064, 640), (130, 12304, 128), (520, 7168, 128), (900, 7184, 128),
         (700, 11280, 128), (2100, 11520, 128), (2100, 10240, 128), (2100, 8208, 256), (2100, 8192, 128),
         (2048, 8192, 128)]


@pytest.mark.parametrize("M,N,K", TILES)
def test_gemm_i8_tiles(moe, M, N, K):
    xq, w = _codes(M, K, seed=M), _codes(N, K, seed=N + 1)
    xs, ws = _scales(M, seed=K), _scales(N, seed=K + 1)
    t = moe.int8_tile(w)
    y = moe.gemm_i8(xq, xs, t, ws)
    # (a float64 product of these codes is exact: its sums stay below 2^53)
    ref = (xq.double() @ w.double().T) * xs.double()[:, None] * ws.double()
    assert ((y.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -21)).all()
    # a row has the same bits alone, from the smallest tile
    one = moe.gemm_i8(xq[:1].contiguous(), xs[:1].contiguous(), t, ws)
    assert torch.equal(one[0], y[0])


def test_gemm_i8_up_to_the_offset_limit(moe):
    """M * K and N * K just below 2^32: rows far apart are the rows of a small product."""
    K = 32640
    n = 2 ** 32 // K // 16 * 16
    assert 2 ** 32 - 16 * K <= n * K < 2 ** 32
    few, fs = _codes(16, K, seed=1), _scales(16, seed=2)
    other, os_ = _codes(48, K, seed=3), _scales(48, seed=4)
    x, xs = few.repeat(n // 16, 1), fs.repeat(n // 16)
    want = moe.gemm_i8(few, fs, moe.int8_tile(other), os_)  # [16, 48]
    y = moe.gemm_i8(x, xs, moe.int8_tile(other), os_)
    assert torch.equal(y.view(-1, 16, 48), want.expand(n // 16, 16, 48))
    t = moe.int8_tile(x)
    for M in (1, 30, 48):
        got = moe.gemm_i8(other[:M].contiguous(), os_[:M].contiguous(), t, xs)
        small = moe.gemm_i8(other[:M].contiguous(), os_[:M].contiguous(), moe.int8_tile(few), fs)
        assert torch.equal(got.view(M, -1, 16), small[:, None].expand(M, n // 16, 16)), M


def test_quant_act_i8_past_32_bit_offsets(moe):
    d = 7168
    T = 2 ** 32 // d + 100
    few = _bf16(4, d, seed=5)
    q, s = moe.quant_act_i8(few.repeat(T // 4, 1))
    wq, ws = moe.quant_act_i8(few)
    assert torch.equal(q.view(-1, 4, d), wq.expand(T // 4, 4, d)) and torch.equal(s.view(-1, 4), ws.expand(T // 4, 4))


# ------------------------------------------------------------------------------------------------
# lists in pieces, and small batches
# ------------------------------------------------------------------------------------------------

# MFMA lists whose last round is cut by token rows: less than a round of tiles (2 and 4 pieces each),
# and a round and some (a tall tile's pieces, a short tail's, empty ones).
PIECES = [([200, 256, 30, 64], 256, 4096), ([256, 129, 1], 128, 2048), ([700, 1, 513], 256, 7168),
          ([300] * 9, 128, 2048), ([256, 40] * 9, 128, 2048)]


@pytest.mark.parametrize("counts,d,f", PIECES, ids=lambda v: str(v).replace(" ", ""))
def test_grouped_ffn_in_pieces(moe, counts, d, f):
    xq, xs, cnt, off = _rows(counts, d, seed=7)
    W = Experts(moe, len(counts), d, f, seed=8)
    n = xq.shape[0]
    y = moe.grouped_ffn(xq, xs, cnt, off, W.ew, n, 1, moe.CONFIG_MFMA)
    assert torch.equal(y, moe.grouped_ffn(xq, xs, cnt, off, W.ew, n, 1, moe.CONFIG_STREAM))
    assert torch.equal(y, moe.grouped_ffn(xq, xs, cnt, off, W.ew, n, 1))
    e = len(counts) - 1
    s = slice(int(off[e]), n)
    ref, slack = R.expert_i8(f64(xq[s]), f64(xs[s]), W.get(e))
    assert (np.abs(f64(y.view(torch.bfloat16))[s] - ref) <=
            slack * (1 + 2.0 ** -7) + np.abs(ref) * (2.0 ** -8 + 2.0 ** -20)).all()


# Few tokens: counts, T, k, d, f.  All rows with one expert (a token's ids may repeat), passes of
# 16 and a tail, a long K in either product, many experts of one row, experts that all hold none.
SMALL = [([0, 32], 16, 2, 256, 256), ([17, 0, 15], 16, 2, 128, 384), ([0] * 7 + [128], 16, 8, 128, 128),
         ([0, 3, 1, 0, 4], 4, 2, 4224, 256), ([1, 1, 0, 2], 2, 2, 256, 4096), ([1] * 8 + [0] * 56, 1, 8, 256, 128),
         ([1, 0] * 64, 8, 8, 128, 128), ([0, 0], 16, 1, 128, 128), ([3, 2] + [0] * 6, 16, 8, 128, 256),
         # one token and a few of a wide expert; up to 32 tokens over many experts, and all rows with one
         ([1, 1], 1, 2, 128, 14336), ([0, 3, 1], 4, 1, 256, 14336), ([4] * 64, 32, 8, 128, 256),
         ([256] + [0] * 63, 32, 8, 128, 128), ([0, 17] * 4 + [0] * 12, 24, 3, 256, 2048)]


@pytest.mark.parametrize("counts,T,k,d,f", SMALL, ids=lambda v: str(v).replace(" ", "")[:24])
def test_grouped_ffn_small_batches(moe, counts, T, k, d, f):
    xq, xs, cnt, off = _rows(counts, d, seed=12)
    W = Experts(moe, len(counts), d, f, seed=13)
    n = xq.shape[0]
    q = torch.zeros(T * k, d, dtype=torch.int8, device="cuda")
    s = torch.ones(T * k, device="cuda")
    q[:n], s[:n] = xq, xs
    y = moe.grouped_ffn(q, s, cnt, off, W.ew, T, k)[:n].view(torch.bfloat16)
    for cfg in (moe.CONFIG_STREAM, moe.CONFIG_MFMA):
        assert torch.equal(y, moe.grouped_ffn(q, s, cnt, off, W.ew, T, k, cfg)[:n].view(torch.bfloat16))
    for e, c in enumerate(counts):
        if c and (e < 3 or c > 1):
            a = slice(int(off[e]), int(off[e + 1]))
            ref, slack = R.expert_i8(f64(xq[a]), f64(xs[a]), W.get(e))
            assert (np.abs(f64(y[a]) - ref) <= slack * (1 + 2.0 ** -7) + np.abs(ref) * (2.0 ** -8 + 2.0 ** -20)).all(), e


def _direct(moe, xq, xs, cnt, off, W, T, k, d, f, y, ws):
    import ctypes
    p = moe.problem(T, d, f, cnt.numel(), k, wdtype=moe.DTYPE_INT8)
    w = W.ew.struct()
    return moe.lib().moe_grouped_ffn(ctypes.byref(p), xq.data_ptr(), xs.data_ptr(), cnt.data_ptr(), off.data_ptr(),
                                     ctypes.byref(w), y.data_ptr(), ws.data_ptr(), ws.numel(),
                                     torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("T", [4, 40])
def test_two_calls_at_once_with_their_own_workspaces(moe, T):
    """Two streams, two workspaces that hold NaN bytes: neither call reads what it has not written, rows
    behind the last expert's stay as they were, and a NaN row stays alone."""
    import ctypes
    d, f, k, E = 384, 512, 2, 6
    counts = [T, 0, T // 2, 1, 0, 0]
    W = Experts(moe, E, d, f, seed=17)
    xq, xs, cnt, off = _rows(counts, d, seed=18)
    n = xq.shape[0]
    want = moe.grouped_ffn(xq, xs, cnt, off, W.ew, n, 1, moe.CONFIG_STREAM)
    bad = xs.clone()
    bad[1] = float("nan")
    q = torch.zeros(T * k, d, dtype=torch.int8, device="cuda")
    q[:n] = xq
    need = moe.lib().moe_grouped_ffn_workspace_bytes(ctypes.byref(moe.problem(T, d, f, E, k, wdtype=moe.DTYPE_INT8)))
    ys, streams, keep = [], [torch.cuda.Stream(), torch.cuda.Stream()], []
    scales = []
    for src in (xs, bad):
        s = torch.full((T * k,), float("nan"), device="cuda")
        s[:n] = src
        scales.append(s)
    torch.cuda.synchronize()
    for rep in range(3):
        for st, s in zip(streams, scales):
            with torch.cuda.stream(st):
                ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
                y = torch.full((T * k, d), 7, dtype=torch.int16, device="cuda")
                assert _direct(moe, q, s, cnt, off, W, T, k, d, f, y, ws) == 0
                ys.append(y)
                keep.append(ws)
    torch.cuda.synchronize()
    ok = torch.arange(n, device="cuda") != 1
    for i, y in enumerate(ys):
        assert (y[n:] == 7).all()
        assert torch.equal(y[:n][ok], want[ok])
        if i % 2:
            assert y[1].view(torch.bfloat16).isnan().all()
        else:
            assert torch.equal(y[1], want[1])


def test_layer_of_one_token_in_a_graph(moe):
    """The small path captured, with eager calls on the same weights between the replays."""
    d, f, E, k = 512, 256, 16, 4
    W = Experts(moe, E, d, f, seed=23)
    x, lg = _bf16(1, d, seed=1), torch.randn(1, E, generator=_gen(2)).cuda()
    moe.layer(lg, x.view(torch.int16), W.ew, k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = moe.layer(lg, x.view(torch.int16), W.ew, k)
    for seed in (1, 5, 6, 7):
        x.copy_(_bf16(1, d, seed=seed))
        lg.copy_(torch.randn(1, E, generator=_gen(seed + 100)).cuda())
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe.layer(lg, x.view(torch.int16), W.ew, k))


@pytest.mark.parametrize("T,d,f,E,k,sf", [(2, 256, 4096, 16, 2, 0), (9, 384, 256, 64, 8, 0), (16, 256, 384, 9, 8, 0),
                                          (16, 256, 4224, 4, 2, 0), (17, 256, 256, 9, 8, 0), (16, 256, 256, 4, 2, 128),
                                          (32, 256, 384, 64, 8, 0), (24, 128, 2048, 12, 2, 0), (33, 256, 384, 64, 8, 0)])
def test_layer_around_the_small_path(moe, T, d, f, E, k, sf):
    """Every way through moe_layer at few tokens gives the same bits; a traced call records the phases, and
    neither writes the bf16 selection's outputs."""
    x, logits = _bf16(T, d, seed=T + 2), torch.randn(T, E, generator=_gen(T + 3)).cuda()
    W = Experts(moe, E, d, f, seed=31, shared_f=sf)
    xb = x.view(torch.int16)
    out = moe.layer(logits, xb, W.ew, k)
    for cfg in (moe.CONFIG_STREAM, moe.CONFIG_MFMA):
        assert torch.equal(out, moe.layer(logits, xb, W.ew, k, cfg))
    keep = dict(eeff=torch.full((1,), 5.0, device="cuda"), policy=torch.full((1,), 77, dtype=torch.int32, device="cuda"))
    L = moe.Layer(W.ew, T, E, k)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(moe.TRACE_EVENTS)]
    for e in ev:
        e.record()  # (creates the handle)
    got = L.traced(logits, xb, [e.cuda_event for e in ev], keep)
    torch.cuda.synchronize()
    assert torch.equal(got, out) and float(keep["eeff"]) == 5.0 and int(keep["policy"]) == 77
    assert all(a.elapsed_time(b) >= 0 for a, b in zip(ev, ev[1:]))
    # and the oracle
    xq, xs = moe.quant_act_i8(x)
    ids, w = moe.route(logits, k)
    want, room = np.zeros((T, d)), np.zeros((T, d))
    idn, wn, qn, sn = ids.cpu().numpy(), f64(w), f64(xq), f64(xs)
    for e in range(E):
        t, j = np.nonzero(idn == e)
        if len(t):
            ref, slack = R.expert_i8(qn[t], sn[t], W.get(e))
            np.add.at(want, t, wn[t, j][:, None] * ref)
            np.add.at(room, t, wn[t, j][:, None] * (slack + np.abs(ref) * 2.0 ** -7))
    if sf:
        r, sk = R.expert_i8(qn, sn, W.get_shared())
        want, room = want + r, room + sk + np.abs(r) * 2.0 ** -7
    assert (np.abs(f64(out.view(torch.bfloat16)) - want) <= room * 1.01 + np.abs(want) * 2.0 ** -8).all()


def test_quant_act_i8_of_the_most_rows(moe):
    """2^25 - 1 rows: the first and the last are those of a small call."""
    T = 2 ** 25 - 1
    few = _bf16(7, 16, seed=9)
    x = torch.zeros(T, 16, dtype=torch.bfloat16, device="cuda")
    x[:7], x[-7:] = few, few
    q, s = moe.quant_act_i8(x)
    wq, ws = moe.quant_act_i8(few)
    for part in (slice(0, 7), slice(T - 7, T)):
        assert torch.equal(q[part], wq) and torch.equal(s[part], ws)
    assert (s[7:-7] == 1).all() and not q[7:-7].any()


@pytest.mark.parametrize("T,E,k", [(1, 16, 2), (16, 64, 8), (32, 64, 4)])
def test_layer_of_few_tokens_selects_nothing(moe, T, E, k):
    """Few tokens stream without a selection, in the whole layer too: the tile lists in the workspace (by far
    its largest piece here) are not written, where a forced family writes the heads of its lists."""
    W = Experts(moe, E, 128, 128, seed=41)
    x, logits = _bf16(T, 128, seed=1).view(torch.int16), torch.randn(T, E, generator=_gen(2)).cuda()

    def untouched(cfg):
        L = moe.Layer(W.ew, T, E, k, cfg)
        L.ws.fill_(0xA5)
        out = L(logits, x).clone()
        at = torch.nonzero(L.ws != 0xA5)[:, 0].cpu().numpy()
        return int(np.diff(np.concatenate([[-1], at, [L.ws.numel()]])).max()), out

    (auto, a), (forced, b) = untouched(moe.CONFIG_AUTO), untouched(moe.CONFIG_STREAM)
    assert auto > 1.5 * forced and torch.equal(a, b)


@pytest.mark.parametrize("cfg", ["auto", "stream"])
def test_grouped_ffn_of_h_past_32_bit_offsets(moe, cfg):
    """fp32 h of more than 2^32 bytes: an expert's rows are eight rows over and over."""
    d, f, rep = 128, 32768, 2064
    assert 16 * rep * f * 4 > 2 ** 32 and 16 * rep * f * 2 < 2 ** 32
    W = Experts(moe, 2, d, f, seed=43)
    xq, xs, cnt, off = _rows([8, 8], d, seed=44)
    few = moe.grouped_ffn(xq, xs, cnt, off, W.ew, 16, 1, moe.CONFIG_MFMA)
    big = xq.view(2, 1, 8, d).expand(2, rep, 8, d).reshape(-1, d)
    y = moe.grouped_ffn(big, xs.view(2, 1, 8).expand(2, rep, 8).reshape(-1), cnt * rep, off * rep, W.ew, 16 * rep, 1,
                        {"auto": moe.CONFIG_AUTO, "stream": moe.CONFIG_STREAM}[cfg])
    assert torch.equal(y.view(2, rep, 8, d), few.view(2, 1, 8, d).expand(2, rep, 8, d))


def test_layer_of_shared_h_past_32_bit_offsets(moe):
    """The same of the shared expert, in the whole layer."""
    d, f, sf, E, rep = 128, 128, 32768, 2, 4128
    assert 8 * rep * sf * 4 > 2 ** 32 and 8 * rep * sf * 2 < 2 ** 32
    W = Experts(moe, E, d, f, seed=45, shared_f=sf)
    x, logits = _bf16(8, d, seed=1).view(torch.int16), torch.randn(8, E, generator=_gen(2)).cuda()
    few = moe.layer(logits, x, W.ew, 1)
    out = moe.layer(logits.repeat(rep, 1), x.repeat(rep, 1), W.ew, 1)
    assert torch.equal(out.view(rep, 8, d), few.expand(rep, 8, d))


@pytest.mark.parametrize("T,k", [(16, 1), (15, 2), (2, 8)])
def test_small_batch_of_the_largest_lds(moe, T, k):
    """Sixteen rows of 4096 codes: the small path's down tiles take 65792 bytes of LDS, more than 64 KB."""
    d, f, E = 128, 4096, 8
    W = Experts(moe, E, d, f, seed=47)
    counts = [T * k, 0, 0, 0, 0, 0, 0, 0] if k == 1 else [16] + [0] * 6 + [T * k - 16]
    xq, xs, cnt, off = _rows(counts, d, seed=48)
    y = moe.grouped_ffn(xq, xs, cnt, off, W.ew, T, k)
    assert torch.equal(y, moe.grouped_ffn(xq, xs, cnt, off, W.ew, T, k, moe.CONFIG_STREAM))
    ref, slack = R.expert_i8(f64(xq[:16]), f64(xs[:16]), W.get(0))
    got = f64(y.view(torch.bfloat16))[:16]
    assert (np.abs(got - ref) <= slack * (1 + 2.0 ** -7) + np.abs(ref) * (2.0 ** -8 + 2.0 ** -20)).all()
