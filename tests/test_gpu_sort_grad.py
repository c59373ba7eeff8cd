"""GPU: gradients of route, combine and the row gather against float64, and the whole way back of the
sort.  u = 2^-24."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_top_amd import moe as _moe
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


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 512, 8), (5, 3, 2), (7, 8, 8), (64, 64, 4), (130, 65, 5), (777, 384, 8)])
def test_route_grad(moe, T, E, k):
    logits = torch.randn(T, E, generator=_gen(T + E)).cuda()
    ids, w = moe.route(logits, k)
    dw = torch.randn(T, k, generator=_gen(k)).cuda()
    dl = moe.route_grad(ids, w, dw, E)
    ref = R.route_grad(ids.cpu().numpy(), f64(w), f64(dw), E)
    # s: k FMAs; then a difference and a product, each rounded once
    room = (np.abs(f64(dw)).max(1) * (k + 3) * 2.0 ** -24)[:, None]
    assert (np.abs(f64(dl) - ref) <= room).all()
    chosen = np.zeros((T, E), bool)
    np.put_along_axis(chosen, ids.cpu().numpy(), True, 1)
    assert (f64(dl)[~chosen] == 0).all()


def test_route_grad_of_a_repeated_expert(moe):
    """Ids from elsewhere may name an expert twice: its slots' gradients add."""
    ids = torch.tensor([[2, 2, 0], [1, 0, 1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 0.25], [0.125, 0.5, 0.375]], device="cuda")
    dw = torch.tensor([[1.0, 2.0, -1.0], [0.5, 0.0, 4.0]], device="cuda")
    ref = R.route_grad(ids.cpu().numpy(), f64(w), f64(dw), 4)
    assert np.array_equal(f64(moe.route_grad(ids, w, dw, 4)), ref)  # exact in fp32


CASES = [(1, 128, 1), (1, 7168, 8), (3, 256, 2), (33, 640, 3), (130, 4096, 4), (257, 1152, 8), (9, 8192, 2),
         (5, 16384, 5), (3, 32768, 2)]


@pytest.mark.parametrize("T,d,k", CASES)
def test_combine_grad(moe, T, d, k):
    n = T * k
    dout, y = _bf16(T, d, seed=1), _bf16(n, d, seed=2)
    w = torch.rand(T, k, generator=_gen(3)).cuda()
    slot = torch.randperm(n, generator=_gen(4)).to(torch.int32).cuda()
    dy, dw = moe.combine_grad(dout, y, slot, w)
    rdy, rdw = R.combine_grad(f64(dout), f64(y), slot.cpu().numpy(), f64(w))
    assert (np.abs(f64(dy) - rdy) <= np.abs(rdy) * (2.0 ** -8 + 2.0 ** -22)).all()
    # a thread's chain of at most 64 products, six exchanges and 7 wavefronts
    size = (np.abs(f64(dout))[:, None] * np.abs(f64(y)[slot.cpu().numpy()].reshape(T, k, d))).sum(-1)
    assert (np.abs(f64(dw) - rdw) <= size * 80 * 2.0 ** -24).all()
    # one output alone
    st = torch.cuda.current_stream().cuda_stream
    dy2, dw2 = torch.zeros_like(dy), torch.zeros_like(dw)
    L = moe.lib()
    assert L.moe_combine_grad(dout.data_ptr(), None, slot.data_ptr(), w.data_ptr(), T, k, d, dy2.data_ptr(), None, st) == 0
    assert L.moe_combine_grad(dout.data_ptr(), y.data_ptr(), slot.data_ptr(), None, T, k, d, None, dw2.data_ptr(), st) == 0
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("T,d,k", CASES)
def test_permute_grad(moe, T, d, k):
    n = T * k
    dxp, slot = _bf16(n, d, seed=5), torch.randperm(n, generator=_gen(6)).to(torch.int32).cuda()
    for add in (None, _bf16(T, d, seed=7)):
        dx = moe.permute_grad(dxp, slot, k, add)
        a = None if add is None else f64(add)
        ref = R.permute_grad(f64(dxp), slot.cpu().numpy(), k, a)
        size = R.permute_grad(np.abs(f64(dxp)), slot.cpu().numpy(), k, None if a is None else np.abs(a))
        assert (np.abs(f64(dx) - ref) <= np.abs(ref) * 2.0 ** -8 + size * k * 2.0 ** -23).all()
    bits = moe.permute_grad(dxp.view(torch.int16), slot, k)
    assert bits.dtype == torch.int16 and torch.equal(bits, moe.permute_grad(dxp, slot, k).view(torch.int16))


def test_zero_tokens_and_non_finite_rows(moe):
    T, d, k = 4, 256, 2
    e = _bf16(0, d)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    dy, dw = moe.combine_grad(e, e, none, torch.zeros(0, k, device="cuda"))
    assert dy.shape == (0, d) and dw.shape == (0, k)
    assert moe.permute_grad(e, none, k).shape == (0, d)
    assert moe.route_grad(none.view(0, k), dw, dw, 8).shape == (0, 8)
    dout, y, w = _bf16(T, d, seed=1), _bf16(T * k, d, seed=2), torch.rand(T, k, generator=_gen(3)).cuda()
    slot = torch.randperm(T * k, generator=_gen(4)).to(torch.int32).cuda()
    dy0, dw0 = moe.combine_grad(dout, y, slot, w)
    y2 = y.clone()
    y2[slot[3].item(), 9] = float("nan")  # slot 3 = token 1, j = 1
    dy1, dw1 = moe.combine_grad(dout, y2, slot, w)
    assert torch.equal(dy0, dy1) and dw1[1, 1].isnan()
    ok = torch.ones(T, k, dtype=torch.bool, device="cuda")
    ok[1, 1] = False
    assert torch.equal(dw0[ok], dw1[ok])


def test_way_back_together(moe):
    """loss = <c, combine(A permute(norm(x)), route(norm(x) R))> for a linear expert step A: the kernels'
    chain against float64 autograd, eager and captured; each replay against the eager result."""
    T, d, E, k = 50, 256, 8, 2
    x, nw, c = _bf16(T, d, seed=1), _bf16(d, seed=2), _bf16(T, d, seed=3)
    Rt = torch.randn(d, E, generator=_gen(4)).cuda() * 0.1
    A = (torch.randn(d, d, generator=_gen(5)) * d ** -0.5).to(torch.bfloat16).cuda()

    def chain(x):
        h, y, _, _ = moe.rmsnorm(x, nw)
        ids, w = moe.route(y.float() @ Rt, k)
        _, _, _, slot, xp, _ = moe.permute(ids, E, y.view(torch.int16))
        yp = (xp.view(torch.bfloat16).float() @ A.float()).to(torch.bfloat16)
        dy, dw = moe.combine_grad(c, yp, slot, w)
        dl = moe.route_grad(ids, w, dw, E)
        dxp = (dy.float() @ A.float().t()).to(torch.bfloat16)
        dyn = moe.permute_grad(dxp, slot, k, (dl @ Rt.t()).to(torch.bfloat16))
        return (*moe.rmsnorm_grad(dyn, h, nw), ids)

    dx, dnw, ids = (t.clone() for t in chain(x))
    xr = x.double().cpu().requires_grad_()
    wr = nw.double().cpu().requires_grad_()
    y = xr / (xr.square().mean(-1, keepdim=True) + 1e-6).sqrt() * wr
    lg = y @ Rt.double().cpu()
    w = torch.softmax(lg.gather(1, ids.long().cpu()), 1)
    out = (w[..., None] * (y @ A.double().cpu())[:, None]).sum(1)
    (out * c.double().cpu()).sum().backward()
    # bf16 is rounded to seven times on the way (y, A y, dy, dx_perm, the sum, its addend, dx): each is
    # off by 2^-8 of its own value, and the terms behind one gradient are of its row's size
    for got, ref in ((dx, xr.grad), (dnw, wr.grad)):
        assert (got.double().cpu() - ref).norm() <= 7 * 2.0 ** -8 * ref.norm()
    sx = x.clone()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        chain(sx)
    torch.cuda.current_stream().wait_stream(warm)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gx, gw, _ = chain(sx)
    for seed in (1, 8, 9):
        sx.copy_(_bf16(T, d, seed=seed))
        g.replay()
        torch.cuda.synchronize()
        ex, ew, _ = chain(sx)
        torch.cuda.synchronize()
        assert torch.equal(gx, ex) and torch.equal(gw, ew)


def test_rows_past_32_bit_offsets(moe):
    """More than 2^32 bytes of rows: every 16th token is the same token."""
    T, k, d = 40000, 8, 7168
    dst = torch.arange(T * k, dtype=torch.int32, device="cuda")
    y, dout, w = _bf16(16 * k, d, seed=1), _bf16(16, d, seed=2), torch.rand(16, k, generator=_gen(3)).cuda()
    dy0, dw0 = moe.combine_grad(dout, y, dst[:16 * k], w)
    rep = T // 16
    big = y.repeat(rep, 1)
    dy, dw = moe.combine_grad(dout.repeat(rep, 1), big, dst, w.repeat(rep, 1))
    assert torch.equal(dy.view(rep, 16 * k, d), dy0.expand(rep, 16 * k, d))
    # (16 tokens and 40000 take different numbers of threads per row: another order of the d products)
    mag = (dout.double()[:, None].abs() * y.double().view(16, k, d).abs()).sum(-1)
    assert ((dw.double().view(rep, 16, k) - dw0.double()).abs() <= 2 * (d // 64 + 16) * 2.0 ** -24 * mag).all()
    dx0 = moe.permute_grad(y, dst[:16 * k], k)
    dx = moe.permute_grad(big, dst, k)
    assert torch.equal(dx.view(rep, 16, d), dx0.expand(rep, 16, d))


@pytest.mark.parametrize("T,d", [(1500, 7168), (70000, 128)])
def test_combine_grad_beyond_the_last_level_cache(moe, T, d):
    """Sizes whose rows pass the caches by give the bits of their parts, which do not."""
    k = 8
    dst = torch.randperm(T * k, generator=_gen(1)).to(torch.int32).cuda()
    y, dout, w = _bf16(T * k, d, seed=2), _bf16(T, d, seed=3), torch.rand(T, k, generator=_gen(4)).cuda()
    dy, dw = moe.combine_grad(dout, y, dst, w)
    half = 800
    p = dst[:half * k].long()
    dyh, dwh = moe.combine_grad(dout[:half].contiguous(), y[p].contiguous(),
                                torch.arange(half * k, dtype=torch.int32, device="cuda"), w[:half].contiguous())
    assert torch.equal(dy[p], dyh) and torch.equal(dw[:half], dwh)
