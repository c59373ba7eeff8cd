"""Refusals of the int8, norm and gradient entry points: on the host, before any GPU work."""
import ctypes

import pytest
import torch

from mixture_experts_layer_top_amd import moe

INV, UNS, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
A = 4096  # stands for an aligned device pointer; no call here gets as far as using it


@pytest.fixture(scope="module")
def L():
    return moe.lib()


def test_rmsnorm_refusals(L):
    def call(x=A, r=None, w=A, eps=1e-6, T=2, d=256, act=moe.DTYPE_BF16, h=None, y=A, q=None, qs=None):
        return L.moe_rmsnorm(x, r, w, eps, T, d, act, h, y, q, qs, None)

    assert call(T=0) == moe.MOE_OK
    assert call(T=-1) == INV and call(d=0) == INV and call(eps=-1.0) == INV
    assert call(eps=float("nan")) == INV
    assert call(x=None) == INV and call(w=None) == INV and call(y=None) == INV
    for name in ("x", "r", "w", "h", "y"):
        assert call(**{name: A + 8}) == INV
    assert call(act=moe.DTYPE_INT8, q=A + 8, qs=A) == INV
    assert call(act=moe.DTYPE_INT8, y=None) == INV and call(act=moe.DTYPE_INT8, q=A) == INV
    assert call(d=252) == UNS and call(d=32776) == UNS
    assert call(d=264, act=moe.DTYPE_INT8, q=A, qs=A) == UNS
    assert call(d=240, act=moe.DTYPE_MXFP4_A8, q=A, qs=A) == UNS
    assert call(d=192, act=moe.DTYPE_FP8, q=A, qs=A) == UNS
    for act in (moe.DTYPE_MXFP4, 5, -1):
        assert call(act=act, q=A, qs=A) == UNS


def test_rmsnorm_grad_refusals(L):
    def call(dy=A, dh=None, h=A, w=A, eps=1e-6, T=2, d=256, dx=A, dw=A, ws=A, n=1 << 30):
        return L.moe_rmsnorm_grad(dy, dh, h, w, eps, T, d, dx, dw, ws, n, None)

    need = L.moe_rmsnorm_grad_workspace_bytes
    assert need(2, 256) >= 2 * 256 * 4 and need(0, 256) == 0
    assert need(2, 252) == 0 and need(2, 16392) == 0 and need(-1, 256) == 0
    assert call(T=0, dw=None) == moe.MOE_OK
    assert call(T=-1) == INV and call(d=-8) == INV and call(eps=-1.0) == INV
    assert call(d=252) == UNS and call(d=16392) == UNS
    for name in ("dy", "h", "w", "dx"):
        assert call(**{name: None}) == INV
    for name in ("dy", "dh", "h", "w", "dx", "dw", "ws"):
        assert call(**{name: A + 8}) == INV
    assert call(ws=None) == WS and call(n=need(2, 256) - 1) == WS


def test_int8_refusals(L):
    assert L.moe_quant_act_i8(A, 0, 128, A, A, None) == moe.MOE_OK
    assert L.moe_quant_act_i8(A, -1, 128, A, A, None) == INV
    assert L.moe_quant_act_i8(A, 1, 120, A, A, None) == UNS
    assert L.moe_quant_act_i8(A, 1, 32784, A, A, None) == UNS
    assert L.moe_quant_act_i8(None, 1, 128, A, A, None) == INV
    assert L.moe_quant_act_i8(A, 1, 128, A + 4, A, None) == INV

    def gemm(xq=A, xs=A, M=4, w=A, ws=A, N=256, K=256, y=A):
        return L.moe_gemm_i8(xq, xs, M, w, ws, N, K, y, None)

    assert gemm(M=0) == moe.MOE_OK
    assert gemm(M=-1) == INV and gemm(N=0) == INV and gemm(K=0) == INV
    assert gemm(N=24) == UNS and gemm(K=192) == UNS and gemm(K=32896) == UNS
    assert gemm(M=1 << 24) == UNS and gemm(N=1 << 24) == UNS  # 2^32 bytes
    for name in ("xq", "xs", "w", "ws", "y"):
        assert gemm(**{name: None}) == INV
    for name in ("xq", "w", "ws", "y"):
        assert gemm(**{name: A + 8}) == INV


def test_int8_experts_refusals(L):
    ptrs = dict(w_gate=256, w_up=512, w_down=768, s_gate=1024, s_up=1280, s_down=1536)
    p = moe.problem(8, 256, 512, 8, 2, wdtype=moe.DTYPE_INT8)
    need = L.moe_layer_workspace_bytes

    def layer(w, p=p):
        return L.moe_layer(ctypes.byref(p), A, A, ctypes.byref(w), A, None, A, 16, None)

    def ffn(w, xs=A, p=p):
        return L.moe_grouped_ffn(ctypes.byref(p), A, xs, A, A, ctypes.byref(w), A, A, 16, None)

    ok = moe.Weights(**ptrs, layout=moe.LAYOUT_TILED)
    assert layer(ok) == WS and ffn(ok) == WS and ffn(ok, xs=None) == INV
    assert layer(moe.Weights(**ptrs, layout=moe.LAYOUT_ROW_MAJOR)) == INV
    for s in ("s_gate", "s_up", "s_down"):
        for v in (None, ptrs[s] + 4):
            bad = moe.Weights(**dict(ptrs, **{s: v}), layout=moe.LAYOUT_TILED)
            assert layer(bad) == INV and ffn(bad) == INV
    # whole rows are quantised: d, d_ff and d_ff_shared up to 32768
    for kw in (dict(d=32896, f=128), dict(d=128, f=32896), dict(d=128, f=128, shared_f=32896)):
        q = moe.problem(2, kw["d"], kw["f"], 4, 2, wdtype=moe.DTYPE_INT8, shared_f=kw.get("shared_f", 0))
        assert need(ctypes.byref(q)) == 0
    assert need(ctypes.byref(moe.problem(2, 32768, 128, 4, 2, wdtype=moe.DTYPE_INT8))) > 0
    for cfg in (moe.CONFIG_POLICY0, moe.CONFIG_FUSED):  # bf16 forms
        assert need(ctypes.byref(moe.problem(1, 256, 512, 8, 2, wdtype=moe.DTYPE_INT8, config=cfg))) == 0
    sh = moe.problem(8, 256, 512, 8, 2, wdtype=moe.DTYPE_INT8, shared_f=256)
    shp = dict(ptrs, sh_gate=256, sh_up=512, sh_down=768, s_sh_gate=1024, s_sh_up=1280, s_sh_down=1536)
    assert layer(moe.Weights(**shp, layout=moe.LAYOUT_TILED), sh) == WS
    for s in ("s_sh_gate", "s_sh_up", "s_sh_down"):
        for v in (None, shp[s] + 4):
            assert layer(moe.Weights(**dict(shp, **{s: v}), layout=moe.LAYOUT_TILED), sh) == INV
    # permute carries int8 rows with one scale each
    assert L.moe_permute(A, 4, 8, 2, A, None, 256, moe.DTYPE_INT8, A, A, A, A, A, A, A, 1 << 20, None) == INV
    assert L.moe_permute(A, 4, 8, 2, A, A, 256, moe.DTYPE_MXFP4, A, A, A, A, A, A, A, 1 << 20, None) == UNS


def test_sort_gradient_refusals(L):
    assert L.moe_route_grad(A, A, A, 0, 8, 2, A, None) == moe.MOE_OK
    assert L.moe_route_grad(A, A, A, 2, 8, 9, A, None) == UNS
    assert L.moe_route_grad(A, A, A, 2, 513, 2, A, None) == UNS
    assert L.moe_route_grad(A, A, A, 2, 8, 0, A, None) == INV
    for i in (0, 1, 2, 6):
        args = [A, A, A, 2, 8, 2, A, None]
        args[i] = None
        assert L.moe_route_grad(*args) == INV

    def cg(dout=A, y=A, slot=A, w=A, T=2, k=2, d=256, dy=A, dw=A):
        return L.moe_combine_grad(dout, y, slot, w, T, k, d, dy, dw, None)

    assert cg(T=0) == moe.MOE_OK
    assert cg(T=-1) == INV and cg(k=0) == INV and cg(d=0) == INV
    assert cg(k=9) == UNS and cg(d=192) == UNS and cg(d=32896) == UNS and cg(T=1 << 30) == UNS
    assert cg(dy=None, dw=None) == INV and cg(dout=None) == INV and cg(slot=None) == INV
    assert cg(y=None) == INV and cg(w=None) == INV
    for name in ("dout", "y", "dy"):
        assert cg(**{name: A + 8}) == INV

    def pg(dxp=A, slot=A, add=None, T=2, k=2, d=256, dx=A):
        return L.moe_permute_grad(dxp, slot, add, T, k, d, dx, None)

    assert pg(T=0) == moe.MOE_OK
    assert pg(T=-1) == INV and pg(k=0) == INV and pg(k=9) == UNS and pg(d=192) == UNS
    assert pg(T=1 << 30) == UNS
    for name in ("dxp", "slot", "dx"):
        assert pg(**{name: None}) == INV
    for name in ("dxp", "add", "dx"):
        assert pg(**{name: A + 8}) == INV


def test_binding_refusals():
    """The binding checks types, shapes, contiguity and device before the library sees a pointer."""
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(moe.MoEError, match="GPU"):
        moe.rmsnorm(x, w)
    with pytest.raises(moe.MoEError, match="x must be"):
        moe.rmsnorm(x.float(), w)
    with pytest.raises(moe.MoEError, match="contiguous"):
        moe.rmsnorm(torch.zeros(256, 4, dtype=torch.bfloat16).t(), w)
    with pytest.raises(moe.MoEError, match="two dimensions"):
        moe.rmsnorm(x[0], w)
    with pytest.raises(moe.MoEError, match="GPU"):
        moe.quant_act_i8(x)
    with pytest.raises(moe.MoEError, match="torch.int8"):
        moe.int8_tile(torch.zeros(16, 128, dtype=torch.uint8))
    with pytest.raises(moe.MoEError, match="multiple of k"):
        moe.permute_grad(x, torch.zeros(4, dtype=torch.int32), 3)
    g = torch.zeros((2, 128, 128), dtype=torch.int8)
    s = torch.ones((2, 128))
    ew = moe.ExpertWeights(gate=g, up=g, down=g, s_gate=s, s_up=s, s_down=s)
    assert ew.wdtype == moe.DTYPE_INT8 and ew.struct().layout == moe.LAYOUT_ROW_MAJOR
    g._moe_tiled = True
    assert ew.struct().layout == moe.LAYOUT_TILED


def test_more_rows_than_a_launch_has_threads_for(L):
    T = 1 << 25
    assert L.moe_quant_act_i8(A, T, 16, A, A, None) == UNS
    assert L.moe_rmsnorm(A, None, A, 1e-6, T, 8, moe.DTYPE_BF16, None, A, None, None, None) == UNS
    assert L.moe_rmsnorm_grad(A, None, A, A, 1e-6, T, 8, A, A, A, 1 << 30, None) == UNS
    assert L.moe_rmsnorm_grad_workspace_bytes(T, 8) == 0 and L.moe_rmsnorm_grad_workspace_bytes(T - 1, 8) > 0
    assert L.moe_route_grad(A, A, A, T, 8, 2, A, None) == UNS
    assert L.moe_combine_grad(A, A, A, A, T, 2, 128, A, A, None) == UNS
    assert L.moe_permute_grad(A, A, None, 1 << 24, 2, 128, A, None) == UNS  # 256 threads each
    assert L.moe_permute_grad(A, A, None, 1 << 26, 2, 512, A, None) == UNS  # 64 threads each


def test_binding_runs_on_the_tensors_gpu(monkeypatch):
    """Tensors of a GPU that is not the current one: the library is called with that GPU current and its
    stream, tiling included."""
    import contextlib
    current = [0]

    @contextlib.contextmanager
    def device(i):
        was, current[0] = current[0], i
        yield
        current[0] = was

    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: calls.append((name, current[0], args[-1])) or 0

    class OnGpu1:
        dtype, is_cuda, device, shape = torch.int8, True, torch.device("cuda", 1), (16, 128)
        get_device = staticmethod(lambda: 1)
        contiguous = empty_like = lambda self: self
        numel = staticmethod(lambda: 2048)
        data_ptr = staticmethod(lambda: 0)

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(moe, "_stream", lambda: 100 + current[0])
    monkeypatch.setattr(moe, "lib", Lib)
    monkeypatch.setattr(torch, "empty_like", lambda t: OnGpu1())
    moe._run("moe_quant_act_i8", 1, 7)
    assert moe.int8_tile(OnGpu1())._moe_tiled
    moe._run("moe_quant_act_i8", 0, 7)
    assert calls == [("moe_quant_act_i8", 1, 101), ("moe_fp8_tile", 1, 101), ("moe_quant_act_i8", 0, 100)]
    assert current == [0]
