"""Host checks of the training operators: bad arguments are refused before
any CUDA call (fake aligned pointers are never touched), and the plain forms
the GPU tests compare with agree with autograd and with differences."""
from __future__ import annotations

import ctypes

import pytest
import torch

import mixture_experts_feed_b200 as moe
import train_helpers as th

FAKE, BIG = 1 << 20, 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def grouped(rows=64, E=4, n=128, k=64, dtype=torch.bfloat16, out=None):
    return ctypes.byref(moe.GroupedMatmul(rows, E, n, k, dtype, out).desc())


CALLS = [moe.LIB.moe_grouped_matmul, moe.LIB.moe_grouped_matmul_dgrad,
         lambda d, a, b, off, out, *r: moe.LIB.moe_grouped_matmul_wgrad(d, a, b, off, out, 0, *r)]


@pytest.mark.parametrize("f", CALLS, ids=["forward", "dgrad", "wgrad"])
def test_grouped_refusals(f):
    d = grouped()
    for i in range(4):                                   # each pointer null, then misaligned
        args = [FAKE] * 4
        args[i] = None
        assert f(d, *args, FAKE, BIG, None) == INVALID
        args[i] = FAKE + 2
        assert f(d, *args, FAKE, BIG, None) == INVALID
    ok = [FAKE] * 4
    assert f(d, *ok, None, BIG, None) == INVALID
    assert f(d, *ok, FAKE + 16, BIG, None) == INVALID    # workspace alignment
    assert f(d, *ok, FAKE, 100, None) == WORKSPACE
    assert f(None, *ok, FAKE, BIG, None) == INVALID
    for bad in (dict(rows=-1), dict(E=0), dict(n=0), dict(k=-8)):
        assert f(grouped(**bad), *ok, FAKE, BIG, None) == INVALID
    assert f(grouped(E=1025), *ok, FAKE, BIG, None) == UNSUPPORTED
    assert f(grouped(rows=1 << 31), *ok, FAKE, BIG, None) == UNSUPPORTED
    raw = moe.GroupedDesc(64, 4, 128, 64, 1, 2)          # bf16 operands, fp16 output
    assert f(ctypes.byref(raw), *ok, FAKE, BIG, None) == INVALID
    raw = moe.GroupedDesc(64, 4, 128, 64, 7, 7)
    assert f(ctypes.byref(raw), *ok, FAKE, BIG, None) == INVALID


def test_grouped_without_rows():
    d = grouped(rows=0)
    assert moe.LIB.moe_grouped_matmul(d, None, None, None, None, None, 0, None) == 0
    assert moe.LIB.moe_grouped_matmul_dgrad(d, None, None, None, None, None, 0, None) == 0
    # the weight gradient of no rows is still written: its pointers are checked
    assert moe.LIB.moe_grouped_matmul_wgrad(d, None, None, None, FAKE, 0, FAKE, BIG, None) == INVALID


def test_grouped_accumulates_in_fp32_only():
    ok = [FAKE] * 4
    assert moe.LIB.moe_grouped_matmul_wgrad(grouped(), *ok, 1, FAKE, BIG, None) == INVALID
    with pytest.raises(ValueError):
        moe.GroupedMatmul(8, 2, 8, 8, torch.bfloat16, torch.float16).desc()
    with pytest.raises(ValueError):
        moe.GroupedMatmul(8, 2, 8, 8, torch.float64).desc()


def test_grouped_workspace_size():
    assert moe.grouped_workspace_size(moe.GroupedMatmul(1 << 20, 256, 6144, 1024)) >= 256
    assert moe.LIB.moe_grouped_workspace_size(grouped(), None) == INVALID
    n = ctypes.c_size_t(0)
    assert moe.LIB.moe_grouped_workspace_size(grouped(E=0), ctypes.byref(n)) == INVALID


def test_grouped_workspace_of_products_cut_along_the_sum():
    """Few tiles and a long sum: the workspace holds the pieces, whatever the
    output's type."""
    for shape in (dict(rows=8192, E=1, n=256, k=256), dict(rows=40000, E=64, n=512, k=512),
                  dict(rows=32, E=1, n=64, k=4096), dict(rows=32, E=1, n=4096, k=64)):
        for dt in (torch.bfloat16, torch.float16):
            size = moe.grouped_workspace_size(moe.GroupedMatmul(dtype=dt, **shape))
            assert 256 < size < 1 << 26
            assert moe.grouped_workspace_size(moe.GroupedMatmul(dtype=dt, out_dtype=torch.float32, **shape)) == size
        assert moe.grouped_workspace_size(moe.GroupedMatmul(dtype=torch.float32, **shape)) == 256
    assert moe.grouped_workspace_size(moe.GroupedMatmul(24576, 64, 2048, 2048)) == 256
    assert moe.grouped_workspace_size(moe.GroupedMatmul(64, 64, 4096, 2048)) == 256


def swiglu_call(name, rows=64, I=32, dtype=moe.MOE_BF16, E=4, off=FAKE, slot=FAKE, w=FAKE, ptrs=None,
                ws=FAKE, nbytes=BIG):
    f = getattr(moe.LIB, name)
    p = dict(a=FAKE, b=FAKE, c=FAKE, d=FAKE, e=FAKE)
    p.update(ptrs or {})
    if name == "moe_swiglu_checkpoint":     # gu; h, q, scale
        return f(rows, I, dtype, p["a"], E, off, slot, w, p["b"], p["c"], p["d"], ws, nbytes, None)
    return f(rows, I, dtype, p["a"], p["b"], p["c"], E, off, slot, w, p["d"], FAKE, p["e"], ws, nbytes,
             None)


@pytest.mark.parametrize("name", ["moe_swiglu_checkpoint", "moe_swiglu_backward"])
def test_swiglu_refusals(name):
    for key in "abcd":
        assert swiglu_call(name, ptrs={key: None}) == INVALID
        assert swiglu_call(name, ptrs={key: FAKE + 4}) == INVALID
    assert swiglu_call(name, rows=-1) == INVALID
    assert swiglu_call(name, I=0) == INVALID
    assert swiglu_call(name, I=24) == UNSUPPORTED
    assert swiglu_call(name, rows=1 << 31) == UNSUPPORTED
    assert swiglu_call(name, dtype=moe.MOE_BF16_F16DOWN) == INVALID
    assert swiglu_call(name, w=None) == INVALID                 # a row map without weights
    assert swiglu_call(name, E=0) == INVALID                    # offsets of no groups
    assert swiglu_call(name, ws=None) == INVALID
    assert swiglu_call(name, nbytes=128) == WORKSPACE
    assert swiglu_call(name, rows=0, ptrs=dict(a=None, b=None, c=None, d=None)) == 0


def test_norm_refusals():
    F32 = moe.MOE_F32
    ln, lb, rb = moe.LIB.moe_layer_norm, moe.LIB.moe_layer_norm_backward, moe.LIB.moe_rmsnorm_backward
    for i in (0, 1, 3):                                          # bias (2) may be null
        p = [FAKE] * 4
        p[i] = None
        assert ln(8, 64, F32, 1e-6, *p, None) == INVALID
    assert ln(8, 64, F32, 1e-6, FAKE, FAKE, FAKE + 8, FAKE, None) == INVALID
    assert ln(-1, 64, F32, 1e-6, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert ln(8, 0, F32, 1e-6, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert ln(8, 64, 2, 1e-6, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert ln(8, 64, F32, -1.0, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert ln(8, 64, F32, float("nan"), FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert ln(0, 64, F32, 1e-6, None, None, None, None, None) == 0
    for i in (0, 1, 2, 4, 5):                                    # dres (3) may be null
        p = [FAKE] * 6
        p[i] = None
        assert lb(8, 64, F32, 1e-6, *p, None, FAKE, BIG, None) == INVALID
        assert rb(8, 64, F32, 1e-6, *p, FAKE, BIG, None) == INVALID
    p = [FAKE] * 6
    assert lb(8, 64, F32, 1e-6, *p, FAKE, FAKE, 1024, None) == WORKSPACE
    assert rb(8, 64, F32, 1e-6, *p, None, BIG, None) == INVALID
    assert lb(8, 64, F32, float("inf"), *p, FAKE, FAKE, BIG, None) == INVALID
    n = ctypes.c_size_t(0)
    assert moe.LIB.moe_norm_workspace_size(8, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert moe.LIB.moe_norm_workspace_size(8, 0, ctypes.byref(n)) == INVALID


def test_binding_refuses_before_the_library():
    """Tensors of a wrong shape, dtype, layout or device raise in the binding."""
    G = moe.GroupedMatmul(4, 2, 8, 16)
    a, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    off, out = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_grouped_matmul(G, a, w, off, out, ws)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_grouped_matmul(G, a[:3], w, off, out, ws)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_grouped_matmul_dgrad(G, out.float(), w, off, a, ws)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_grouped_matmul_wgrad(G, out.t().contiguous().t(), a, off, w, ws)
    with pytest.raises(ValueError):
        moe.moe_layer_norm(torch.zeros(4, 8, dtype=torch.float16), a, a, a)
    with pytest.raises(ValueError):
        moe.moe_swiglu_checkpoint(torch.zeros(4, 33), None, None, None, a, a, a, ws)


def test_quantise_definition():
    """The helper's search for the scale, on values worked by hand: 448 fits
    2^0 exactly, the next bf16 above it needs 2^1; 17/16 is a tie between 1
    and 1.125 and goes to the even 1."""
    x = torch.zeros(1, 96)
    x[0, 0], x[0, 1] = 448.0, 17 / 16
    x[0, 32], x[0, 33] = 450.0, -3.0
    q, b = th.quantise_exact(x)
    assert b.tolist() == [[127, 128, 0]]
    assert q[0, 0] == 448 and q[0, 1] == 1.0 and q[0, 32] == 224 and q[0, 33] == -1.5
    assert torch.equal(th.dequantise(q.to(torch.float8_e4m3fn), b)[0, 64:], torch.zeros(32, dtype=torch.float64))


def test_plain_gradients_agree_with_differences():
    """The formulas the header gives, against central differences in fp64."""
    torch.manual_seed(0)
    g, u, dh = (torch.randn(3, 8, dtype=torch.float64) for _ in range(3))
    w = torch.rand(3, 1, dtype=torch.float64)
    f = lambda g, u, w: (dh * w * g * torch.sigmoid(g) * u).sum()   # noqa: E731
    s = torch.sigmoid(g)
    dg, du, dw = w * dh * u * s * (1 + g * (1 - s)), w * dh * g * s, (dh * g * s * u).sum(1, keepdim=True)
    t = 1e-5
    for i in range(3):
        v = torch.randn_like(g)
        assert abs((f(g + t * v, u, w) - f(g - t * v, u, w)) / (2 * t) - (dg * v).sum()) < 1e-8
        assert abs((f(g, u + t * v, w) - f(g, u - t * v, w)) / (2 * t) - (du * v).sum()) < 1e-8
        v = torch.randn_like(w)
        assert abs((f(g, u, w + t * v) - f(g, u, w - t * v)) / (2 * t) - (dw * v).sum()) < 1e-8
    x, wt, b, do = (torch.randn(5, 12, dtype=torch.float64) for _ in range(4))
    wt, b = wt[0], b[0]
    for layer in (False, True):
        n = lambda x, wt: (do * th.norm_exact(x, wt, b, 1e-6, layer)[2]).sum()   # noqa: E731
        xh, r, _ = th.norm_exact(x, wt, b, 1e-6, layer)
        gy = do * wt
        dx = r * (gy - (gy.mean(1, keepdim=True) if layer else 0) - xh * (gy * xh).mean(1, keepdim=True))
        v = torch.randn_like(x)
        assert abs((n(x + t * v, wt) - n(x - t * v, wt)) / (2 * t) - (dx * v).sum()) < 1e-7
        v = torch.randn_like(wt)
        assert abs((n(x, wt + t * v) - n(x, wt - t * v)) / (2 * t) - ((do * xh).sum(0) * v).sum()) < 1e-7
