"""GPU tests of the training operators (grouped products and their gradients,
SwiGLU with its 8-bit checkpoint, the norms' passes) against plain fp64
forms, at the sizes and masks where such kernels go wrong, and of a run of
them together as a training step uses them."""
from __future__ import annotations

import pytest
import torch

import train_helpers as th

pytestmark = pytest.mark.gpu

try:
    import mixture_experts_feed_b200 as moe
except ImportError:   # collected on CPU-only machines too; the gpu marker deselects
    moe = None

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
CALL = {"forward": "moe_grouped_matmul", "dgrad": "moe_grouped_matmul_dgrad",
        "wgrad": "moe_grouped_matmul_wgrad"}


# ---------------------------------------------------------- grouped products
def grouped_inputs(form, sizes, n, k, dtype, out, pad=0, seed=0, device="cuda"):
    """Operands of a product; rows behind the last group hold NaN, the output
    a pattern of its own."""
    g = torch.Generator(device=device).manual_seed(seed)
    E, R = len(sizes), sum(sizes) + pad
    rnd = lambda *s: torch.randn(*s, generator=g, device=device)   # noqa: E731
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device=device)
    rows_p = rnd(R, k if form == "forward" else n).to(dtype)
    rows_p[R - pad:] = float("nan")
    if form == "wgrad":
        q = rnd(R, k).to(dtype)
        q[R - pad:] = float("nan")
        o = rnd(E, n, k).to(out)
    else:
        q = (rnd(E, n, k) * 0.1).to(dtype)
        o = rnd(R, n if form == "forward" else k).to(out)
    return moe.GroupedMatmul(R, E, n, k, dtype, out), rows_p, q, off, o


def run_grouped(form, G, p, q, off, out, ws=None, **kw):
    ws = moe.new_grouped_workspace(G) if ws is None else ws
    getattr(moe, CALL[form])(G, p, q, off, out, ws, **kw)
    torch.cuda.synchronize()
    assert moe.read_device_status(ws) == 0
    return out


def check_grouped(form, sizes, n, k, dtype, out, pad=0, accumulate=False, seed=0):
    G, p, q, off, o = grouped_inputs(form, sizes, n, k, dtype, out, pad, seed)
    o0 = o.clone()
    kw = dict(accumulate=True) if accumulate else {}
    run_grouped(form, G, p, q, off, o, **kw)
    ref, mag, n_sum = th.grouped_exact(form, p, q, off, o0, accumulate)
    th.check(o, ref, th.grouped_bound(ref, mag, n_sum, out), f"{form} {sizes[:6]} {n} {k}")
    again = o0.clone()
    run_grouped(form, G, p, q, off, again, **kw)
    assert torch.equal(again, o), "two runs differ"


RAGGED = [5, 0, 130, 1, 64, 0, 0, 257, 63, 128, 16, 17]
SHAPES = [  # n, k
    (128, 64), (256, 256), (320, 448), (8, 8), (72, 1000), (520, 40), (1000, 136)]


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (F32, F32)],
                         ids=["bf16", "bf16-f32", "f16", "f32"])
def test_grouped_ragged(form, n, k, dtype, out):
    check_grouped(form, RAGGED, n, k, dtype, out, pad=37)


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, F32), (F32, F32)])
def test_grouped_sizes_tma_cannot_take(form, dtype, out):
    """Row lengths that are no whole 16-byte vectors."""
    check_grouped(form, [3, 0, 70, 65], 33, 51, dtype, out, pad=2)
    check_grouped(form, [1], 1, 1, dtype, out)


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("sizes", [[1], [0, 0, 1, 0], [300], [2000, 0, 3], [1] * 40, [0, 0],
                                   [512, 256, 384], [15, 1, 31, 33, 47, 49], [4096]])
def test_grouped_group_sizes(form, sizes):
    check_grouped(form, sizes, 264, 328, BF, BF, pad=5)


# weight gradients of few tiles and many rows, input gradients and forward
# products of few tiles and long sums: cut along the sum
@pytest.mark.parametrize("sizes", [[0, 20000, 0], [4073], [10000, 1, 0, 7000, 3],
                                   [0] * 300 + [16001, 500] + [0] * 9, [0, 64 * 74 * 8 + 65], [409] * 40, [2500]])
@pytest.mark.parametrize("n,k", [(8, 8), (136, 264), (520, 40), (256, 256)])
@pytest.mark.parametrize("dtype,out,accumulate", [(BF, BF, False), (HF, F32, False), (BF, F32, True), (HF, HF, False)])
def test_wgrad_cut_along_the_rows(sizes, n, k, dtype, out, accumulate):
    check_grouped("wgrad", sizes, n, k, dtype, out, pad=37, accumulate=accumulate)


@pytest.mark.parametrize("sizes", [[1], [0, 7, 0, 2], [31, 33], [200, 0, 1], [700]])
@pytest.mark.parametrize("wide,deep", [(8, 4096), (136, 4000), (264, 6152), (1000, 2056)])
@pytest.mark.parametrize("form", ["forward", "dgrad"])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, F32), (HF, HF), (BF, F32)])
def test_products_cut_along_the_sum(form, sizes, wide, deep, dtype, out):
    n, k = (wide, deep) if form == "forward" else (deep, wide)
    check_grouped(form, sizes, n, k, dtype, out, pad=5)


@pytest.mark.parametrize("form", ["forward", "dgrad"])
@pytest.mark.parametrize("sizes", [[1], [3, 0, 9, 8, 0, 1], [64], [0, 50], [63]])
@pytest.mark.parametrize("n,k", [(64, 128), (33, 51), (200, 4), (7, 260)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_grouped_few_rows_on_the_cuda_cores(form, sizes, n, k, dtype):
    check_grouped(form, sizes, n, k + (dtype == BF), dtype, dtype, pad=64 - sum(sizes))


# four rows an expert at most, and the rows at once around their limit
@pytest.mark.parametrize("form", ["forward", "dgrad"])
@pytest.mark.parametrize("sizes", [[1], [2], [3], [4], [2, 0, 0, 10], [0] * 40 + [17, 2, 1] + [0] * 5, [4] * 30])
@pytest.mark.parametrize("n,k", [(64, 128), (36, 260), (1000, 4), (132, 1000)])
def test_grouped_up_to_four_rows_an_expert(form, sizes, n, k):
    check_grouped(form, sizes, n, k, F32, F32)


# enough 64 x 64 tiles for every SM, and fewer full ones of 128
@pytest.mark.parametrize("sizes,n,k", [([700, 0, 500, 300], 392, 332), ([1500], 333, 391), ([90, 1, 260, 700], 700, 321)])
@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF, BF), (HF, F32)])
def test_grouped_many_tiles_on_the_cuda_cores(form, sizes, n, k, dtype, out):
    check_grouped(form, sizes, n, k + (k % 8 == 0 and dtype != F32), dtype, out, pad=3)
    if form == "wgrad" and out == F32:
        check_grouped(form, sizes, n, k + (k % 8 == 0 and dtype != F32), dtype, out, pad=3, accumulate=True)


@pytest.mark.parametrize("sizes", [RAGGED, [0, 0], [3000, 0, 1]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_wgrad_accumulates(sizes, dtype):
    check_grouped("wgrad", sizes, 136, 200, dtype, F32, pad=11, accumulate=True)


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
def test_grouped_many_experts(form):
    g = torch.Generator().manual_seed(3)
    sizes = torch.randint(0, 4, (1024,), generator=g).tolist()
    check_grouped(form, sizes, 64, 72, BF, BF, pad=1)


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("sizes", [[300] + [0] * 300 + [40], [0] * 400, [0, 1] * 150],
                         ids=["one", "none", "every other"])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_grouped_runs_of_experts_without_rows(form, sizes, out):
    check_grouped(form, sizes, 520, 264, BF, out, pad=3)


@pytest.mark.parametrize("form,n,k", [("forward", 256, 6144), ("dgrad", 6144, 256), ("wgrad", 256, 264)])
def test_grouped_long_sums_in_fp32(form, n, k):
    """Long reductions with fp32 outputs: at most twice the error of fp32 sums
    that round (rms of the result's 2-norm; 2e-5 / 2 is a tenth of a bf16
    step's thousandth)."""
    sizes = [9000, 500] if form == "wgrad" else [300, 100]
    G, p, q, off, o = grouped_inputs(form, sizes, n, k, BF, F32)
    run_grouped(form, G, p, q, off, o)
    ref, _, _ = th.grouped_exact(form, p, q, off, o)
    rel = float((o.double() - ref).norm() / ref.norm())
    assert rel < 1e-5, rel


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
def test_grouped_non_finite_values_stay_in_their_rows(form):
    """An infinity or NaN of one group reaches no other group's result, also
    where two groups share a tile of rows."""
    sizes = [70, 20, 50]
    G, p, q, off, o = grouped_inputs(form, sizes, 136, 128, BF, BF)
    p[75, 3] = float("inf")
    p[80, 5] = float("nan")
    if form == "wgrad":
        q[85, 7] = float("-inf")
    run_grouped(form, G, p, q, off, o)
    if form == "wgrad":
        assert not bool(torch.isfinite(o[1]).all())
        fine = torch.tensor([0, 2], device="cuda")
        assert bool(torch.isfinite(o[fine]).all())
        ref, mag, m = th.grouped_exact(form, p.nan_to_num(0, 0, 0), q.nan_to_num(0, 0, 0), off, o)
        th.check(o[fine], ref[fine], th.grouped_bound(ref, mag, m, BF)[fine], "other groups")
    else:
        rows = torch.ones(140, dtype=torch.bool, device="cuda")
        rows[75] = rows[80] = False
        assert not bool(torch.isfinite(o[75]).any()) and bool(torch.isnan(o[80]).all())
        ref, mag, m = th.grouped_exact(form, p.nan_to_num(0, 0, 0), q, off, o)
        th.check(o[rows], ref[rows], th.grouped_bound(ref, mag, m, BF)[rows], "other rows")


def test_grouped_products_of_no_rows():
    """A batch without rows: nothing is written but the weight gradient's zeros."""
    for dtype, out in ((BF, BF), (BF, F32), (F32, F32)):
        G = moe.GroupedMatmul(0, 3, 72, 40, dtype, out)
        ws = moe.new_grouped_workspace(G)
        z = lambda *s: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
        off = torch.zeros(4, dtype=torch.int32, device="cuda")
        moe.moe_grouped_matmul(G, z(0, 40), z(3, 72, 40), off, z(0, 72).to(out), ws)
        moe.moe_grouped_matmul_dgrad(G, z(0, 72), z(3, 72, 40), off, z(0, 40).to(out), ws)
        dw = torch.full((3, 72, 40), 5.0, dtype=out, device="cuda")
        moe.moe_grouped_matmul_wgrad(G, z(0, 72), z(0, 40), off, dw, ws)
        assert bool((dw == 0).all())
        if out == F32:
            dw.fill_(5.0)
            moe.moe_grouped_matmul_wgrad(G, z(0, 72), z(0, 40), off, dw, ws, accumulate=True)
            assert bool((dw == 5.0).all())
        assert moe.read_device_status(ws) == 0


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_grouped_infinite_and_nan_operands_stay_out_of_padding(form, dtype):
    """The summed side ends inside a block of 64 and the outputs inside a tile:
    what lies behind them in memory (here infinities in the next expert's
    weights and rows) must not leak in."""
    sizes, n, k = [33, 7], 72, 88
    G, p, q, off, o = grouped_inputs(form, sizes, n, k, dtype, dtype)
    p[33:] = float("inf")
    q[(slice(33, None) if form == "wgrad" else 1)] = float("inf")
    run_grouped(form, G, p, q, off, o)
    mine = o[0] if form == "wgrad" else o[:33]
    ref, mag, m = th.grouped_exact(form, p.nan_to_num(0, 0, 0), q.nan_to_num(0, 0, 0), off, torch.zeros_like(o))
    pick = 0 if form == "wgrad" else slice(0, 33)
    th.check(mine, ref[pick], th.grouped_bound(ref, mag, m, dtype)[pick], form)


def test_grouped_bad_offsets_are_recorded():
    G, p, q, off, o = grouped_inputs("forward", [10, 10], 64, 64, BF, BF)
    ws = moe.new_grouped_workspace(G)
    bad = torch.tensor([0, 12, 500], dtype=torch.int32, device="cuda")
    moe.moe_grouped_matmul(G, p, q, bad, o, ws)
    with pytest.raises(moe.MoEError):
        moe.read_device_status(ws)
    # read as [0, 12, 20]
    ref, mag, m = th.grouped_exact("forward", p, q, torch.tensor([0, 12, 20]), o)
    th.check(o, ref, th.grouped_bound(ref, mag, m, BF), "clamped offsets")


def test_grouped_bad_offsets_of_a_cut_product():
    G, p, q, off, o = grouped_inputs("wgrad", [9000, 9000], 64, 72, BF, F32)
    ws = moe.new_grouped_workspace(G)
    assert ws.numel() > 256
    bad = torch.tensor([0, 17000, 1 << 30], dtype=torch.int32, device="cuda")
    moe.moe_grouped_matmul_wgrad(G, p, q, bad, o, ws)
    with pytest.raises(moe.MoEError):
        moe.read_device_status(ws)
    ref, mag, m = th.grouped_exact("wgrad", p, q, torch.tensor([0, 17000, 18000]), o)
    th.check(o, ref, th.grouped_bound(ref, mag, m, F32), "clamped offsets")


def test_products_in_a_smaller_workspace_run_uncut():
    for form, sizes, n, k in (("wgrad", [9000, 9000], 64, 72), ("forward", [40, 3], 64, 4096), ("dgrad", [40, 3], 4096, 64)):
        G, p, q, off, o = grouped_inputs(form, sizes, n, k, BF, F32)
        full = moe.grouped_workspace_size(G)
        assert full > 256
        ref, mag, m = th.grouped_exact(form, p, q, off, o)
        for size in (256, full - 1, full):
            ws = torch.zeros(full + 64, dtype=torch.uint8, device="cuda")
            ws[size:] = 77
            o.fill_(float("nan"))
            run_grouped(form, G, p, q, off, o, ws[:size])
            th.check(o, ref, th.grouped_bound(ref, mag, m, F32), f"{form} {size}")
            assert bool((ws[size:] == 77).all())


def test_cut_products_in_a_graph():
    """A forward product, its gradients and an accumulation, all cut, over one
    workspace: captured and replayed with other rows and other group lengths."""
    R, E, n, k = 20000, 5, 64, 4104
    G, GF = moe.GroupedMatmul(R, E, n, k, BF), moe.GroupedMatmul(200, E, n, k, BF)
    GD, GW = moe.GroupedMatmul(200, E, k, n, BF, F32), moe.GroupedMatmul(R, E, n, 136, BF, F32)
    ws = max((moe.new_grouped_workspace(g) for g in (G, GF, GD, GW)), key=torch.Tensor.numel)
    mk = lambda *s: torch.randn(*s, device="cuda").to(BF)   # noqa: E731
    st = dict(x=mk(200, k), w=mk(E, n, k), w2=mk(E, k, n), d=mk(R, n), a=mk(R, 136))
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off_few = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    mko = lambda: (torch.zeros(200, n, dtype=BF, device="cuda"), torch.zeros(200, n, device="cuda"),   # noqa: E731
                   torch.zeros(E, n, 136, device="cuda"))

    def step(o, ws):
        moe.moe_grouped_matmul(GF, st["x"], st["w"], off_few, o[0], ws)
        moe.moe_grouped_matmul_dgrad(GD, st["x"], st["w2"], off_few, o[1], ws)
        moe.moe_grouped_matmul_wgrad(GW, st["d"], st["a"], off, o[2], ws)
        moe.moe_grouped_matmul_wgrad(GW, st["d"], st["a"], off, o[2], ws, accumulate=True)

    o = mko()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(o, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o, ws)
    for sizes in ([0, 19000, 0, 600, 3], [4000] * 5, [0] * 5, [1, 2, 3, 4, 5]):
        for t in st.values():
            t.copy_(torch.randn(t.shape, device="cuda"))
        off[1:].copy_(torch.tensor(sizes).cumsum(0))
        off_few[1:].copy_(torch.tensor(sizes).cumsum(0).clamp(max=200))
        graph.replay()
        torch.cuda.synchronize()
        assert moe.read_device_status(ws) == 0
        ref, mag, m = th.grouped_exact("wgrad", st["d"], st["a"], off, o[2])
        th.check(o[2], 2 * ref, 2 * th.grouped_bound(ref, mag, m + 1, F32), f"dW {sizes}")
        live = int(off_few[-1])
        for got, form, w, dt in ((o[0], "forward", st["w"], BF), (o[1], "dgrad", st["w2"], F32)):
            ref, mag, m = th.grouped_exact(form, st["x"], w, off_few, got)
            th.check(got[:live], ref[:live], th.grouped_bound(ref, mag, m, dt)[:live], f"{form} {sizes}")
        o2 = mko()
        step(o2, torch.cat([ws[:256], torch.empty_like(ws[256:])]))
        for x, y in zip(o, o2):
            assert torch.equal(x[:live], y[:live])


def test_grouped_output_past_2_to_31_elements():
    n, k, rows = 8192, 64, 300_000
    G = moe.GroupedMatmul(rows, 2, n, k, BF, BF)
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn(rows, k, generator=g, device="cuda").to(BF)
    w = torch.randn(2, n, k, generator=g, device="cuda").to(BF)
    off = torch.tensor([0, 299_000, rows], dtype=torch.int32, device="cuda")
    out = torch.zeros(rows, n, dtype=BF, device="cuda")
    run_grouped("forward", G, a, w, off, out)
    pick = torch.tensor([0, 1, 262_143, 262_144, 262_145, 298_999, 299_000, rows - 1], device="cuda")
    e = (pick >= 299_000).long()
    ref = torch.einsum("rk,rnk->rn", a[pick].double(), w[e].double())
    mag = torch.einsum("rk,rnk->rn", a[pick].double().abs(), w[e].double().abs())
    th.check(out[pick], ref, th.grouped_bound(ref, mag, torch.full_like(ref, k), BF), "far rows")
    # and back: the far rows as an operand
    da = torch.zeros(rows, k, dtype=BF, device="cuda")
    run_grouped("dgrad", G, out, w, off, da)
    ref = torch.einsum("rn,rnk->rk", out[pick].double(), w[e].double())
    mag = torch.einsum("rn,rnk->rk", out[pick].double().abs(), w[e].double().abs())
    th.check(da[pick], ref, th.grouped_bound(ref, mag, torch.full_like(ref, n), BF), "far operand rows")


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
def test_grouped_directional_difference(form):
    """The products are bilinear, so a central difference of <out, c> along a
    direction equals the gradient's product with it up to fp32 rounding."""
    sizes, n, k = [20, 0, 33], 48, 40
    G, a, w, off, out = grouped_inputs("forward", sizes, n, k, F32, F32, seed=5)
    c = torch.randn_like(out)
    loss = lambda a, w: float((run_grouped("forward", G, a, w, off, torch.empty_like(out)).double() * c).sum())   # noqa: E731
    if form == "forward":
        v = torch.randn_like(a)
        lhs = (loss(a + v, w) - loss(a - v, w)) / 2
        rhs = loss(v, w)
    elif form == "dgrad":
        v, da = torch.randn_like(a), torch.empty_like(a)
        run_grouped("dgrad", G, c, w, off, da)
        lhs, rhs = (loss(a + v, w) - loss(a - v, w)) / 2, float((da.double() * v).sum())
    else:
        v, dw = torch.randn_like(w), torch.empty_like(w)
        run_grouped("wgrad", G, c, a, off, dw)
        lhs, rhs = (loss(a, w + v) - loss(a, w - v)) / 2, float((dw.double() * v).sum())
    # every product is rounded at relative k 2^-24 at most; terms of size <= 10 k each
    assert abs(lhs - rhs) <= 64 * th.U24 * 50 * float(out.numel()), (lhs, rhs)


# ------------------------------------------------------------------- SwiGLU
def swiglu_inputs(R, I, dtype, live=None, slots=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    gu = rnd(R, 2 * I) * torch.exp(2 * rnd(2 * I))
    gu[:, : min(32, 2 * I)] *= 1e-3
    d = dict(gu=gu.to(dtype), dh=rnd(R, I).to(dtype), w=torch.rand(R, generator=g, device="cuda") * 3)
    d["slot"] = torch.randperm(R, generator=g, device="cuda").to(torch.int32) if slots else None
    d["off"] = None if live is None else torch.tensor([0, live // 2, live], dtype=torch.int32, device="cuda")
    d["live"] = R if live is None else live
    return d


def run_checkpoint(d, fill=3.0):
    R, C = d["gu"].shape
    h = torch.full((R, C // 2), fill, dtype=d["gu"].dtype, device="cuda")
    q = torch.full((R, C), 0x33, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale = torch.full((R, C // 32), 77, dtype=torch.uint8, device="cuda")
    ws = moe.new_status_workspace()
    moe.moe_swiglu_checkpoint(d["gu"], d["off"], d["slot"], d["w"], h, q, scale, ws)
    torch.cuda.synchronize()
    assert moe.read_device_status(ws) == 0
    return h, q, scale


def run_swiglu_backward(d, q, scale, want_h=True, want_w=True, fill=3.0):
    R, I = d["dh"].shape
    dgu = torch.full((R, 2 * I), fill, dtype=d["dh"].dtype, device="cuda")
    h = torch.full((R, I), fill, dtype=d["dh"].dtype, device="cuda") if want_h else None
    dw = torch.full((R,), fill, device="cuda") if want_w else None
    ws = moe.new_status_workspace()
    moe.moe_swiglu_backward(q, scale, d["dh"], d["off"], d["slot"], d["w"], dgu, dw, h, ws)
    torch.cuda.synchronize()
    assert moe.read_device_status(ws) == 0
    return dgu, dw, h


def row_weights(d):
    R = d["gu"].shape[0]
    if d["w"] is None:
        return torch.ones(R, dtype=torch.float64), torch.arange(R)
    slot = torch.arange(R) if d["slot"] is None else d["slot"].cpu().long()
    return d["w"].cpu().double()[slot], slot


SWIGLU = [(1, 16, None, True), (300, 640, None, True), (77, 48, 50, True), (5, 2048, 0, True),
          (129, 1040, 128, False), (1000, 64, 999, True), (33, 24576, None, False)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,I,live,slots", SWIGLU)
def test_swiglu_checkpoint(R, I, live, slots, dtype):
    d = swiglu_inputs(R, I, dtype, live, slots)
    h, q, scale = run_checkpoint(d)
    n = d["live"]
    w, _ = row_weights(d)
    gu = d["gu"].cpu().double()
    ref, g = th.swiglu_exact(gu, w)
    tol = (th.half_ulp(dtype) + th.expf_rel(g)) * ref.abs() + torch.finfo(dtype).tiny
    th.check(h[:n], ref[:n], tol[:n], "h")
    qe, be = th.quantise_exact(d["gu"])
    assert torch.equal(scale.cpu()[:n], be[:n]), "scales"
    assert torch.equal(q.double().cpu()[:n], qe[:n]), "checkpoint values"
    # rows behind the last group are left as they were
    assert bool((h[n:] == 3.0).all()) and bool((scale[n:] == 77).all())
    assert bool((q.view(torch.uint8)[n:] == 0x33).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,I,live,slots", SWIGLU)
def test_swiglu_backward(R, I, live, slots, dtype):
    d = swiglu_inputs(R, I, dtype, live, slots, seed=1)
    qe, be = th.quantise_exact(d["gu"])
    q, scale = qe.to(F32).to(torch.float8_e4m3fn).cuda(), be.cuda()
    dgu, dw, h = run_swiglu_backward(d, q, scale)
    n = d["live"]
    w, slot = row_weights(d)
    gu = th.dequantise(q, scale)
    g, u, dh = gu[:, ::2], gu[:, 1::2], d["dh"].cpu().double()
    s, wc, rel = torch.sigmoid(g), w[:, None], th.expf_rel(g)
    a = g * s
    half, tiny = th.half_ulp(dtype), torch.finfo(dtype).tiny
    dg, du, hr = wc * dh * u * s * (1 + g * (1 - s)), wc * dh * a, wc * a * u
    # 1 + g (1 - s): the errors of s and of 1 - s enter times |g|
    slack = (wc * dh * u).abs() * s * ((1 + g.abs() * (1 - s)) * 2 * rel + g.abs() * s * rel)
    th.check(dgu[:n, ::2], dg[:n], (half * dg.abs() + slack + tiny)[:n], "d gate")
    th.check(dgu[:n, 1::2], du[:n], ((half + rel) * du.abs() + tiny)[:n], "d up")
    th.check(h[:n], hr[:n], ((half + rel) * hr.abs() + tiny)[:n], "h")
    dwr = torch.zeros(R, dtype=torch.float64)
    tol = torch.full((R,), 1e-30, dtype=torch.float64)
    terms = dh * a * u
    dwr[slot[:n]] = terms.sum(1)[:n]
    tol[slot[:n]] += (terms.abs() * (rel + (I + 4) * th.U24)).sum(1)[:n]
    th.check(dw, dwr, tol, "d topk_w (0 for slots without a row)")
    assert bool((dgu[n:] == 3.0).all()) and bool((h[n:] == 3.0).all())
    # two runs agree, and leaving out the optional outputs changes nothing
    dgu2, dw2, _ = run_swiglu_backward(d, q, scale, want_h=False)
    assert torch.equal(dgu2, dgu) and torch.equal(dw2, dw)
    dgu3, _, h3 = run_swiglu_backward(d, q, scale, want_w=False)
    assert torch.equal(dgu3, dgu) and torch.equal(h3, h)


def test_swiglu_weight_of_one_and_no_row_map():
    d = swiglu_inputs(40, 64, BF, None, slots=False)
    d["w"] = None
    h, q, scale = run_checkpoint(d)
    ref, g = th.swiglu_exact(d["gu"].cpu().double(), torch.ones(40, dtype=torch.float64))
    th.check(h, ref, (th.half_ulp(BF) + th.expf_rel(g)) * ref.abs() + torch.finfo(BF).tiny, "h, weight 1")
    d2 = dict(d, w=torch.ones(40, device="cuda"))
    assert torch.equal(run_checkpoint(d2)[0], h)
    a, b = run_swiglu_backward(d, q, scale), run_swiglu_backward(d2, q, scale)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_checkpoint_of_special_values():
    """Non-finite values become NaN and leave their block's scale alone; zero
    blocks, the largest and the smallest values keep exact scales."""
    x = torch.zeros(4, 128)
    x[0, 0], x[0, 5], x[0, 7] = float("inf"), float("nan"), 3.0
    x[0, 40] = float("-inf")
    x[1, :32] = torch.finfo(F32).max
    x[1, 33], x[1, 34] = 2.0 ** -149, -(2.0 ** -140)
    x[2, 0], x[2, 32], x[2, 64], x[2, 96] = 448.0, 448.0000305, 447.99997, 2.0 ** -119 * 448
    x[3, :32] = torch.linspace(-1, 1, 32)
    for dtype in (F32, BF):
        d = dict(gu=x.to(dtype).cuda(), slot=None, w=None, off=None)
        _, q, scale = run_checkpoint(d)
        qe, be = th.quantise_exact(d["gu"])
        assert torch.equal(scale.cpu(), be)
        got = q.double().cpu()
        assert torch.equal(got.isnan(), qe.isnan()) and torch.equal(got.nan_to_num(), qe.nan_to_num())
        assert got[0].isnan().sum() == 3


def test_swiglu_bad_slots_are_recorded():
    d = swiglu_inputs(8, 32, BF)
    d["slot"][3], d["slot"][5] = 8, -1
    h, q, scale = (torch.zeros(8, 32, dtype=BF, device="cuda"),
                   torch.zeros(8, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                   torch.zeros(8, 2, dtype=torch.uint8, device="cuda"))
    ws = moe.new_status_workspace()
    moe.moe_swiglu_checkpoint(d["gu"], None, d["slot"], d["w"], h, q, scale, ws)
    with pytest.raises(moe.MoEError):
        moe.read_device_status(ws)
    assert bool((h[3] == 0).all()) and bool((h[5] == 0).all()) and bool((h[0] != 0).any())
    dgu, dw = torch.ones(8, 64, dtype=BF, device="cuda"), torch.ones(8, device="cuda")
    moe.moe_swiglu_backward(q, scale, d["dh"], None, d["slot"], d["w"], dgu, dw, None, ws)
    with pytest.raises(moe.MoEError):
        moe.read_device_status(ws)
    assert bool((dgu[3] == 0).all()) and bool((dgu[5] == 0).all())
    assert moe.read_device_status(ws) == 0


def test_swiglu_directional_difference():
    """A central difference of <h, dh> through the forward kernel at the
    checkpoint's values against the backward kernel's gradients."""
    d = swiglu_inputs(6, 32, F32, seed=4)
    d["gu"] = torch.randn(6, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    _, q, scale = run_checkpoint(d)
    gu = th.dequantise(q, scale).float().cuda()
    dgu, dw, _ = run_swiglu_backward(d, q, scale)
    loss = lambda gu, w: float((run_checkpoint(dict(d, gu=gu, w=w))[0].double() * d["dh"]).sum())   # noqa: E731
    v, t = torch.randn_like(gu), 1e-2
    lhs = (loss(gu + t * v, d["w"]) - loss(gu - t * v, d["w"])) / (2 * t)
    rhs = float((dgu.double() * v).sum())
    # third derivatives of at most ~10 a term: t^2 / 6 * 10 * 192 terms, and
    # fp32 rounding of losses of magnitude ~50 over 2 t
    assert abs(lhs - rhs) < 192 * 10 * t * t / 6 + 50 * 2.0 ** -21 / t, (lhs, rhs)
    v = torch.randn_like(d["w"])
    lhs = (loss(gu, d["w"] + v) - loss(gu, d["w"] - v)) / 2
    assert abs(lhs - float((dw.double() * v).sum())) < 192 * 50 * 2.0 ** -21, (lhs, rhs)


# -------------------------------------------------------------------- norms
NORMS = [(1, 1), (3, 7), (300, 512), (1, 64), (77, 192), (32, 6144), (1001, 8192), (33, 8256),
         (5, 2112), (64, 1001), (700, 40), (9, 16384), (3000, 1024)]


def norm_inputs(T, H, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T * 131 + H)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    x = rnd(T, H) + 3.0 * rnd(T, 1)
    if T > 2:
        x[1] = 0
        x[2] *= 1e-3
    return (x.to(dtype), (1 + 0.3 * rnd(H)).to(dtype), rnd(H).to(dtype), rnd(T, H).to(dtype),
            rnd(T, H).to(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", NORMS)
def test_layer_norm(T, H, dtype):
    eps = 1e-5
    x, w, b, _, _ = norm_inputs(T, H, dtype)
    for bias in (b, None):
        out = torch.full_like(x, 9.0)
        moe.moe_layer_norm(x, w, bias, out, eps)
        xh, r, ref = th.norm_exact(x, w, bias, eps, True)
        c, dxh = th.norm_errors(x, xh, r, H, True)
        mag = (xh * w.double()).abs() + (0 if bias is None else bias.double().abs())
        tol = th.half_ulp(dtype) * ref.abs() + w.double().abs() * dxh + 4 * th.U24 * mag + 1e-37
        th.check(out, ref, tol, f"layer norm {T} {H}")
    inplace = x.clone()
    moe.moe_layer_norm(inplace, w, None, inplace, eps)
    assert torch.equal(inplace, out)


def norm_backward(layer, x, w, do, eps, dres=None, dx=None, bias=True):
    T, H = x.shape
    dx = torch.full_like(x, 9.0) if dx is None else dx
    dw, db = torch.full((H,), 9.0, device="cuda"), torch.full((H,), 9.0, device="cuda")
    ws = moe.new_norm_workspace(T, H)
    ws.fill_(0xFF)                                       # NaN partials: each must be written first
    if layer:
        moe.moe_layer_norm_backward(x, w, do, dx, dw, db if bias else None, ws, eps, dres=dres)
    else:
        moe.moe_rmsnorm_backward(x, w, do, dx, dw, ws, eps, dres=dres)
    torch.cuda.synchronize()
    return dx, dw, db


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("T,H", NORMS)
def test_norm_backward(T, H, layer, dtype):
    eps = 1e-5
    x, w, _, do, dres = norm_inputs(T, H, dtype, seed=7)
    xh, r, _ = th.norm_exact(x, w, None, eps, layer)
    c, dxh = th.norm_errors(x, xh, r, H, layer)
    dod = do.double()
    gy = dod * w.double()
    mean = lambda v: v.mean(1, keepdim=True)   # noqa: E731
    m1, m2 = (mean(gy) if layer else 0 * r), mean(gy * xh)
    ref0 = r * (gy - m1 - xh * m2)
    dm2 = c * mean((gy * xh).abs()) + mean(gy.abs() * dxh)
    err = r * (c * gy.abs() + c * mean(gy.abs()) + xh.abs() * dm2 + dxh * m2.abs() + c * (xh * m2).abs()) + \
        c * ref0.abs()
    chain = T / 148 + 592 + 32
    dw_ref, db_ref = (dod * xh).sum(0), dod.sum(0)
    dw_tol = (dod.abs() * dxh).sum(0) + chain * th.U24 * (dod * xh).abs().sum(0) + 1e-30
    db_tol = chain * th.U24 * dod.abs().sum(0) + 1e-30
    for res in (None, dres):
        ref = ref0 if res is None else ref0 + res.double()
        tol = th.half_ulp(dtype) * ref.abs() + err + 2 * th.U24 * ref.abs() + 1e-37
        dx, dw, db = norm_backward(layer, x, w, do, eps, res)
        th.check(dx, ref, tol, f"dx {T} {H}")
        th.check(dw, dw_ref, dw_tol, "dweight")
        if layer:
            th.check(db, db_ref, db_tol, "dbias")
    # the same bits again, in place over dout and over dres, and without dbias
    d1 = norm_backward(layer, x, w, do.clone(), eps, dres)
    c1 = do.clone()
    d2 = norm_backward(layer, x, w, c1, eps, dres, dx=c1, bias=False)
    c2 = dres.clone()
    d3 = norm_backward(layer, x, w, do, eps, c2, dx=c2)
    for d in (d1, d2, d3):
        assert torch.equal(d[0], dx) and torch.equal(d[1], dw)


def test_norm_backward_of_no_rows():
    for layer in (True, False):
        x = torch.zeros(0, 64, dtype=BF, device="cuda")
        _, dw, db = norm_backward(layer, x, torch.ones(64, dtype=BF, device="cuda"), x, 1e-6)
        assert bool((dw == 0).all()) and (not layer or bool((db == 0).all()))


@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
def test_norm_directional_difference(layer):
    T, H, eps = 4, 96, 1e-5
    x, w, b, do, _ = norm_inputs(T, H, F32, seed=3)
    x = torch.randn_like(x)

    def loss(x, w):
        out = torch.empty_like(x)
        moe.moe_layer_norm(x, w, b, out, eps) if layer else moe.moe_rmsnorm(x, w, out, eps)
        return float((out.double() * do).sum())
    if not layer:
        x, w, do = (torch.cat([t, t[..., :32]], -1).contiguous() for t in (x, w, do))   # H % 64 == 0
    dx, dw, _ = norm_backward(layer, x, w, do, eps)
    t = 1e-2
    v = torch.randn_like(x)
    lhs = (loss(x + t * v, w) - loss(x - t * v, w)) / (2 * t)
    # third derivatives of a few units a term; fp32 rounding of a loss of ~100
    assert abs(lhs - float((dx.double() * v).sum())) < 512 * 10 * t * t / 6 + 100 * 2.0 ** -21 / t
    v = torch.randn_like(w)
    lhs = (loss(x, w + v) - loss(x, w - v)) / 2
    assert abs(lhs - float((dw.double() * v).sum())) < 512 * 20 * 2.0 ** -21


# ------------------------------------------- streams, graphs, the step together
def test_operators_on_a_side_stream_and_in_a_graph():
    """Every operator captured once and replayed on new inputs gives what a
    direct call on another stream gives."""
    sizes, n, k = [70, 0, 61, 5], 128, 192
    R, E, I = sum(sizes) + 4, len(sizes), n // 2
    G = moe.GroupedMatmul(R, E, n, k, BF, BF)
    GW = moe.GroupedMatmul(R, E, n, k, BF, F32)
    off = torch.tensor([0, 70, 70, 131, 136], dtype=torch.int32, device="cuda")
    mk = lambda *s: torch.randn(*s, device="cuda").to(BF)   # noqa: E731
    st = dict(x=mk(R, k), w=mk(E, n, k), nw=mk(k), dh=mk(R, I), tw=torch.rand(R, device="cuda"))
    ws, nws = moe.new_grouped_workspace(G), moe.new_norm_workspace(R, k)
    z = lambda t, *s: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    o = dict(xn=z(BF, R, k), gu=z(BF, R, n), h=z(BF, R, I), q=z(torch.uint8, R, n).view(torch.float8_e4m3fn),
             sc=z(torch.uint8, R, n // 32), dgu=z(BF, R, n), dtw=z(F32, R), h2=z(BF, R, I),
             dx=z(BF, R, k), dw=z(F32, E, n, k), dxn=z(BF, R, k), dnw=z(F32, k), dnb=z(F32, k),
             dx2=z(BF, R, k), dnw2=z(F32, k))

    def step(s, o, ws, nws, stream=None):
        kw = dict(stream=stream)
        moe.moe_layer_norm(s["x"], s["nw"], None, o["xn"], **kw)
        moe.moe_grouped_matmul(G, o["xn"], s["w"], off, o["gu"], ws, **kw)
        moe.moe_swiglu_checkpoint(o["gu"], off, None, s["tw"], o["h"], o["q"], o["sc"], ws, **kw)
        moe.moe_swiglu_backward(o["q"], o["sc"], s["dh"], off, None, s["tw"], o["dgu"], o["dtw"], o["h2"], ws, **kw)
        moe.moe_grouped_matmul_dgrad(G, o["dgu"], s["w"], off, o["dx"], ws, **kw)
        moe.moe_grouped_matmul_wgrad(GW, o["dgu"], o["xn"], off, o["dw"], ws, **kw)
        moe.moe_layer_norm_backward(s["x"], s["nw"], o["dx"], o["dxn"], o["dnw"], o["dnb"], nws, **kw)
        moe.moe_rmsnorm_backward(s["x"], s["nw"], o["dx"], o["dx2"], o["dnw2"], nws, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(st, o, ws, nws)                 # warm-up
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(st, o, ws, nws)
    for seed in (1, 2):
        torch.manual_seed(seed)
        for t in st.values():
            t.copy_(torch.randn(t.shape, device="cuda").abs() if t.dtype == F32 else torch.randn(t.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert moe.read_device_status(ws) == 0
        o2 = {a: torch.zeros_like(b) for a, b in o.items()}
        ws2, nws2 = moe.new_grouped_workspace(G), moe.new_norm_workspace(R, k)
        torch.cuda.synchronize()
        step(st, o2, ws2, nws2, stream=side)
        side.synchronize()
        for a in o:
            assert torch.equal(o[a].view(torch.uint8), o2[a].view(torch.uint8)), a
            assert bool((o2[a].float() != 0).any()), a


def test_two_calls_at_once_on_two_streams():
    """Calls with workspaces of their own run side by side and agree with
    calls one after the other."""
    ins = [grouped_inputs(f, [300, 0, 500, 40], 512, 384, BF, BF, seed=i)
           for i, f in enumerate(["forward", "dgrad"])]
    want = [run_grouped(f, *i[:4], torch.zeros_like(i[4])) for f, i in zip(["forward", "dgrad"], ins)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.zeros_like(i[4]) for i in ins]
    wss = [moe.new_grouped_workspace(i[0]) for i in ins]
    torch.cuda.synchronize()
    for _ in range(20):
        for f, i, o, w, s in zip(["forward", "dgrad"], ins, outs, wss, streams):
            getattr(moe, CALL[f])(*i[:4], o, w, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_training_step_of_the_expert_block(dtype):
    """The operators together: norm, route, permute, grouped products around
    the checkpointed SwiGLU, combine, and all gradients back to the block's
    input, the norm's weight, the expert weights and the routing weights,
    against fp64 with the checkpoint's values in the backward pass."""
    T, H, E, k, I, eps = 150, 192, 6, 2, 128, 1e-6
    L = moe.Layer(T, H, E, k, 0, I, dtype, 2.5)
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    x, nw, dout = rnd(T, H).to(dtype), (1 + 0.1 * rnd(H)).to(dtype), rnd(T, H).to(dtype)
    wr, cb = rnd(E, H) * 0.1, rnd(E) * 0.01
    wgu, wd = (rnd(E, 2 * I, H) * 0.08).to(dtype), (rnd(E, H, I) * 0.08).to(dtype)
    pad = torch.zeros(T, dtype=torch.uint8, device="cuda")
    pad[::17] = 1
    z = lambda t, *s: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    i32 = torch.int32
    R = T * k
    ws, nws = moe.new_workspace(L), moe.new_norm_workspace(T, H)
    xn, tw, ti = z(dtype, T, H), z(F32, T, k), z(i32, T, k)
    off, slot, inv, xp = z(i32, E + 1), z(i32, R), z(i32, R), z(dtype, R, H)
    moe.moe_rmsnorm(x, nw, xn, eps)
    moe.moe_route(L, xn, wr, cb, tw, ti, None, ws)
    moe.moe_permute(L, ti, pad, xn, off, slot, inv, xp, ws)
    GU = moe.GroupedMatmul(R, E, 2 * I, H, dtype)
    GU32 = moe.GroupedMatmul(R, E, 2 * I, H, dtype, F32)
    DN32 = moe.GroupedMatmul(R, E, H, I, dtype, F32)
    DN = moe.GroupedMatmul(R, E, H, I, dtype)
    gu, h, q, sc = z(dtype, R, 2 * I), z(dtype, R, I), z(torch.uint8, R, 2 * I).view(torch.float8_e4m3fn), z(torch.uint8, R, I // 16)
    y, out = z(F32, R, H), z(dtype, T, H)
    moe.moe_grouped_matmul(GU, xp, wgu, off, gu, ws)
    moe.moe_swiglu_checkpoint(gu, off, slot, tw, h, q, sc, ws)
    moe.moe_grouped_matmul(DN32, h, wd, off, y, ws)
    moe.moe_combine(L, y, None, inv, out, ws)
    # backward
    dy = z(dtype, R, H)
    moe.moe_permute(L, ti, pad, dout, off, slot, inv, dy, ws)
    dh, dgu, dtw, h2 = z(dtype, R, I), z(dtype, R, 2 * I), z(F32, T, k), z(dtype, R, I)
    dwd, dwgu = z(F32, E, H, I), z(F32, E, 2 * I, H)
    moe.moe_grouped_matmul_dgrad(DN, dy, wd, off, dh, ws)
    moe.moe_swiglu_backward(q, sc, dh, off, slot, tw, dgu, dtw, h2, ws)
    moe.moe_grouped_matmul_wgrad(DN32, dy, h2, off, dwd, ws)
    dxp, dxn = z(F32, R, H), z(dtype, T, H)
    moe.moe_grouped_matmul_dgrad(GU32, dgu, wgu, off, dxp, ws)
    moe.moe_grouped_matmul_wgrad(GU32, dgu, xp, off, dwgu, ws, accumulate=True)
    moe.moe_combine(L, dxp, None, inv, dxn, ws)
    dx, dnw = z(dtype, T, H), z(F32, H)
    moe.moe_rmsnorm_backward(x, nw, dxn, dx, dnw, nws, eps, dres=dout)
    torch.cuda.synchronize()
    assert moe.read_device_status(ws) == 0

    # fp64: the same routing, gate_up's values in the backward from the checkpoint
    D = torch.float64
    xhat, r, xn64 = th.norm_exact(x, nw, None, eps, False)
    tw64, live = tw.to(D), pad == 0
    W1, W2 = wgu.to(D), wd.to(D)
    ref = {n: torch.zeros(s, dtype=D, device="cuda") for n, s in
           dict(out=(T, H), dxn=(T, H), dtw=(T, k), dwd=(E, H, I), dwgu=(E, 2 * I, H)).items()}
    row_of = inv.reshape(T, k).long()
    ckpt = th.dequantise(q, sc).cuda()
    for e in range(E):
        for j in range(k):
            t = torch.nonzero(live & (ti[:, j] == e)).reshape(-1)
            if t.numel() == 0:
                continue
            w = tw64[t, j][:, None]
            v = xn64[t] @ W1[e].t()
            ref["out"][t] += (w * v[:, ::2] * torch.sigmoid(v[:, ::2]) * v[:, 1::2]) @ W2[e].t()
            c = ckpt[row_of[t, j]]
            gg, u, s = c[:, ::2], c[:, 1::2], torch.sigmoid(c[:, ::2])
            dy64 = dout.to(D)[t]
            dh64 = dy64 @ W2[e]
            ref["dwd"][e] += dy64.t() @ (w * gg * s * u)
            ref["dtw"][t, j] = (dh64 * gg * s * u).sum(1)
            d = torch.zeros_like(c)
            d[:, ::2], d[:, 1::2] = w * dh64 * u * s * (1 + gg * (1 - s)), w * dh64 * gg * s
            ref["dwgu"][e] += d.t() @ xn64[t]
            ref["dxn"][t] += d @ W1[e]
    gy = ref["dxn"] * nw.to(D)
    ref["dx"] = r * (gy - xhat * (gy * xhat).mean(1, keepdim=True)) + dout.to(D)
    ref["dnw"] = (ref["dxn"] * xhat).sum(0)
    got = dict(out=out, dxn=dxn, dtw=dtw, dwd=dwd, dwgu=dwgu, dx=dx, dnw=dnw)
    # at most 6 roundings to dtype lie between the inputs and any output (xn,
    # gu, h | xn, dh, dgu, dxn, dx); each changes a 2-norm by at most half a
    # step, products pass them on with a factor of about one (2 allowed), and
    # fp32 sums add 1e-5
    bound = 12 * th.half_ulp(dtype) + 1e-5
    for name, a in got.items():
        rel = float((a.to(D) - ref[name]).norm() / ref[name].norm())
        assert rel < bound, (name, rel, bound)
    assert bool((dtw[pad != 0] == 0).all()) and torch.equal(dx[pad != 0], dout[pad != 0])
