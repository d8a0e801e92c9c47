"""GPU tests of the training operators where their results could be lost or
unsafe: rows of neighbours beside ragged groups, precision over long sums,
and index arrays that are out of range."""
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
@pytest.mark.parametrize("out,accumulate", [(BF, False), (F32, True)], ids=["bf16", "f32-accumulate"])
def test_wgrad_rows_of_neighbours_never_enter(out, accumulate):
    """Every group ends inside a block of 64 rows, and every other group is all
    NaN: the rows that a group's last block brings along beyond its own are
    zeroed in both CTAs of a pair before its products run.  Over many pairs and
    calls the finite groups stay finite and the same."""
    E, n, k = 148, 512, 256
    g = torch.Generator().manual_seed(5)
    sizes = (1 + torch.randint(0, 150, (E,), generator=g)).tolist()
    sizes = [s + 1 if s % 16 == 0 else s for s in sizes]
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    R = int(off[-1])
    gd = torch.Generator(device="cuda").manual_seed(6)
    p = torch.randn(R, n, generator=gd, device="cuda").to(BF)
    q = torch.randn(R, k, generator=gd, device="cuda").to(BF)
    for e in range(1, E, 2):
        p[off[e]:off[e + 1]] = float("nan")
        q[off[e]:off[e + 1]] = float("nan")
    G = moe.GroupedMatmul(R, E, n, k, BF, out)
    ws = moe.new_grouped_workspace(G)
    o0 = torch.randn(E, n, k, generator=gd, device="cuda").to(out)
    kw = dict(accumulate=True) if accumulate else {}
    ref, mag, m = th.grouped_exact("wgrad", p.nan_to_num(0), q.nan_to_num(0), off, o0, accumulate)
    first = None
    for _ in range(30):
        o = o0.clone()
        moe.moe_grouped_matmul_wgrad(G, p, q, off, o, ws, **kw)
        assert bool(torch.isnan(o[1::2]).all()) and bool(torch.isfinite(o[::2]).all())
        first = o if first is None else first
        assert torch.equal(o[::2], first[::2])
    th.check(first[::2], ref[::2], th.grouped_bound(ref, mag, m, out)[::2], "finite groups")
    assert moe.read_device_status(ws) == 0


def product(form, sizes, n, k, dtype, out, cut, values=torch.randn, accumulate=False, old=0.0, seed=1):
    """(output, exact output) of a product.  `cut`: None for sizes that are never
    cut along the sum; else the workspace holds the pieces (True) or does not."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, R = len(sizes), sum(sizes)
    mk = lambda *s: values(*s, generator=g, device="cuda")   # noqa: E731
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    p = mk(R, k if form == "forward" else n).to(dtype)
    q = (mk(R, k) if form == "wgrad" else mk(E, n, k)).to(dtype)
    o = mk(*((E, n, k) if form == "wgrad" else (R, n if form == "forward" else k))).to(out) * old
    G = moe.GroupedMatmul(R, E, n, k, dtype, out)
    full = moe.grouped_workspace_size(G)
    assert (full > 256) == (cut is not None)
    ws = moe.new_grouped_workspace(G)[:full if cut else 256]
    ref = th.grouped_exact(form, p, q, off, o, accumulate)[0]
    getattr(moe, CALL[form])(G, p, q, off, o, ws, **(dict(accumulate=True) if accumulate else {}))
    torch.cuda.synchronize()
    assert moe.read_device_status(ws) == 0
    return o, ref


LONG = [("forward", [300, 100], 256, 6144, True), ("forward", [300, 100], 256, 6144, False),
        ("forward", [300, 100, 200, 50], 4096, 6144, None),
        ("dgrad", [300, 100], 6144, 256, True), ("dgrad", [300, 100], 6144, 256, False),
        ("wgrad", [9000, 500], 256, 264, True), ("wgrad", [9000, 500], 256, 264, False),
        ("wgrad", [9000, 0], 2048, 2048, None)]


@pytest.mark.parametrize("form,sizes,n,k,cut", LONG)
def test_long_sums_in_fp32_are_added_in_short_chains(form, sizes, n, k, cut):
    """A tensor-core accumulator truncates at each step of 16 terms: by half a
    unit of 2^-23 on average, 32 times in a chain of 512 terms, so at most
    16 x 2^-23 of the result's 2-norm if all of them added up (chains are
    joined by additions that round).  One chain of 6144 terms is past 6e-6."""
    o, ref = product(form, sizes, n, k, BF, F32, cut)
    rel = float((o.double() - ref).norm() / ref.norm())
    assert rel < 16 * 2.0 ** -23, rel


@pytest.mark.parametrize("form,rows,n,k,cut", [
    ("wgrad", 65536, 2048, 2048, None), ("wgrad", 65536, 512, 512, True), ("wgrad", 65536, 512, 512, False),
    ("forward", 512, 256, 32768, True), ("forward", 512, 256, 32768, False), ("dgrad", 5120, 65536, 2048, None)])
@pytest.mark.parametrize("dtype", [HF, BF], ids=["f16", "bf16"])
def test_long_sums_of_one_sign_in_16_bits_are_not_biased(form, rows, n, k, cut, dtype):
    """Rounding to nearest errs to both sides, half a step at most; truncated
    sums of one sign lean toward zero together.  They may add a sixteenth of
    that half step (one chain of 65536 terms adds a whole one in fp16)."""
    values = lambda *s, **kw: 0.25 + 0.75 * torch.rand(*s, **kw)   # noqa: E731
    o, ref = product(form, [rows], n, k, dtype, dtype, cut, values)
    bias = float(((o.double() - ref) / ref).mean())
    assert abs(bias) < th.half_ulp(dtype) / 16, bias


@pytest.mark.parametrize("cut", [True, False], ids=["cut", "uncut"])
@pytest.mark.parametrize("sizes,n,k", [([20000], 256, 264), ([0, 18000, 700], 512, 512)])
def test_large_old_weight_gradients_are_rounded_once(sizes, n, k, cut):
    """An old weight gradient a thousand times the product: the sum is rounded
    once, by half a unit of 2^-23 at most, and the product's own error (16 x
    2^-23, above) is a thousandth of that size."""
    old = 1e3 * max(sizes) ** 0.5
    o, ref = product("wgrad", sizes, n, k, BF, F32, cut, accumulate=True, old=old)
    rel = float((o.double() - ref).norm() / ref.norm())
    assert rel < 2.0 ** -24 * 1.05, rel


# ------------------------------------------------------------------- SwiGLU
@pytest.mark.parametrize("last", [-1, -(1 << 31), 41, (1 << 31) - 1])
def test_swiglu_live_rows_out_of_range_are_recorded(last):
    """The last offset says how many rows are live: outside [0, R] it is recorded
    and read as 0 or R, by both passes."""
    R, I = 40, 32
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)   # noqa: E731
    gu, dh, w = rnd(R, 2 * I), rnd(R, I), torch.rand(R, generator=g, device="cuda")
    ws = moe.new_status_workspace()

    def both(off):
        h, q = torch.full_like(dh, 3.0), torch.full((R, 2 * I), 0x33, dtype=torch.uint8, device="cuda")
        scale = torch.full((R, I // 16), 77, dtype=torch.uint8, device="cuda")
        dgu, h2, dw = torch.full_like(gu, 3.0), torch.full_like(dh, 3.0), torch.full((R,), 3.0, device="cuda")
        q8 = q.view(torch.float8_e4m3fn)
        outs, bad = [h, q, scale], []
        for call in (lambda: moe.moe_swiglu_checkpoint(gu, off, None, w, h, q8, scale, ws),
                     lambda: moe.moe_swiglu_backward(q8, scale, dh, off, None, w, dgu, dw, h2, ws)):
            call()
            try:
                moe.read_device_status(ws)
                bad.append(False)
            except moe.MoEError:
                bad.append(True)
        return outs + [dgu, dw, h2], bad

    offsets = lambda n: torch.tensor([0, 7, n], dtype=torch.int32, device="cuda")   # noqa: E731
    want, bad = both(offsets(0 if last < 0 else R))
    assert bad == [False, False]
    got, bad = both(offsets(last))
    assert bad == [True, True]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    if last < 0:
        assert bool((got[0] == 3.0).all()) and bool((got[4] == 0).all())


@pytest.mark.parametrize("R,I", [(300, 640), (33, 4096), (1000, 64)])
def test_swiglu_fp32_rows_keep_fp32_precision(R, I):
    """fp32 rows, gates out to where e^-g leaves the fp32 range.  In units of 2^-24
    (half a step): t = e^-|g| is 4 off (expf's 2 ulp), which t / (1 + t) and
    1 / (1 + t) pass on at most whole; 1 + t adds 1, its reciprocal 4 (2 ulp), the
    product with t 1: the sigmoid and its complement are 10 off, a 11, h 13 after
    the weight and u, du 13, a term of d topk_w 13 before the sum.  dg: w dh, u,
    1 + g (1 - s) and the outer products add 5 to s and to g (1 - s), 25 of the
    terms' magnitudes."""
    U, tiny = th.U24, torch.finfo(F32).tiny
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    gu, dh, w = rnd(R, 2 * I), rnd(R, I), torch.rand(R, generator=g, device="cuda") + 0.5
    gu[:, ::2] *= 40.0
    gu[0, 0], gu[0, 2], gu[0, 4], gu[0, 6] = -88.0, -87.99999, -104.0, 120.0
    h, q = torch.empty_like(dh), torch.empty(R, 2 * I, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale, ws = torch.empty(R, I // 16, dtype=torch.uint8, device="cuda"), moe.new_status_workspace()
    moe.moe_swiglu_checkpoint(gu, None, None, w, h, q, scale, ws)
    wc = w.double().cpu()[:, None]
    ref, _ = th.swiglu_exact(gu.double().cpu(), w.double().cpu())
    th.check(h, ref, 13.01 * U * ref.abs() + tiny, "h")
    dgu, dw, h2 = torch.empty_like(gu), torch.empty(R, device="cuda"), torch.empty_like(dh)
    moe.moe_swiglu_backward(q, scale, dh, None, None, w, dgu, dw, h2, ws)
    v, d = th.dequantise(q, scale), dh.double().cpu()
    ga, u = v[:, ::2], v[:, 1::2]
    s, c = torch.sigmoid(ga), torch.sigmoid(-ga)
    du, hr, terms = wc * d * ga * s, wc * ga * s * u, d * ga * s * u
    th.check(dgu[:, 1::2], du, 13.01 * U * du.abs() + tiny, "d up")
    th.check(h2, hr, 13.01 * U * hr.abs() + tiny, "h again")
    th.check(dgu[:, ::2], wc * d * u * s * (1 + ga * c), 25.01 * U * (wc * d * u).abs() * s * (1 + ga.abs() * c) + tiny,
             "d gate")
    th.check(dw, terms.sum(1), (13 + I) * U * terms.abs().sum(1) + tiny, "d topk_w")
    assert moe.read_device_status(ws) == 0


# -------------------------------------------------------------------- norms
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(9, 64), (301, 256), (300, 1024), (20, 6144), (7, 8192), (5, 1001), (3, 16384)])
def test_rmsnorm_backward_of_rows_past_the_fp32_squares(T, H, dtype):
    """Rows of 1e20 to 1e37, whose squares pass the fp32 range, between ordinary
    ones: moe_rmsnorm, which sums in fp64, gives them finite results, so they
    have gradients like any other row's.  Bounds as of ordinary rows."""
    eps = 1e-5
    g = torch.Generator(device="cuda").manual_seed(T + H)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    x = rnd(T, H)
    for i, scale in enumerate((1e20, 1e28, 1e37)):
        x[i::7] *= scale
    x, w, do, dres = x.to(dtype), (1 + 0.3 * rnd(H)).to(dtype), rnd(T, H).to(dtype), rnd(T, H).to(dtype)
    xh, r, _ = th.norm_exact(x, w, None, eps, False)
    c, dxh = th.norm_errors(x, xh, r, H, False)
    dod, mean = do.double(), lambda v: v.mean(1, keepdim=True)   # noqa: E731
    gy = dod * w.double()
    m2 = mean(gy * xh)
    ref0 = r * (gy - xh * m2)
    err = r * (c * gy.abs() + xh.abs() * (c * mean((gy * xh).abs()) + mean(gy.abs() * dxh)) + dxh * m2.abs() +
               c * (xh * m2).abs()) + c * ref0.abs()
    dw_ref = (dod * xh).sum(0)
    dw_tol = (dod.abs() * dxh).sum(0) + (T / 148 + 592 + 32) * th.U24 * (dod * xh).abs().sum(0) + 1e-30
    ws = moe.new_norm_workspace(T, H)
    for res in (None, dres):
        dx, dw = torch.full_like(x, 9.0), torch.empty(H, device="cuda")
        moe.moe_rmsnorm_backward(x, w, do, dx, dw, ws, eps, dres=res)
        ref = ref0 if res is None else ref0 + res.double()
        # results of the largest rows reach the subnormals: their step, a few times
        small = 2.0 ** (-133 if dtype == BF else -149) * 4
        th.check(dx, ref, (th.half_ulp(dtype) + 2 * th.U24) * ref.abs() + err + small, f"dx {T} {H}")
        th.check(dw, dw_ref, dw_tol, "dweight")
