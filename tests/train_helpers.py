"""Plain fp64 forms of the training operators and the error bounds their
tests use.

Bounds count roundings: one rounding to dtype t changes a value by at most
eps(t)/2 of its magnitude; an fp32 sum of n terms in any order differs from
the exact sum by at most n * 2^-24 * sum|terms| (2^-23 where an accumulator
truncates instead of rounding).
"""
from __future__ import annotations

import torch

U24 = 2.0 ** -24
BLOCK = 32


def half_ulp(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


def check(got, ref, tol, what):
    """|got - ref| <= tol elementwise; nothing else may be non-finite."""
    got = got.double().cpu()
    ref, tol = ref.cpu(), tol.cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {got.numel()} outside the bound, first at {i}: got "
            f"{got.reshape(-1)[i]:.9g}, exact {ref.reshape(-1)[i]:.9g}, bound {tol.reshape(-1)[i]:.3g}")


# ---------------------------------------------------------- grouped products
def grouped_exact(form, p, q, offsets, out0, accumulate=False):
    """(exact output, sum of |products|, length of the sum) in fp64, over the
    rows / experts the operator writes; the rest as out0 holds it."""
    out = out0.double().clone()
    mag = torch.zeros_like(out)
    n_sum = torch.zeros_like(out)
    off = offsets.tolist()
    for e in range(len(off) - 1):
        lo, hi = off[e], off[e + 1]
        pe = p[lo:hi].double()
        if form == "wgrad":
            qe = q[lo:hi].double()
            d, m = pe.t() @ qe, pe.abs().t() @ qe.abs()
            if accumulate:
                m = m + out[e].abs() if hi > lo else torch.zeros_like(m)
                d = out[e] + d
            out[e], mag[e], n_sum[e] = d, m, float(hi - lo)
        elif hi > lo:
            qe = q[e].double()
            qe = qe.t() if form == "forward" else qe
            out[lo:hi], mag[lo:hi], n_sum[lo:hi] = pe @ qe, pe.abs() @ qe.abs(), float(pe.shape[1])
    return out, mag, n_sum


def grouped_bound(out, mag, n_sum, out_dtype):
    # products of two 16-bit values are exact in fp32 (fp32 operands: one
    # rounding each, inside the + 2); tensor-core accumulators truncate
    return half_ulp(out_dtype) * out.abs() + (n_sum + 2) * 2 * U24 * mag + torch.finfo(out_dtype).tiny


# ------------------------------------------------------------------- SwiGLU
def quantise_exact(x):
    """e4m3 values (fp64) and scale bytes of blocks of 32 columns, straight
    from the definition: the least byte whose scale holds the block."""
    R, C = x.shape
    v = x.double().cpu().reshape(R, C // BLOCK, BLOCK)
    fine = torch.isfinite(v)
    amax = torch.where(fine, v.abs(), torch.zeros_like(v)).amax(-1)
    grid = torch.exp2(torch.arange(0, 255, dtype=torch.float64) - 127) * 448.0
    byte = torch.searchsorted(grid, amax.contiguous())          # least b with amax <= grid[b]
    y = v / torch.exp2(byte.double() - 127)[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    q = torch.where(fine, torch.round(y / step) * step, torch.full_like(y, float("nan")))
    return q.reshape(R, C), byte.to(torch.uint8)


def dequantise(q, scale):
    R, C = q.shape
    s = torch.exp2(scale.double().cpu() - 127)[..., None]
    return (q.double().cpu().reshape(R, C // BLOCK, BLOCK) * s).reshape(R, C)


def swiglu_exact(gu, w):
    """h and its bound's scale (relative fp32 error of the expression)."""
    g, u = gu[:, ::2], gu[:, 1::2]
    h = w[:, None] * g * torch.sigmoid(g) * u
    return h, g


def expf_rel(g):
    """Relative fp32 error of silu(g) and of 1 / (1 + e^-g): __expf is within
    2 + 1.173 |x| ulp, the sum, the division (2 ulp) and products add to it."""
    return (12 + 1.2 * g.abs()) * 2.0 ** -23


# -------------------------------------------------------------------- norms
def norm_exact(x, weight, bias, eps, layer):
    """x^, r, out of the norm in fp64."""
    x, w = x.double(), weight.double()
    mean = x.mean(1, keepdim=True) if layer else torch.zeros(x.shape[0], 1, dtype=torch.float64, device=x.device)
    xc = x - mean
    r = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + eps)
    xh = xc * r
    out = xh * w
    if bias is not None:
        out = out + bias.double()
    return xh, r, out


def norm_errors(x, xh, r, H, layer):
    """(c, bound on x^'s fp32 error): row sums of H terms run in chains of at
    most H/32 + 32 additions."""
    c = (H / 32 + 32 + 16) * U24
    mx = x.double().abs().mean(1, keepdim=True) if layer else torch.zeros_like(r)
    return c, c * (r * (mx + x.double().abs() * layer) + xh.abs())
