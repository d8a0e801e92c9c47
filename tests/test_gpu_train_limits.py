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
