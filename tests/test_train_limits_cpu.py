"""Host checks of the training operators' limits: sizes that the kernels' index
arithmetic could not hold are refused before any CUDA call (fake aligned
pointers are never touched)."""
from __future__ import annotations

import ctypes

import pytest

import mixture_experts_feed_b200 as moe

FAKE, BIG = 1 << 20, 1 << 40
UNSUPPORTED = 2
LIMIT = 1 << 24


@pytest.mark.parametrize("dtype", [0, 1, 2], ids=["f32", "bf16", "f16"])
def test_grouped_features_past_the_limit_are_refused(dtype):
    """1024 groups of one row, n = 2^25: 2^31 tiles of 1 x 16 on the CUDA cores,
    one more than 32 bits count."""
    ok = [FAKE] * 4
    for n, k in ((1 << 25, 1), (1, 1 << 25), (LIMIT + 1, 8), (8, LIMIT + 8)):
        d = ctypes.byref(moe.GroupedDesc(1024, 1024, n, k, dtype, dtype))
        assert moe.LIB.moe_grouped_matmul(d, *ok, FAKE, BIG, None) == UNSUPPORTED
        assert moe.LIB.moe_grouped_matmul_dgrad(d, *ok, FAKE, BIG, None) == UNSUPPORTED
        assert moe.LIB.moe_grouped_matmul_wgrad(d, *ok, 0, FAKE, BIG, None) == UNSUPPORTED
        assert moe.LIB.moe_grouped_workspace_size(d, ctypes.byref(ctypes.c_size_t(0))) == UNSUPPORTED
    for n, k in ((LIMIT, 1), (1, LIMIT), (LIMIT, LIMIT)):
        d = ctypes.byref(moe.GroupedDesc(1024, 1024, n, k, dtype, dtype))
        assert moe.LIB.moe_grouped_workspace_size(d, ctypes.byref(ctypes.c_size_t(0))) == 0
