"""Sizes at the edge of what the group norm's kernels count in an int, without a GPU:
refused where a step beyond the last row would not fit."""
import ctypes

import pytest
import torch

import gated_delta_rule_157_b200 as kda
from test_packed_abi import UNSUPPORTED, norm_args

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers are only used without a GPU")
MOST = 0x7FFFFFFF - (1 << 26)
F32, BF16 = 0, 1
TOO_LARGE = [
    dict(N=0x7FFFFFFF, L=1, C=1, G=1), dict(N=MOST + 1, L=1, C=1, G=1), dict(N=1, L=0x7FFFFFFF, C=1, G=1),
    dict(N=3, L=MOST // 3 + 1, C=1, G=1), dict(N=1, L=1, C=0x7FFFFFFF, G=1), dict(N=1, L=1 << 16, C=1 << 15, G=1),
    dict(N=1, L=1, C=MOST, G=MOST), dict(N=2, L=4096, C=65536 * 256 * 8, G=1 << 16),
    dict(N=1, L=600, C=(1 << 30) + (1 << 10), G=1 << 10),
]


@no_gpu_only
@pytest.mark.parametrize("kw", TOO_LARGE)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sizes_beyond_an_int_are_refused(kw, dtype):
    lib = kda.load()
    for fn, backward in ((lib.kda_group_norm_fwd, 0), (lib.kda_group_norm_bwd, 1)):
        assert fn(ctypes.byref(norm_args(dtype=dtype, **kw)), None) == UNSUPPORTED
        assert lib.kda_group_norm_workspace(kw["N"], kw["L"], kw["C"], kw["G"], dtype, backward) == 0


@no_gpu_only
@pytest.mark.parametrize("kw", [dict(N=MOST - 2, L=1, C=1, G=1), dict(N=1, L=MOST, C=1, G=1), dict(N=1, L=1, C=4096, G=1)])
def test_the_largest_sizes_are_not(kw):
    lib = kda.load()
    for fn in (lib.kda_group_norm_fwd, lib.kda_group_norm_bwd):
        assert fn(ctypes.byref(norm_args(**kw)), None) != UNSUPPORTED      # (the made-up pointers overlap)


def test_workspace_stays_below_the_data():
    """A bounded share of x: 2 C floats per block of rows."""
    ws = kda.load().kda_group_norm_workspace
    for N, L, C, G in ((1, MOST, 1, 1), (1, 1 << 24, 64, 4), (200000, 1, 4096, 32), (256, 4096, 1280, 32)):
        for backward in (0, 1):
            assert ws(N, L, C, G, BF16, backward) <= max(1 << 23, N * L * C * 2 // 4)
