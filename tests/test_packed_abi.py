"""Refusals of the packed and group-norm entry points, without a GPU: the
library's own checks on made-up pointers (skipped where a device exists, so that
a hole in them can never send such a pointer to a kernel) and the binding's."""
import ctypes

import pytest
import torch

import gated_delta_rule_157_b200 as kda
from gated_delta_rule_157_b200 import _lib

OK, INVALID, UNSUPPORTED, ALIGN, ALIAS, CUDA = 0, 1, 2, 3, 4, 5
no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers are only used without a GPU")
BASE = 0x7f3000000000
MB = 1 << 20


def _fill(a, names, **kw):
    for i, n in enumerate(names):
        setattr(a, n, BASE + (i + 1) * 16 * MB)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def packed_args(**kw):
    a = _lib.PackedArgs()
    a.N, a.T, a.P, a.H, a.HV, a.Dk, a.Dv = 3, 64, 8, 2, 4, 128, 128
    a.dtype, a.algo, a.g_min, a.scale, a.l2_eps = 1, 0, -5.0, 1.0, 1e-6
    a.qk_l2norm_in_kernel = a.beta_sigmoid_in_kernel = a.gate_in_kernel = a.g_per_head = 1
    a.ld_q = a.ld_k = 256
    a.ld_v = a.ld_o = 512
    a.ld_g = a.ld_beta = 4
    return _fill(a, ["q", "k", "v", "g", "beta", "A_log", "dt_bias", "cu_seqlens", "slots", "fresh", "pool", "o"], **kw)


def packed(**kw):
    return kda.load().kda_packed_fwd(ctypes.byref(packed_args(**kw)), None)


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(H=3), INVALID), (dict(N=-1), INVALID), (dict(P=-1), INVALID), (dict(max_seqlen=-1), INVALID),
    (dict(T=0x7FFFFFFF), INVALID), (dict(dtype=3), INVALID), (dict(algo=5), INVALID), (dict(g_min=0.0), INVALID),
    (dict(gate_in_kernel=3), INVALID), (dict(l2_eps=float("nan")), INVALID), (dict(A_log=None), INVALID),
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(pool=None), INVALID),
    (dict(cu_seqlens=None), INVALID),                       # 3 sequences, 64 rows
    (dict(slots=None, P=2), INVALID),                       # sequence 2 would have no slot
    (dict(ld_q=255), INVALID), (dict(ld_o=511), INVALID), (dict(ld_g=3), INVALID),
    (dict(Dk=129, ld_q=258, ld_k=258), UNSUPPORTED), (dict(Dv=126, ld_v=504, ld_o=504), UNSUPPORTED),
    (dict(N=1 << 30, algo=1), UNSUPPORTED),
    (dict(algo=2, dtype=0), UNSUPPORTED), (dict(algo=2, g_per_head=0, ld_g=512), UNSUPPORTED),
    (dict(algo=2, Dv=64), UNSUPPORTED),
    (dict(algo=2, ld_q=260), ALIGN),                        # rows not 16-byte aligned
    (dict(q=BASE + 1), ALIGN), (dict(pool=BASE + 16 * MB * 11 + 4), ALIGN), (dict(slots=BASE + 2), ALIGN),
    (dict(o=BASE + 16 * MB), ALIAS),                        # o over q
    (dict(o=BASE + 16 * MB * 11), ALIAS),                   # o over the pool
    (dict(pool=BASE + 16 * MB * 3), ALIAS),                 # the pool over v
    (dict(o=BASE + 16 * MB * 9), ALIAS),                    # o over the slots
    (dict(N=0), OK), (dict(T=0), OK),
    (dict(), CUDA), (dict(algo=1), CUDA), (dict(P=0), CUDA),
])
def test_packed_refusals(kw, want):
    if kw.get("P") == 0:
        kw = dict(kw, pool=None)
    assert packed(**kw) == want


def conv_args(**kw):
    a = _lib.PackedConvArgs()
    a.N, a.T, a.P, a.C, a.K, a.head_dim, a.silu, a.dtype, a.l2_eps = 3, 64, 8, 256, 4, 128, 1, 1, 1e-6
    a.ld_x = a.ld_y = 256
    return _fill(a, ["x", "w", "bias", "cu_seqlens", "slots", "fresh", "pool", "y"], **kw)


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(K=5), INVALID), (dict(K=0), INVALID), (dict(N=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(l2_eps=-1.0), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(pool=None), INVALID),
    (dict(cu_seqlens=None), INVALID), (dict(slots=None, P=1), INVALID), (dict(ld_x=255), INVALID),
    (dict(C=100), UNSUPPORTED), (dict(head_dim=64), UNSUPPORTED),
    (dict(ld_x=260), ALIGN), (dict(x=BASE + 8), ALIGN), (dict(pool=BASE + 16 * MB * 7 + 8), ALIGN),
    (dict(y=BASE + 16 * MB), ALIAS), (dict(y=BASE + 16 * MB * 7), ALIAS), (dict(pool=BASE + 16 * MB), ALIAS),
    (dict(N=0), OK), (dict(T=0), OK), (dict(), CUDA), (dict(K=1, pool=None), CUDA),
])
def test_packed_conv_refusals(kw, want):
    assert kda.load().kda_packed_conv(ctypes.byref(conv_args(**kw)), None) == want


def norm_args(**kw):
    a = _lib.GroupNormArgs()
    a.N, a.L, a.C, a.G, a.act, a.dtype, a.eps = 2, 4096, 256, 8, 1, 1, 1e-5
    return _fill(a, ["x", "gate", "weight", "bias", "y", "mean", "rstd", "dy", "dx", "dgate", "dweight", "dbias",
                     "workspace"], **kw)


COMMON = [(dict(L=0), INVALID), (dict(G=3), INVALID), (dict(G=0), INVALID), (dict(act=3), INVALID),
          (dict(dtype=4), INVALID), (dict(eps=-1.0), INVALID), (dict(x=None), INVALID), (dict(mean=None), INVALID),
          (dict(workspace=None), INVALID), (dict(workspace=BASE + 16 * MB * 13 + 4), ALIGN), (dict(x=BASE + 1), ALIGN),
          (dict(weight=BASE + 2), ALIGN), (dict(), CUDA), (dict(L=1 << 30), UNSUPPORTED)]


@no_gpu_only
@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(y=None), INVALID), (dict(y=BASE + 16 * MB), ALIAS), (dict(y=BASE + 16 * MB * 2 + 64), ALIAS),
    (dict(mean=BASE + 16 * MB * 5), ALIAS), (dict(workspace=BASE + 16 * MB), ALIAS), (dict(N=0), OK)])
def test_group_norm_forward_refusals(kw, want):
    assert kda.load().kda_group_norm_fwd(ctypes.byref(norm_args(**kw)), None) == want


@no_gpu_only
@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(dy=None), INVALID), (dict(gate=None), INVALID), (dict(dx=BASE + 16 * MB), ALIAS),
    (dict(dx=BASE + 16 * MB * 8), ALIAS), (dict(dgate=BASE + 16 * MB * 9), ALIAS),
    (dict(dbias=BASE + 16 * MB * 11), ALIAS), (dict(N=0, dweight=None, dbias=None), OK)])
def test_group_norm_backward_refusals(kw, want):
    assert kda.load().kda_group_norm_bwd(ctypes.byref(norm_args(**kw)), None) == want


def test_null_arguments():
    lib = kda.load()
    for fn in (lib.kda_packed_fwd, lib.kda_packed_conv, lib.kda_group_norm_fwd, lib.kda_group_norm_bwd):
        assert fn(None, None) == INVALID


def test_group_norm_workspace_sizes():
    ws = kda.load().kda_group_norm_workspace
    assert ws(2, 4096, 256, 8, 1, 0) > 0 and ws(2, 4096, 256, 8, 1, 1) > 0
    assert ws(2, 4096, 256, 7, 1, 0) == 0 and ws(0, 4096, 256, 8, 1, 0) == 0 and ws(2, 0, 256, 8, 1, 1) == 0
    assert ws(1000, 1, 4096, 32, 1, 0) == 0          # one pass, nothing to keep


def test_binding_refuses_what_is_no_cuda_tensor():
    x = torch.zeros(4, 1, 16)
    with pytest.raises(ValueError):
        kda.kda_packed_fwd(x, x, x, x, torch.zeros(4, 1), torch.zeros(4, 1, 16, 16))
    with pytest.raises(ValueError):
        kda.kda_packed_conv(torch.zeros(4, 128), torch.zeros(128, 4), torch.zeros(4, 3, 128))
    with pytest.raises(ValueError):
        kda.kda_group_norm_fwd(x, 4)


@pytest.mark.parametrize("make,ok", [
    (lambda: torch.zeros(4, 3, 5), True), (lambda: torch.zeros(4, 40)[:, :15].unflatten(1, (3, 5)), True),
    (lambda: torch.zeros(4, 5, 3).transpose(1, 2), False), (lambda: torch.zeros(3, 5).expand(4, 3, 5), False),
    (lambda: torch.zeros(1, 40)[:, :15].unflatten(1, (3, 5)), None)])
def test_rows_may_lie_apart_but_not_overlap(make, ok):
    t = make()
    shape = tuple(t.shape)
    if ok is False:
        with pytest.raises(ValueError):
            _lib._check_rows(t, "t", shape, torch.float32, t.device)
    else:
        assert _lib._check_rows(t, "t", shape, torch.float32, t.device) == (t.stride(0) if ok else 15)
