"""Runs the host-emulated packed and group-norm kernels on small seeded
problems and compares them with the FP64 oracle.

TEST INFRASTRUCTURE, started by tests/test_packed_emu_cpu.py in a process with
the AddressSanitizer runtime preloaded; prints one line per case and exits
non-zero on a mismatch.  With ``--races LIB`` it runs a few cases through the
ThreadSanitizer build without the oracle.
"""
import ctypes
import os
import sys

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, os.path.dirname(os.path.dirname(HERE)))
from helpers import max_rel, to_np  # noqa: E402
from oracle import packed  # noqa: E402

_P, _I, _F, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong


class PackedParams(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("N", "T", "P", "H", "HV", "Dk", "Dv", "group")] + \
        [(n, _F) for n in ("g_min", "scale", "l2_eps")] + \
        [(n, _I) for n in ("l2norm", "beta_sigmoid", "gate_in", "g_per_head", "split")] + \
        [(n, _L) for n in ("ldq", "ldk", "ldv", "ldg", "ldb", "ldo")] + \
        [(n, _P) for n in ("q", "k", "v", "g", "beta", "A_log", "dt_bias", "cu", "slots", "fresh", "pool", "o")]


class ConvParams(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("N", "T", "P", "C", "K", "head_dim", "silu")] + [("l2_eps", _F)] + \
        [(n, _L) for n in ("ldx", "ldy")] + \
        [(n, _P) for n in ("x", "w", "bias", "cu", "slots", "fresh", "pool", "y")]


class NormParams(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("N", "L", "C", "G", "D", "act")] + [("eps", _F)] + \
        [(n, _P) for n in ("x", "gate", "dy", "weight", "bias", "y", "dx", "dgate", "mean", "rstd", "dweight",
                           "dbias", "ws")]


ACT = {"none": 0, "silu": 1, "sigmoid": 2}
GATE = {False: 0, "bounded": 1, "softplus": 2}


def _ptr(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _i32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32)


# Largest difference over the largest reference value: fp32 sums of at most 128
# terms over tens of tokens, exp and sqrt of a few ulp; bf16 outputs a half step.
TOL = {"f32": 1e-5, "bf16": 2.0 ** -8 + 1e-5}

PACK = dict(cu=[0, 3, 3, 20, 21, 40], slots=[2, 0, 5, -1, 1], fresh=[0, 1, 1, 0, 0], P=6)
ODD = dict(cu=[2, 4, 9, 7, 30, 33], slots=[3, 3, 1, 9, 0], fresh=None, P=4)      # repeat, backwards, slot 9
LONG = dict(cu=[0, 70, 199, 199, 226, 230], slots=[2, 0, 5, -1, 1], fresh=[0, 1, 1, 0, 0], P=6)
FEW = dict(cu=[0, 8, 8, 9, 12], slots=[1, 0, -1, 2], fresh=[0, 0, 0, 1], P=3)
STEP = dict(cu=None, slots=None, fresh=None, P=7)


def pack_of(pack, T=None):
    cu = pack["cu"]
    n = T if cu is None else len(cu) - 1
    fresh = None if pack["fresh"] is None else torch.tensor(pack["fresh"], dtype=torch.uint8)
    return n, _i32(cu), _i32(pack["slots"]), fresh


def run_delta(lib, pack, T, H, HV, Dk, Dv, dtype, gate, per_head, flags=True, pad=0, warps=4,
              ctas=0, z_mean=0.0, seed=0, check=True):
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16

    def rows(*shape):      # rows `pad` elements apart
        w = int(np.prod(shape))
        return torch.randn(T, w + pad, generator=gen).to(dt)[:, :w].unflatten(1, shape)

    gk = () if per_head else (Dk,)
    q, k, v, g, beta = rows(H, Dk), rows(H, Dk), rows(HV, Dv), rows(HV, *gk), rows(HV)
    g += z_mean
    if not flags:
        g, beta = (g.abs() * -0.3).to(dt), beta.abs().clamp(max=1)
        q, k = (q / Dk ** 0.5).to(dt), (k / Dk ** 0.5).to(dt)
        if pad:
            raise ValueError("pad needs flags")
    A, b = torch.rand(HV, generator=gen) * 2 - 1, torch.randn((HV,) + gk, generator=gen) * 0.5
    pool = torch.randn(pack["P"], HV, Dk, Dv, generator=gen) * 0.1
    o = torch.full((T, HV, Dv), 0.0625).to(dt)
    n, cu, slots, fresh = pack_of(pack, T)
    want = packed.packed_fwd(*map(to_np, (q, k, v, g, beta, pool, o)), cu=pack["cu"], slots=pack["slots"],
                             fresh=pack["fresh"], A_log=to_np(A), dt_bias=to_np(b), gate=gate if flags else False,
                             per_head=per_head, scale=0.3, l2norm=flags, beta_sigmoid=flags) if check else None
    p = PackedParams(n, T, pack["P"], H, HV, Dk, Dv, HV // H, -5.0, 0.3, 1e-6, int(flags), int(flags),
                     GATE[gate] if flags else 0, int(per_head), 1 << 30,
                     *(t.stride(0) for t in (q, k, v, g, beta, o)),
                     *map(_ptr, (q, k, v, g, beta, A, b, cu, slots, fresh, pool, o)))
    if ctas:
        p.split = 0
        word = lib.emu_packed_chunk(ctypes.byref(p), ctas)
    else:
        word = lib.emu_packed_recurrent(ctypes.byref(p), int(dtype == "bf16"), warps)
    if not check:
        return None
    assert bool(word) == packed.live(pack["cu"], pack["slots"], T, pack["P"], n)[1]
    return {"o": (max_rel(to_np(o), want[0]), TOL[dtype]), "pool": (max_rel(to_np(pool), want[1]), TOL["f32"])}


def run_conv(lib, pack, T, C, K, dtype, head_dim, silu, run, pad=0, seed=0, check=True):
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = torch.randn(T, C + pad, generator=gen).to(dt)[:, :C]
    w, bias = torch.randn(C, K, generator=gen), torch.randn(C, generator=gen) * 0.1
    pool = torch.randn(pack["P"], K - 1, C, generator=gen).to(dt)
    y = torch.full((T, C), 0.0625).to(dt)
    n, cu, slots, fresh = pack_of(pack, T)
    want = packed.packed_conv(*map(to_np, (x, w, pool, y, bias)), cu=pack["cu"], slots=pack["slots"],
                              fresh=pack["fresh"], head_dim=head_dim, silu=silu) if check else None
    p = ConvParams(n, T, pack["P"], C, K, head_dim, int(silu), 1e-6, x.stride(0), y.stride(0),
                   *map(_ptr, (x, w, bias, cu, slots, fresh, pool, y)))
    word = lib.emu_packed_conv(ctypes.byref(p), int(dtype == "bf16"), run)
    if not check:
        return None
    assert bool(word) == packed.live(pack["cu"], pack["slots"], T, pack["P"], n)[1]
    return {"y": (max_rel(to_np(y), want[0]), TOL[dtype]), "pool": (max_rel(to_np(pool), want[1]), 0.0)}


def run_norm(lib, N, L, C, G, dtype, act, gated, aligned=1, params=True, seed=0, check=True):
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    bf = int(dtype == "bf16")
    x = (torch.randn(N, L, C, generator=gen) + 3).to(dt)
    dy = torch.randn(N, L, C, generator=gen).to(dt)
    z = torch.randn(N, L, C, generator=gen).to(dt) if gated else None
    w = 1 + 0.3 * torch.randn(C, generator=gen) if params else None
    b = 0.3 * torch.randn(C, generator=gen) if params else None
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    dz = torch.zeros_like(x) if gated else None
    mean, rstd, dw, db = torch.zeros(N, G), torch.zeros(N, G), torch.full((C,), 9.0), torch.full((C,), 9.0)
    args = (x, G) + tuple(None if t is None else to_np(t) for t in (w, b, z))
    for backward in (0, 1):
        ws = torch.full((max(1, lib.emu_group_norm_ws(N, L, C, G, bf, backward, aligned)),), float("nan"))
        p = NormParams(N, L, C, G, C // G, ACT[act], 1e-5,
                       *map(_ptr, (x, z, dy, w, b, y, dx, dz, mean, rstd, dw, db, ws)))
        lib.emu_group_norm(ctypes.byref(p), bf, backward, aligned)
    if not check:
        return None
    xn = to_np(x)
    wy, wm, wr = packed.group_norm(xn, *args[1:], act=act)
    g = packed.group_norm_backward(to_np(dy), xn, *args[1:], act=act)
    got = {"y": (max_rel(to_np(y), wy), TOL[dtype]), "mean": (max_rel(to_np(mean), wm), 1e-6),
           "rstd": (max_rel(to_np(rstd), wr), 1e-5), "dx": (max_rel(to_np(dx), g["dx"]), TOL[dtype])}
    for name, t in (("dweight", dw), ("dbias", db)):
        got[name] = (float(np.max(np.abs(to_np(t) - g[name])) / np.max(g["l1"])), 1e-5)
    if gated:
        got["dgate"] = (max_rel(to_np(dz), g["dgate"]), TOL[dtype])
    return got


CASES = [
    (run_delta, dict(pack=PACK, T=43, H=1, HV=2, Dk=24, Dv=20, dtype="f32", gate="bounded", per_head=False)),
    (run_delta, dict(pack=PACK, T=40, H=1, HV=1, Dk=65, Dv=36, dtype="bf16", gate="softplus", per_head=True, pad=3)),
    (run_delta, dict(pack=ODD, T=33, H=1, HV=2, Dk=16, Dv=4, dtype="f32", gate="softplus", per_head=False, warps=1)),
    (run_delta, dict(pack=STEP, T=5, H=2, HV=2, Dk=128, Dv=128, dtype="bf16", gate="bounded", per_head=False)),
    (run_delta, dict(pack=STEP, T=5, H=1, HV=2, Dk=40, Dv=20, dtype="f32", gate="softplus", per_head=True, warps=0)),
    (run_delta, dict(pack=FEW, T=12, H=1, HV=1, Dk=128, Dv=128, dtype="bf16", gate="bounded", per_head=False, warps=0)),
    (run_delta, dict(pack=PACK, T=43, H=1, HV=1, Dk=40, Dv=8, dtype="f32", gate="bounded", per_head=True,
                     flags=False, warps=1)),
    (run_delta, dict(pack=LONG, T=230, H=1, HV=2, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=True,
                     ctas=2)),
    (run_delta, dict(pack=ODD, T=33, H=1, HV=1, Dk=128, Dv=128, dtype="bf16", gate="bounded", per_head=True, ctas=1,
                     pad=8)),
    (run_delta, dict(pack=LONG, T=230, H=1, HV=1, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=True,
                     ctas=3, z_mean=8.0)),
    (run_delta, dict(pack=LONG, T=230, H=1, HV=1, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=True,
                     flags=False, ctas=1)),
    (run_conv, dict(pack=PACK, T=43, C=128, K=4, dtype="f32", head_dim=128, silu=True, run=1)),
    (run_conv, dict(pack=PACK, T=43, C=384, K=4, dtype="bf16", head_dim=0, silu=True, run=4, pad=8)),
    (run_conv, dict(pack=PACK, T=41, C=128, K=3, dtype="bf16", head_dim=128, silu=False, run=2)),
    (run_conv, dict(pack=ODD, T=33, C=128, K=2, dtype="f32", head_dim=0, silu=True, run=8)),
    (run_conv, dict(pack=STEP, T=7, C=256, K=4, dtype="bf16", head_dim=128, silu=True, run=1)),
    (run_conv, dict(pack=PACK, T=40, C=128, K=1, dtype="f32", head_dim=0, silu=False, run=16)),
    (run_norm, dict(N=9, L=1, C=256, G=2, dtype="bf16", act="silu", gated=True)),
    (run_norm, dict(N=5, L=1, C=60, G=3, dtype="f32", act="sigmoid", gated=False)),
    (run_norm, dict(N=3, L=1, C=1100, G=1, dtype="f32", act="none", gated=True)),
    (run_norm, dict(N=2, L=1, C=700, G=2, dtype="bf16", act="silu", gated=False, aligned=0)),
    (run_norm, dict(N=2, L=3, C=64, G=4, dtype="bf16", act="silu", gated=False)),
    (run_norm, dict(N=2, L=67, C=40, G=4, dtype="f32", act="silu", gated=True)),
    (run_norm, dict(N=1, L=300, C=48, G=1, dtype="bf16", act="none", gated=False, params=False)),
    (run_norm, dict(N=2, L=33, C=18, G=3, dtype="f32", act="sigmoid", gated=False)),
]
RACES = (0, 1, 5, 8, 12, 15, 17, 19, 22)


def load(path):
    lib = ctypes.CDLL(path)
    lib.emu_group_norm_ws.restype = ctypes.c_longlong
    assert lib.emu_sizeof_packed_params() == ctypes.sizeof(PackedParams)
    assert lib.emu_sizeof_packed_conv_params() == ctypes.sizeof(ConvParams)
    assert lib.emu_sizeof_group_norm_params() == ctypes.sizeof(NormParams)
    return lib


def main():
    if "--races" in sys.argv:
        lib = load(sys.argv[sys.argv.index("--races") + 1])
        for i in RACES:
            CASES[i][0](lib, check=False, **CASES[i][1])
        print("race run done")
        return 0
    import emu_packed
    lib = load(emu_packed.LIB)
    bad = 0
    for i, (fn, kw) in enumerate(CASES):
        errs = fn(lib, seed=i, **kw)
        wrong = {n: e for n, (e, tol) in errs.items() if not e <= tol}
        bad += bool(wrong)
        print(fn.__name__, {n: v for n, v in kw.items() if n != "pack"}, "MISMATCH" if wrong else "ok",
              {n: "%.1e" % e for n, (e, _) in errs.items()}, flush=True)
    return 1 if bad else 0


if __name__ == "__main__":
    sys.exit(main())
