"""More host-emulated runs of the packed kernels -- TEST INFRASTRUCTURE, started by
tests/test_packed_emu_more_cpu.py in a process with a sanitizer's runtime
preloaded: ``run_packed_more.py NAME [LIB]`` runs the function of that name and
exits non-zero if it fails.
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
import run_packed as rp  # noqa: E402
from helpers import to_np  # noqa: E402
from oracle import packed  # noqa: E402


def fp32_recurrence(q, k, v, g, beta, S, scale):
    """One chain token by token in 32 bits (q, k normalised in 64), o and S."""
    f = np.float32
    o = np.empty_like(v, dtype=f)
    S = S.astype(f)
    q = (q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6) * scale).astype(f)
    k = (k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)).astype(f)
    v, a, b = v.astype(f), np.exp(g).astype(f), (1 / (1 + np.exp(-beta))).astype(f)
    for t in range(len(v)):
        S = S * a[t]
        S = S + np.outer(k[t], b[t] * (v[t] - k[t] @ S))
        o[t] = q[t] @ S
    return o, S


def precision(lib):
    """The chunk form of one chain with hardly any decay, where errors of the state
    stay longest: no further from 64 bits than a recurrence in 32 bits, in the
    state and in the share of bf16 outputs that are not the rounded exact ones."""
    T, bf = 256, torch.bfloat16
    for seed, z_mean in ((1, -8.0), (2, -4.0)):
        gen = torch.Generator().manual_seed(seed)
        q, k, v = (torch.randn(T, 1, 128, generator=gen).to(bf) for _ in range(3))
        g, beta = (torch.randn(T, 1, generator=gen) + z_mean).to(bf), torch.randn(T, 1, generator=gen).to(bf)
        A, b = torch.zeros(1), torch.zeros(1)
        pool, o = torch.randn(1, 1, 128, 128, generator=gen) * 0.05, torch.zeros(T, 1, 128, dtype=bf)
        scale = 128 ** -0.5
        want_o, want_S = packed.packed_fwd(*map(to_np, (q, k, v, g, beta, pool, o)), cu=[0, T], A_log=to_np(A),
                                           dt_bias=to_np(b), gate="softplus", per_head=True, scale=scale)
        decay = packed.log_decay(to_np(g), to_np(A), to_np(b), "softplus", True, 1)[:, 0, 0]
        rec_o, rec_S = fp32_recurrence(*(to_np(t)[:, 0] for t in (q, k, v)), decay, to_np(beta)[:, 0],
                                       to_np(pool)[0, 0], scale)
        cu = torch.tensor([0, T], dtype=torch.int32)
        p = rp.PackedParams(1, T, 1, 1, 1, 128, 128, 1, -5.0, scale, 1e-6, 1, 1, 2, 1, 0,
                            *(t.stride(0) for t in (q, k, v, g, beta, o)),
                            *map(rp._ptr, (q, k, v, g, beta, A, b, cu, None, None, pool, o)))
        lib.emu_packed_chunk(ctypes.byref(p), 1)

        def off(S):
            return np.linalg.norm(to_np(S) - want_S[0, 0]) / np.linalg.norm(want_S)

        rounded = torch.from_numpy(want_o[:, 0]).to(bf)
        flips = [int((x != rounded).sum()) for x in (o[:, 0], torch.from_numpy(rec_o).to(bf))]
        errs = [off(pool[0, 0]), off(torch.from_numpy(rec_S))]
        print("state off by %.2e (32 bits: %.2e), outputs %d (%d) of %d" % (*errs, *flips, rounded.numel()), flush=True)
        assert errs[0] <= errs[1]
        # counts of rare events: three standard deviations of the recurrence's own count
        assert flips[0] <= flips[1] + 3 * flips[1] ** 0.5 + 3


# Chunk-kernel runs that come round: several chunks a chain, chains and sequences one
# after another, so that every stage, parity and buffer is used again.
ONE = dict(cu=[0, 330], slots=[0], fresh=None, P=1)
LAST = dict(cu=[0, 150, 150, 341], slots=[1, 0, 2], fresh=[0, 0, 1], P=3)
ROUNDS = [
    dict(pack=rp.LONG, T=230, H=1, HV=2, ctas=2), dict(pack=ONE, T=330, H=1, HV=1, ctas=1),
    dict(pack=LAST, T=341, H=1, HV=1, ctas=1),
]


def chunk_rounds(lib):
    for i, kw in enumerate(ROUNDS):
        errs = rp.run_delta(lib, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=True, seed=20 + i, **kw)
        print({n: "%.1e" % e for n, (e, _) in errs.items()}, flush=True)
        assert all(e <= tol for e, tol in errs.values())


def chunk_rounds_races(lib):
    """For the thread sanitizer: no oracle."""
    for kw in ROUNDS:
        rp.run_delta(lib, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=True, check=False, **kw)


# Sequences without rows that name another's slot, behind it, ahead of it and among
# themselves: legal, nothing is reported and nobody is skipped.
SHARED = dict(cu=[0, 0, 3, 3, 70, 70, 70], slots=[1, 0, 0, 1, 2, 2], fresh=None, P=3)


def empty_sequences(lib):
    runs = [(rp.run_delta, dict(H=1, HV=1, Dk=24, Dv=8, dtype="f32", gate="bounded", per_head=False)),
            (rp.run_delta, dict(H=1, HV=1, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=True, ctas=1)),
            (rp.run_conv, dict(C=128, K=4, dtype="f32", head_dim=0, silu=True, run=4))]
    assert not packed.live(SHARED["cu"], SHARED["slots"], 70, 3, 6)[1]
    for i, (fn, kw) in enumerate(runs):
        errs = fn(lib, pack=SHARED, T=70, seed=40 + i, **kw)
        print(fn.__name__, {n: "%.1e" % e for n, (e, _) in errs.items()}, flush=True)
        assert all(e <= tol for e, tol in errs.values())


def conv_bounds(lib):
    """The convolution over bounds of which some lie outside the rows or run backwards:
    every sequence whose own bounds are good is computed, whatever the others hold."""
    rng = np.random.default_rng(5)
    packs = [[0, 5, -3, 12], [0, 6, 40, 41, 9, 12], [-2, 4, 4, 9, 100, 12]]
    for n in (5, 40, 70):
        cu = np.sort(rng.integers(0, 61, n + 1))
        bad = rng.choice(n + 1, 3, replace=False)
        packs.append(np.where(np.isin(np.arange(n + 1), bad), rng.choice([-7, 70, 1 << 30, 3], n + 1), cu).tolist())
    for i, cu in enumerate(packs):
        T, n = max(x for x in cu if x <= 61), len(cu) - 1
        pack = dict(cu=cu, slots=list(range(n)), fresh=None, P=n)
        gen = torch.Generator().manual_seed(i)
        for dtype, run in ((torch.float32, 1), (torch.bfloat16, 4), (torch.float32, 8))[: 3 if n < 6 else 2]:
            C, K = 128, 4
            x, w = torch.randn(T, C, generator=gen).to(dtype), torch.randn(C, K, generator=gen)
            pool, y = torch.randn(n, K - 1, C, generator=gen).to(dtype), torch.full((T, C), 0.0625).to(dtype)
            want_y, want_pool = packed.packed_conv(*map(to_np, (x, w, pool, y)), cu=cu, slots=pack["slots"], silu=False)
            live, report = packed.live(cu, pack["slots"], T, n, n)
            once = np.zeros(T, dtype=int)             # rows of two sequences hold either's result
            for _, b, e, _ in live:
                once[b:e] += 1
            n_, cut, slots, _ = rp.pack_of(pack, T)
            p = rp.ConvParams(n, T, n, C, K, 0, 0, 1e-6, C, C, *map(rp._ptr, (x, w, None, cut, slots, None, pool, y)))
            word = lib.emu_packed_conv(ctypes.byref(p), int(dtype == torch.bfloat16), run)
            assert bool(word) == report and report, cu
            assert np.array_equal(to_np(pool), want_pool), (cu, run)
            tol = rp.TOL["bf16" if dtype == torch.bfloat16 else "f32"]
            err = np.abs(to_np(y) - want_y)[once < 2].max() / np.abs(want_y).max()
            assert err <= tol, (cu, run, err)


def main():
    import emu_packed
    lib = rp.load(sys.argv[2] if len(sys.argv) > 2 else emu_packed.LIB)
    globals()[sys.argv[1]](lib)
    print("done")


if __name__ == "__main__":
    main()
