"""Host emulation of the packed kernels and of group norm -- TEST INFRASTRUCTURE.

Compiles kda_packed.cu, kda_packed_conv.cu, kda_group_norm.cu and
kda_packed_tc.cu (cut before their launchers, as emu_build does for the other
kernels; the last over tcinc/tc_ptx.cuh, the host model of the tcgen05, TMA and
mbarrier instructions) with g++ and AddressSanitizer or ThreadSanitizer.  The library never uses any of this.
"""
import os
import re

import emu_build
from emu_build import CSRC, HERE, OUT, _POISON, SMEM_FLOATS

LIB = os.path.join(OUT, "libkda_packed_emu.so")

# What the packed kernels use beyond the stand-in headers.
_MORE = r'''
inline int __any_sync(unsigned m, int pred) {
    float r = pred ? 1.f : 0.f;
    for (int off = 16; off > 0; off >>= 1) r += __shfl_xor_sync(m, r, off);
    return r != 0.f;
}
inline unsigned __ballot_sync(unsigned m, int pred) {
    unsigned r = 0;
    const int lane = threadIdx.x & 31;
    for (int x = 0; x < 32; ++x)
        if (__shfl_xor_sync(m, pred ? 1.f : 0.f, x) != 0.f) r |= 1u << (lane ^ x);
    return r;
}
inline int __popc(unsigned v) { return __builtin_popcount(v); }
// Any other lane's value, in xor steps: the lanes meet five times.
inline float emu_lane_value(unsigned m, float v, int src) {
    const int lane = threadIdx.x & 31;
    float r = 0.f;
    for (int x = 0; x < 32; ++x) {
        const float o = __shfl_xor_sync(m, v, x);
        if ((lane ^ x) == src) r = o;
    }
    return r;
}
inline float __shfl_up_sync(unsigned m, float v, int off) {
    const int lane = threadIdx.x & 31;
    return emu_lane_value(m, v, lane >= off ? lane - off : lane);
}
inline float __shfl_sync(unsigned m, float v, int src) { return emu_lane_value(m, v, src); }
inline unsigned __byte_perm(unsigned a, unsigned b, unsigned s) {
    const unsigned long long v = ((unsigned long long)b << 32) | a;
    unsigned r = 0;
    for (int i = 0; i < 4; ++i) r |= (unsigned)((v >> (8 * ((s >> (4 * i)) & 7))) & 0xFF) << (8 * i);
    return r;
}
using std::memcpy;
'''

_RUN_RECURRENT = _POISON + r'''
extern "C" int emu_sizeof_packed_params(void) { return (int)sizeof(kda::PackedParams); }
template <typename Tin, int RPL, bool PER_HEAD, int TPW, bool LOOP>
static void run_one(const kda::PackedParams &p, int warps) {
    using namespace kda;
    const int all = (p.Dv + kCW - 1) / kCW;
    emu_poison((size_t)(LOOP ? 2 : 1) * TPW * warps * token_floats(RPL * kRG, PER_HEAD) * sizeof(float));
    emu_launch(dim3(p.N * p.HV, (all + warps - 1) / warps), dim3(32 * warps),
               [&] { packed_recurrent_kernel<Tin, RPL, PER_HEAD, TPW, LOOP>(p); });
}
// warps = 0: every sequence fits one tile of a token per warp
template <typename Tin, int RPL, bool PER_HEAD>
static void run_len(const kda::PackedParams &p, int warps) {
    if (warps == 0) run_one<Tin, RPL, PER_HEAD, 1, false>(p, (p.Dv + kda::kCW - 1) / kda::kCW);
    else run_one<Tin, RPL, PER_HEAD, 2, true>(p, warps);
}
template <typename Tin>
static void run_type(const kda::PackedParams &p, int warps) {
    if (p.Dk <= 64) p.g_per_head ? run_len<Tin, 8, true>(p, warps) : run_len<Tin, 8, false>(p, warps);
    else p.g_per_head ? run_len<Tin, 16, true>(p, warps) : run_len<Tin, 16, false>(p, warps);
}
extern "C" int emu_packed_recurrent(kda::PackedParams *p, int bf16, int warps) {
    kda::g_packed_error = 0;
    if (bf16) run_type<__nv_bfloat16>(*p, warps);
    else run_type<float>(*p, warps);
    return (int)kda::g_packed_error;
}
'''
_RUN_CONV = _POISON + r'''
extern "C" int emu_sizeof_packed_conv_params(void) { return (int)sizeof(kda::PackedConvParams); }
template <typename Tin>
static void run_conv(const kda::PackedConvParams &p, int run) {
    using namespace kda;
    emu_poison(0);
    const long long warps = ((long long)p.T + run - 1) / run * ((p.C + 255) / 256);
    const dim3 grid((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
#define KDA_RUN(K) \
    if (run == 1) emu_launch(grid, dim3(kThreads), [&] { packed_conv_kernel<Tin, K, 1>(p, run); }); \
    else emu_launch(grid, dim3(kThreads), [&] { packed_conv_kernel<Tin, K, 4>(p, run); })
    switch (p.K) {
        case 1: KDA_RUN(1); break;
        case 2: KDA_RUN(2); break;
        case 3: KDA_RUN(3); break;
        default: KDA_RUN(4); break;
    }
#undef KDA_RUN
}
extern "C" int emu_packed_conv(kda::PackedConvParams *p, int bf16, int run) {
    kda::g_packed_conv_error = 0;
    if (bf16) run_conv<__nv_bfloat16>(*p, run);
    else run_conv<float>(*p, run);
    return (int)kda::g_packed_conv_error;
}
'''
_RUN_NORM = _POISON + r'''
extern "C" int emu_sizeof_group_norm_params(void) { return (int)sizeof(kda::GroupNormParams); }
extern "C" long long emu_group_norm_ws(int N, int L, int C, int G, int bf16, int backward, int aligned) {
    return (long long)kda::group_norm_plan(N, L, C, G, bf16, backward, aligned).ws_floats;
}
template <typename Tin, int VEC, int VPT, bool GATED>
static void run_held(const kda::GroupNormParams &p, const kda::GroupNormPlan &pl, bool backward) {
    using namespace kda;
    emu_poison(kHeldSmem);
    const dim3 grid(pl.gx, pl.gy);
    if (!backward) {
        emu_launch(grid, dim3(kThreads), [&] { gn_held_fwd_kernel<Tin, VEC, VPT, GATED>(p, pl); });
        return;
    }
    if constexpr (VPT <= 2) {
        emu_launch(grid, dim3(kThreads), [&] { gn_held_bwd_kernel<Tin, VEC, VPT, GATED>(p, pl); });
        emu_poison(kSumSmem);
        emu_launch(dim3((p.C + 31) / 32), dim3(kSumThreads),
                   [&] { gn_sum_kernel(p.ws, pl.gy, p.C, p.dweight, p.dbias); });
    }
}
template <typename Tin, int VEC, bool GATED>
static void run_tiled(const kda::GroupNormParams &p, const kda::GroupNormPlan &pl, bool backward) {
    using namespace kda;
    emu_poison(kTileSmem);
    const dim3 grid(pl.gx, pl.gy);
    if (!backward) {
        emu_launch(grid, dim3(kThreads), [&] { gn_tile_stats_kernel<Tin, VEC>(p, pl); });
        emu_launch(dim3(p.N * p.G), dim3(kThreads), [&] { gn_tile_mean_kernel(p, pl); });
        emu_launch(grid, dim3(kThreads), [&] { gn_tile_fwd_kernel<Tin, VEC, GATED>(p, pl); });
        return;
    }
    float *gsum = p.ws + (size_t)p.N * pl.tiles * 2 * p.C;
    emu_launch(grid, dim3(kThreads), [&] { gn_tile_dsum_kernel<Tin, VEC, GATED>(p, pl); });
    emu_poison(kSumSmem);
    emu_launch(dim3(p.N * p.G + (p.C + 31) / 32), dim3(kSumThreads), [&] { gn_tile_gsum_kernel(p, pl, gsum); });
    emu_poison(kTileSmem);
    emu_launch(grid, dim3(kThreads), [&] { gn_tile_bwd_kernel<Tin, VEC, GATED>(p, pl, gsum); });
}
template <typename Tin, int VEC, bool GATED>
static void run_norm(const kda::GroupNormParams &p, const kda::GroupNormPlan &pl, bool backward) {
    if (!pl.held) run_tiled<Tin, VEC, GATED>(p, pl, backward);
    else if (pl.vpt == 1) run_held<Tin, VEC, 1, GATED>(p, pl, backward);
    else if (pl.vpt == 2) run_held<Tin, VEC, 2, GATED>(p, pl, backward);
    else run_held<Tin, VEC, 4, GATED>(p, pl, backward);
}
template <typename Tin, int FULL>
static void run_norm_type(const kda::GroupNormParams &p, const kda::GroupNormPlan &pl, bool backward) {
    if (pl.vec == FULL) p.gate ? run_norm<Tin, FULL, true>(p, pl, backward) : run_norm<Tin, FULL, false>(p, pl, backward);
    else p.gate ? run_norm<Tin, 1, true>(p, pl, backward) : run_norm<Tin, 1, false>(p, pl, backward);
}
extern "C" int emu_group_norm(kda::GroupNormParams *p, int bf16, int backward, int aligned) {
    kda::GroupNormPlan pl = kda::group_norm_plan(p->N, p->L, p->C, p->G, bf16, backward, aligned);
    if (pl.held && pl.gy > 2) pl.gy = 2;      // few blocks, so that each walks several rows
    if (bf16) run_norm_type<__nv_bfloat16, 8>(*p, pl, backward);
    else run_norm_type<float, 4>(*p, pl, backward);
    return pl.held;
}
'''

_RUN_CHUNK = r'''
#include <sanitizer/asan_interface.h>
namespace kda { namespace tc { EmuCta *g_cta = nullptr; EmuTf32Slots g_tf32[32]; } }
static kda::tc::EmuTensorMap emu_map(const void *base, int heads, long long rows, long long ld, bool swizzle) {
    kda::tc::EmuTensorMap m{};
    m.base = static_cast<const uint8_t *>(base);
    m.dims[0] = 128; m.dims[1] = (uint64_t)heads; m.dims[2] = (uint64_t)rows;
    m.strides[0] = 256; m.strides[1] = (uint64_t)ld * 2;
    m.box[0] = swizzle ? 64 : 128; m.box[1] = 1; m.box[2] = 64;
    m.swizzle128 = swizzle ? 1 : 0;
    return m;
}
extern "C" int emu_packed_chunk(kda::PackedParams *pp, int ctas) {
    using namespace kda;
    PackedTcParams tp;
    tp.p = *pp;
    const tc::EmuTensorMap maps[3] = {emu_map(pp->k, pp->H, pp->T, pp->ldk, true),
                                      emu_map(pp->q, pp->H, pp->T, pp->ldq, true),
                                      emu_map(pp->v, pp->HV, pp->T, pp->ldv, false)};
    for (int i = 0; i < 3; ++i) std::memcpy(&tp.tm[i], &maps[i], sizeof maps[i]);
    static tc::EmuCta cta;
    static tc::EmuMBar bars[sizeof smem_raw / 8];
    cta.smem = smem_raw;
    cta.smem_bytes = SMEM_BYTES;
    cta.bars = bars;
    g_packed_chunk_error = 0;
    emu_launch_cb(dim3(ctas), dim3(kThreads),
                  [&](unsigned, unsigned) {
                      ASAN_UNPOISON_MEMORY_REGION(smem_raw, sizeof smem_raw);
                      std::memset(cta.tmem, 0xFF, sizeof cta.tmem);
                      std::memset(smem_raw, 0xFF, sizeof smem_raw);
                      ASAN_POISON_MEMORY_REGION(smem_raw + SMEM_BYTES, sizeof smem_raw - SMEM_BYTES);
                      tc::g_cta = &cta;
                  },
                  [&] { packed_chunk_kernel(tp); });
    return (int)g_packed_chunk_error;
}
'''


def _chunk_unit():
    s = open(os.path.join(CSRC, "kda_packed_tc.cu")).read()
    s = s[: s.index("bool packed_chunk_shape")] + "}  // namespace kda\n"
    s = s.replace("extern __shared__", "extern").replace("__shared__", "static")
    head = ('#include <functional>\n#include "cuda_runtime.h"\n' + _MORE +
            "void emu_launch_cb(dim3 grid, dim3 block, const std::function<void(unsigned, unsigned)> &on_block,\n"
            "                   const std::function<void()> &fn);\n"
            "namespace kda { namespace { alignas(1024) uint8_t smem_raw[240 * 1024]; } }\n")
    return head + '#line 1 "kda_packed_tc.cu"\n' + s + _RUN_CHUNK


def _unit(src_name, runner, extra=None):
    """As emu_build._unit; `extra` = (from, to): a stretch of the source behind
    the cut (host functions that the runner needs), kept too."""
    s = open(os.path.join(CSRC, src_name)).read()
    m = re.search(r"^(template <[^>]*>\n(static )?)?cudaError_t launch_", s, re.M)
    body = s[: m.start()]
    if "\n}  // namespace\n" not in body:
        body += "\n}  // namespace\n"
    if extra:
        a = s.index(extra[0])
        body += "namespace {\n" + s[a: s.index(extra[1])] if extra[2] else s[a: s.index(extra[1])]
    body += "}  // namespace kda\n"
    body = body.replace("extern __shared__", "extern").replace("__shared__", "static")
    head = ('#include <functional>\n#include "cuda_runtime.h"\n' + _MORE +
            "void emu_launch(dim3 grid, dim3 block, const std::function<void()> &fn);\n"
            "namespace kda { namespace { alignas(16) float smem[%d]; } }\n" % SMEM_FLOATS)
    return head + "#line 1 \"%s\"\n" % src_name + body + runner


def _deps():
    return [os.path.join(CSRC, f) for f in ("kda_packed.cu", "kda_packed_conv.cu", "kda_group_norm.cu",
                                            "kda_packed_tc.cu", "kda_packed.cuh", "kda_group_norm.cuh", "kda_internal.cuh")] + \
        [os.path.join(HERE, f) for f in ("emu_packed.py", "emu_build.py", "emu_rt.cpp", "fakeinc/cuda_runtime.h",
                                         "fakeinc/cuda_bf16.h", "tcinc/tc_ptx.cuh")]


def build(force=False, sanitizer="address"):
    lib = LIB if sanitizer == "address" else LIB[:-3] + "_tsan.so"
    if not force and os.path.exists(lib) and all(os.path.getmtime(d) <= os.path.getmtime(lib) for d in _deps()):
        return lib
    units = {"emu_packed.cpp": _unit("kda_packed.cu", _RUN_RECURRENT),
             "emu_packed_conv.cpp": _unit("kda_packed_conv.cu", _RUN_CONV),
             "emu_group_norm.cpp": _unit("kda_group_norm.cu", _RUN_NORM,
                                         ("int pow2_at_least", "cudaError_t launch_group_norm_fwd", True)),
             "emu_packed_chunk.cpp": _chunk_unit()}
    if sanitizer != "address":
        units = {n: t.replace("#include <sanitizer/asan_interface.h>", "#define ASAN_POISON_MEMORY_REGION(a, b)\n"
                              "#define ASAN_UNPOISON_MEMORY_REGION(a, b)") for n, t in units.items()}
    return emu_build.compile_units(units, lib, sanitizer)


if __name__ == "__main__":
    print(build(force=True))
