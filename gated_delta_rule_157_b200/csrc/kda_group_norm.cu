// Group norm with an activation over channels-last rows x [N, L, C], forward
// and backward.  Statistics per (n, group) over L positions and D = C / G
// channels, in fp32:
//
//     h = (x - mean) rstd,   u = h w + b,   y = f(u)   or, with a gate z,   y = u f(z)
//     du = dy f'(u)          or   dy f(z), dz = dy u f'(z)
//     db = sum du,  dw = sum du h,  dh = du w,
//     dx = rstd (dh - mean(dh) - h mean(dh h))
//
// Memory bounds all of it: x (gate, dy) read once, y (dx, dz) written once.
//
// Held form (a slab of L * D values fits one block's registers; L = 1 is the
// per-token form): one pass.  A thread keeps the same channels over all rows n
// it visits, so weight and bias sit in registers and the backward's dw, db add
// up there; the next row's vectors are requested while one is computed.  The
// variance is the sum of squared distances from the mean (two sweeps over the
// registers), so a large mean costs no digits.
//
// Tiled form: (1) per tile of rows and channel, mean and squared distances from it
// (forward) or sum du, sum du h (backward); (2) their sums over tiles and the
// group's channels in a fixed order -- no atomics, the same bits every run; (3) the
// result.  Vectors may straddle groups in (1) and (3), so D is free there.  A thread
// squares distances from the mean of four rows at a time and joins (mean, squares) of
// two sets a, b by M2 = M2_a + M2_b + (mean_b - mean_a)^2 n_a n_b / n: no large sums are
// subtracted, whatever the rows.  Sums stay short at any length: at most kDepth
// steps a thread, trees over threads, compensated sums over tiles.
//
// Measured on the device (bf16): 16384 rows of 32 groups of 128 with a gate 88 us, 4.6
// TB/s (issue slots 77 % busy, 40 % of the warps), and their gradient for 8192 rows 84
// us, 4.0 TB/s (issue 65 %, 24 % of the warps); rows of 8192 x 1024 in 4 slabs, gradient
// 85 us: x and dy are read twice, from memory both times.
#include "kda_group_norm.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;                   // rows a thread requests together
constexpr int kDepth = 64;                 // steps a thread of the tiled form sums one after another
extern __shared__ float smem[];

template <typename Tin, int VEC> struct Vec;
template <> struct Vec<__nv_bfloat16, 8> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const unsigned u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&f)[8]) {
        unsigned u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&u[i], &b, 4);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Vec<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float *p) { r = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; }
    static __device__ __forceinline__ void put(float *p, const float (&f)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <typename Tin> struct Vec<Tin, 1> {
    Tin r;
    __device__ __forceinline__ void load(const Tin *p) { r = *p; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = ld_act(&r, 0); }
    static __device__ __forceinline__ void put(Tin *p, const float (&f)[1]) { st_act(p, 0, f[0]); }
};

// Sigmoid of a forward pass: library exp and division for fp32 values; for bf16 ones
// the hardware approximations, off by 2^-21 of the value near 0 and by 2^-18 at |u| =
// 88 (the product by log2 e is rounded), which vanishes in the output's rounding to
// 8 bits.
template <typename Tin> __device__ __forceinline__ float sig(float u) { return 1.f / (1.f + expf(-u)); }
template <> __device__ __forceinline__ float sig<__nv_bfloat16>(float u) {
    return rcpf_(1.f + ex2f_(-kLog2E * u));
}
template <typename Tin> __device__ __forceinline__ float act_f(int act, float u) {
    if (act == 0) return u;
    const float p = sig<Tin>(u);
    return act == 1 ? u * p : p;
}
// f(u) and f'(u).  SUMS: for dweight and dbias, which are fp32 whatever the inputs:
// library exp, and a reciprocal of one ulp (7 % of the one-pass gradient's time).
template <typename Tin, bool SUMS> __device__ __forceinline__ void act_fd(int act, float u, float &f, float &d) {
    if (act == 0) {
        f = u;
        d = 1.f;
        return;
    }
    const float p = SUMS ? rcpf_(1.f + expf(-u)) : sig<Tin>(u), r = p * (1.f - p);
    f = act == 1 ? u * p : p;
    d = act == 1 ? fmaf(u, r, p) : r;
}

// Sums of two values over the `tps` threads of a slab (tps a power of two, the
// slab's threads consecutive); more than a warp meet in shared memory.
__device__ __forceinline__ void slab_sum2(float &a, float &b, int tps) {
    for (int off = (tps < 32 ? tps : 32) >> 1; off > 0; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    if (tps > 32) {
        const int warp = threadIdx.x >> 5, per = tps >> 5, first = warp / per * per;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            smem[2 * warp] = a;
            smem[2 * warp + 1] = b;
        }
        __syncthreads();
        a = b = 0.f;
        for (int i = 0; i < per; ++i) {
            a += smem[2 * (first + i)];
            b += smem[2 * (first + i) + 1];
        }
    }
}

__device__ __forceinline__ float slab_sum(float a, int tps) {
    for (int off = (tps < 32 ? tps : 32) >> 1; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    if (tps > 32) {
        const int warp = threadIdx.x >> 5, per = tps >> 5, first = warp / per * per;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) smem[warp] = a;
        __syncthreads();
        a = 0.f;
        for (int i = 0; i < per; ++i) a += smem[first + i];
    }
    return a;
}

// ------------------------------------------------------------- held form
template <typename Tin, int VEC, int VPT>
struct HeldPlace {
    int g, sub;
    bool on;                         // this thread has a group
    long long off[VPT];              // element offset inside one n, -1: none
    int ch[VPT];
    __device__ __forceinline__ HeldPlace(const GroupNormParams &p, const GroupNormPlan &pl) {
        const int slab = threadIdx.x / pl.tps, lane = threadIdx.x % pl.tps;
        g = blockIdx.x * pl.gpc + slab % pl.gpc;
        sub = slab / pl.gpc;
        on = sub < pl.nsub && g < p.G;
        const int dv = p.D / VEC, nvec = p.L * dv;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int idx = i * pl.tps + lane, l = idx / dv;
            ch[i] = on && idx < nvec ? g * p.D + (idx - l * dv) * VEC : 0;
            off[i] = on && idx < nvec ? (long long)l * p.C + ch[i] : -1;
        }
    }
};

template <typename Tin, int VEC, int VPT, bool GATED>
__global__ void __launch_bounds__(kThreads)
gn_held_fwd_kernel(const GroupNormParams p, const GroupNormPlan pl) {
    const HeldPlace<Tin, VEC, VPT> at(p, pl);
    float w[VPT][VEC], b[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            w[i][j] = at.off[i] >= 0 && p.weight ? p.weight[at.ch[i] + j] : 1.f;
            b[i][j] = at.off[i] >= 0 && p.bias ? p.bias[at.ch[i] + j] : 0.f;
        }
    const long long row = (long long)p.L * p.C;
    const float inv = 1.f / ((float)p.L * (float)p.D);
    const Tin *x = static_cast<const Tin *>(p.x), *gate = static_cast<const Tin *>(p.gate);
    constexpr int PF = 1;                  // rows requested ahead: a second took the fourth block (90 -> 94 us)
    Vec<Tin, VEC> xq[PF][VPT], zq[PF][VPT];
    auto request = [&](int n, Vec<Tin, VEC> (&xr)[VPT], Vec<Tin, VEC> (&zr)[VPT]) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (at.off[i] >= 0 && n < p.N) {
                xr[i].load(x + n * row + at.off[i]);
                if (GATED) zr[i].load(gate + n * row + at.off[i]);
            }
    };
    const int step = gridDim.y * pl.nsub;
#pragma unroll
    for (int k = 0; k < PF; ++k) request(blockIdx.y * pl.nsub + at.sub + k * step, xq[k], zq[k]);
    auto one = [&](int n0, Vec<Tin, VEC> (&xr)[VPT], Vec<Tin, VEC> (&zr)[VPT]) {
        const int n = n0 + at.sub;
        const bool on = at.on && n < p.N;
        float v[VPT][VEC], z[VPT][VEC];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (at.off[i] >= 0 && on) {
                xr[i].get(v[i]);
                if (GATED) zr[i].get(z[i]);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] = z[i][j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += v[i][j];
        }
        request(n + PF * step, xr, zr);
        const float mean = slab_sum(sum, pl.tps) * inv;
        float m2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (at.off[i] >= 0) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    v[i][j] -= mean;
                    m2 = fmaf(v[i][j], v[i][j], m2);
                }
            }
        const float rstd = 1.f / sqrtf(fmaf(slab_sum(m2, pl.tps), inv, p.eps));
        if (!on) return;
        Tin *y = static_cast<Tin *>(p.y) + n * row;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (at.off[i] >= 0) {
                float o[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float u = fmaf(v[i][j] * rstd, w[i][j], b[i][j]);
                    o[j] = GATED ? u * act_f<Tin>(p.act, z[i][j]) : act_f<Tin>(p.act, u);
                }
                Vec<Tin, VEC>::put(y + at.off[i], o);
            }
        if (threadIdx.x % pl.tps == 0) {
            if (p.mean) p.mean[(size_t)n * p.G + at.g] = mean;
            if (p.rstd) p.rstd[(size_t)n * p.G + at.g] = rstd;
        }
    };
    for (int n0 = blockIdx.y * pl.nsub; n0 < p.N; n0 += PF * step) {
#pragma unroll
        for (int k = 0; k < PF; ++k)
            if (n0 + k * step < p.N) one(n0 + k * step, xq[k], zq[k]);       // (the same for the whole block)
    }
}

// Backward, L = 1.  Partial dw, db of block row y go to ws[y][2][C].
template <typename Tin, int VEC, int VPT, bool GATED>
__global__ void __launch_bounds__(kThreads)
gn_held_bwd_kernel(const GroupNormParams p, const GroupNormPlan pl) {
    const HeldPlace<Tin, VEC, VPT> at(p, pl);
    float w[VPT][VEC], b[VPT][VEC], dw[VPT][VEC], db[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            w[i][j] = at.off[i] >= 0 && p.weight ? p.weight[at.ch[i] + j] : 1.f;
            b[i][j] = at.off[i] >= 0 && p.bias ? p.bias[at.ch[i] + j] : 0.f;
            dw[i][j] = db[i][j] = 0.f;
        }
    const long long row = (long long)p.L * p.C;
    const float inv = 1.f / ((float)p.L * (float)p.D);
    const Tin *x = static_cast<const Tin *>(p.x), *gate = static_cast<const Tin *>(p.gate);
    const Tin *dy = static_cast<const Tin *>(p.dy);
    constexpr int PF = VPT == 1 ? 2 : 1;   // rows requested ahead
    Vec<Tin, VEC> xq[PF][VPT], zq[PF][VPT], dq[PF][VPT];
    float meanq[PF], rstdq[PF];
    auto request = [&](int n, Vec<Tin, VEC> (&xr)[VPT], Vec<Tin, VEC> (&zr)[VPT], Vec<Tin, VEC> (&dr)[VPT], float &mean_n,
                       float &rstd_n) {
        mean_n = rstd_n = 0.f;
        if (!at.on || n >= p.N) return;
        mean_n = p.mean[(size_t)n * p.G + at.g];
        rstd_n = p.rstd[(size_t)n * p.G + at.g];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (at.off[i] >= 0) {
                xr[i].load(x + n * row + at.off[i]);
                dr[i].load(dy + n * row + at.off[i]);
                if (GATED) zr[i].load(gate + n * row + at.off[i]);
            }
    };
    const int step = gridDim.y * pl.nsub;
#pragma unroll
    for (int k = 0; k < PF; ++k)
        request(blockIdx.y * pl.nsub + at.sub + k * step, xq[k], zq[k], dq[k], meanq[k], rstdq[k]);
    auto one = [&](int n0, Vec<Tin, VEC> (&xr)[VPT], Vec<Tin, VEC> (&zr)[VPT], Vec<Tin, VEC> (&dr)[VPT], float &mean_n,
                   float &rstd_n) {
        const int n = n0 + at.sub;
        const bool on = at.on && n < p.N;
        const float mean = mean_n, rstd = rstd_n;
        float h[VPT][VEC], dh[VPT][VEC], z[VPT][VEC];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (at.off[i] < 0 || !on) continue;
            xr[i].get(h[i]);
            dr[i].get(dh[i]);
            if (GATED) zr[i].get(z[i]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float hh = (h[i][j] - mean) * rstd, g = dh[i][j];
                const float u = fmaf(hh, w[i][j], b[i][j]);
                float f, d, du;
                if (GATED) {
                    act_fd<Tin, true>(p.act, z[i][j], f, d);
                    z[i][j] = g * u * d;
                    du = g * f;
                } else {
                    act_fd<Tin, true>(p.act, u, f, d);
                    du = g * d;
                }
                dw[i][j] = fmaf(du, hh, dw[i][j]);
                db[i][j] += du;
                const float e = du * w[i][j];
                s1 += e;
                s2 = fmaf(e, hh, s2);
                h[i][j] = hh;
                dh[i][j] = e;
            }
        }
        request(n + PF * step, xr, zr, dr, mean_n, rstd_n);
        slab_sum2(s1, s2, pl.tps);
        if (!on) return;
        s1 *= inv;
        s2 *= inv;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (at.off[i] >= 0) {
                if (p.dx) {
                    float o[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) o[j] = rstd * (dh[i][j] - s1 - h[i][j] * s2);
                    Vec<Tin, VEC>::put(static_cast<Tin *>(p.dx) + n * row + at.off[i], o);
                }
                if (GATED && p.dgate) Vec<Tin, VEC>::put(static_cast<Tin *>(p.dgate) + n * row + at.off[i], z[i]);
            }
    };
    for (int n0 = blockIdx.y * pl.nsub; n0 < p.N; n0 += PF * step) {
#pragma unroll
        for (int k = 0; k < PF; ++k)
            if (n0 + k * step < p.N) one(n0 + k * step, xq[k], zq[k], dq[k], meanq[k], rstdq[k]);
    }
    // the block's rows side by side (sub) meet in shared memory, in order
    float *mine = smem + 64 + threadIdx.x;
    const int next = pl.gpc * pl.tps;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            __syncthreads();
            mine[0] = dw[i][j];
            mine[kThreads] = db[i][j];
            __syncthreads();
            if (at.on && at.sub == 0 && at.off[i] >= 0) {
                float a = 0.f, c = 0.f;
                for (int k = 0; k < pl.nsub; ++k) {
                    a += mine[k * next];
                    c += mine[kThreads + k * next];
                }
                p.ws[((size_t)blockIdx.y * 2 + 0) * p.C + at.ch[i] + j] = a;
                p.ws[((size_t)blockIdx.y * 2 + 1) * p.C + at.ch[i] + j] = c;
            }
        }
}

// A sum that carries what its additions round off.  (Where it leaves the range of
// finite values it is what it is.)
struct LongSum {
    float s = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float t = s + x, v = t - s;
        lost += (s - (t - v)) + (x - v);
        s = t;
    }
    __device__ __forceinline__ float value() const { return fabsf(s) < INFINITY ? s + lost : s; }
};

// out[k][c] = sum over the `rows` partial rows ws[row][k][c], in a fixed order:
// 32 threads per channel, each every 32nd row; block = 32 channels.
constexpr int kSumThreads = 1024;
__device__ __forceinline__ void sum_rows(const float *ws, int rows, int C, float *dw, float *db, int block) {
    const int c = block * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    LongSum sa, sb;
    if (c < C) {
#pragma unroll 4
        for (int r = part; r < rows; r += 32) {
            sa.add(ws[((size_t)r * 2 + 0) * C + c]);
            sb.add(ws[((size_t)r * 2 + 1) * C + c]);
        }
    }
    smem[threadIdx.x] = sa.value();
    smem[kSumThreads + threadIdx.x] = sb.value();
    __syncthreads();
    if (part == 0 && c < C) {
        float a = 0.f, b = 0.f;
        for (int k = 0; k < 32; ++k) {
            a += smem[32 * k + threadIdx.x];
            b += smem[kSumThreads + 32 * k + threadIdx.x];
        }
        if (dw) dw[c] = a;
        if (db) db[c] = b;
    }
}
__global__ void __launch_bounds__(kSumThreads)
gn_sum_kernel(const float *ws, int rows, int C, float *dw, float *db) {
    sum_rows(ws, rows, C, dw, db, blockIdx.x);
}

// ------------------------------------------------------------- tiled form
// Block (x, y): vectors [y cvb, (y + 1) cvb) of the rows of tile x % tiles of
// slab row n = x / tiles.  Thread = (vector, row lane).
struct TilePlace {
    int n, l0, l1, cv, rl, lanes;
    // The last pass goes backwards: what the first read last is still in L2.
    __device__ __forceinline__ TilePlace(const GroupNormParams &p, const GroupNormPlan &pl, bool backwards = false) {
        const int x = backwards ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
        n = x / pl.tiles;
        const int tile = x % pl.tiles;
        l0 = tile * pl.rt;
        l1 = min(l0 + pl.rt, p.L);
        cv = blockIdx.y * pl.cvb + threadIdx.x % pl.cvb;
        rl = threadIdx.x / pl.cvb;
        lanes = kThreads / pl.cvb;
    }
};

// Sums of (a, b) over a column's row lanes, in its lane 0 (a tree).
__device__ __forceinline__ void lane_sum2(float &a, float &b, const TilePlace &at, int cvb) {
    for (int half = at.lanes >> 1; half > 0; half >>= 1) {
        __syncthreads();
        if (at.rl >= half && at.rl < 2 * half) {
            smem[threadIdx.x] = a;
            smem[kThreads + threadIdx.x] = b;
        }
        __syncthreads();
        if (at.rl < half) {
            a += smem[threadIdx.x + half * cvb];
            b += smem[kThreads + threadIdx.x + half * cvb];
        }
    }
}
// Joins nb values of mean mb and squared distances qb to na of (mean, m2); na + nb > 0.
__device__ __forceinline__ void join(float &mean, float &m2, float na, float mb, float qb, float nb) {
    const float w = nb / (na + nb), d = mb - mean;
    mean = na > 0.f ? fmaf(d, w, mean) : mb;
    m2 = na > 0.f ? m2 + fmaf(d, d * (na * w), qb) : qb;
}
// ws[(n * tiles + tile)][0][c] = mean, [1][c] = sum of squared distances from it.
template <typename Tin, int VEC>
__global__ void __launch_bounds__(kThreads, 4)
gn_tile_stats_kernel(const GroupNormParams p, const GroupNormPlan pl) {
    const TilePlace at(p, pl);
    const bool in = at.cv * VEC < p.C;
    const Tin *x = static_cast<const Tin *>(p.x) + (long long)at.n * p.L * p.C + (long long)at.cv * VEC;
    float mean[VEC], m2[VEC], cnt = 0.f;
#pragma unroll
    for (int j = 0; j < VEC; ++j) mean[j] = m2[j] = 0.f;
    if (in) {
        Vec<Tin, VEC> v[kRows];
        for (int l = at.l0 + at.rl; l < at.l1; l += kRows * at.lanes) {
            float rows = 0.f;
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                if (l + q * at.lanes >= at.l1) break;
                v[q].load(x + (long long)(l + q * at.lanes) * p.C);
                rows += 1.f;
            }
            float s[VEC], sq[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[j] = sq[j] = 0.f;
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                if (l + q * at.lanes >= at.l1) break;
                float f[VEC];
                v[q].get(f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[j] += f[j];
            }
            const float inv = 1.f / rows;
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                if (l + q * at.lanes >= at.l1) break;
                float f[VEC];
                v[q].get(f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float d = f[j] - s[j] * inv;
                    sq[j] = fmaf(d, d, sq[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) join(mean[j], m2[j], cnt, s[j] * inv, sq[j], rows);
            cnt += rows;
        }
    }
    // the row lanes meet two by two
    for (int half = at.lanes >> 1; half > 0; half >>= 1) {
        float *other = smem + 2 * kThreads;
        __syncthreads();
        if (at.rl >= half && at.rl < 2 * half) other[threadIdx.x] = cnt;
        __syncthreads();
        const float nb = at.rl < half ? other[threadIdx.x + half * pl.cvb] : 0.f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            __syncthreads();
            if (at.rl >= half && at.rl < 2 * half) {
                smem[threadIdx.x] = mean[j];
                smem[kThreads + threadIdx.x] = m2[j];
            }
            __syncthreads();
            if (nb > 0.f)
                join(mean[j], m2[j], cnt, smem[threadIdx.x + half * pl.cvb], smem[kThreads + threadIdx.x + half * pl.cvb], nb);
        }
        cnt += nb;
    }
    if (at.rl == 0 && in) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float *o = p.ws + (size_t)blockIdx.x * 2 * p.C + (size_t)at.cv * VEC + j;
            o[0] = mean[j];
            o[p.C] = m2[j];
        }
    }
}

// mean and rstd of (n, g) from the tiles' (mean, squared distances) per channel.
__global__ void __launch_bounds__(kThreads)
gn_tile_mean_kernel(const GroupNormParams p, const GroupNormPlan pl) {
    const int n = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const float *ws = p.ws + (size_t)n * pl.tiles * 2 * p.C + (size_t)g * p.D;
    const int items = pl.tiles * p.D;
    const float inv = 1.f / ((float)p.L * (float)p.D);
    LongSum sum;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int t = i / p.D, d = i - t * p.D;
        const float cnt = (float)(min((t + 1) * pl.rt, p.L) - t * pl.rt);
        sum.add(cnt * ws[(size_t)t * 2 * p.C + d]);
    }
    const float mean = slab_sum(sum.value(), kThreads) * inv;
    LongSum sq;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int t = i / p.D, d = i - t * p.D;
        const float cnt = (float)(min((t + 1) * pl.rt, p.L) - t * pl.rt);
        const float e = ws[(size_t)t * 2 * p.C + d] - mean;
        sq.add(fmaf(cnt * e, e, ws[((size_t)t * 2 + 1) * p.C + d]));
    }
    const float m2 = slab_sum(sq.value(), kThreads);
    if (threadIdx.x == 0) {
        p.mean[(size_t)n * p.G + g] = mean;
        p.rstd[(size_t)n * p.G + g] = 1.f / sqrtf(fmaf(m2, inv, p.eps));
    }
}

template <typename Tin, int VEC, bool GATED>
__global__ void __launch_bounds__(kThreads)
gn_tile_fwd_kernel(const GroupNormParams p, const GroupNormPlan pl) {
    const TilePlace at(p, pl, true);
    if (at.cv * VEC >= p.C) return;
    const long long base = (long long)at.n * p.L * p.C + (long long)at.cv * VEC;
    float w[VEC], b[VEC], m[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int c = at.cv * VEC + j;
        const size_t ng = (size_t)at.n * p.G + c / p.D;
        m[j] = p.mean[ng];
        w[j] = p.rstd[ng] * (p.weight ? p.weight[c] : 1.f);
        b[j] = p.bias ? p.bias[c] : 0.f;
    }
#pragma unroll 4
    for (int l = at.l0 + at.rl; l < at.l1; l += at.lanes) {
        Vec<Tin, VEC> v, zv;
        float f[VEC], z[VEC];
        const long long o = base + (long long)l * p.C;
        v.load(static_cast<const Tin *>(p.x) + o);
        if (GATED) zv.load(static_cast<const Tin *>(p.gate) + o);
        v.get(f);
        if (GATED) zv.get(z);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float u = fmaf(f[j] - m[j], w[j], b[j]);
            f[j] = GATED ? u * act_f<Tin>(p.act, z[j]) : act_f<Tin>(p.act, u);
        }
        Vec<Tin, VEC>::put(static_cast<Tin *>(p.y) + o, f);
    }
}

// Backward, first pass: ws[(n * tiles + tile)][0][c] = sum du h, [1][c] = sum du.
template <typename Tin, int VEC, bool GATED>
__global__ void __launch_bounds__(kThreads)
gn_tile_dsum_kernel(const GroupNormParams p, const GroupNormPlan pl) {
    const TilePlace at(p, pl);
    const bool in = at.cv * VEC < p.C;
    const long long base = (long long)at.n * p.L * p.C + (long long)at.cv * VEC;
    float w[VEC], b[VEC], m[VEC], r[VEC], sh[VEC], su[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int c = in ? at.cv * VEC + j : 0;
        const size_t ng = (size_t)at.n * p.G + c / p.D;
        m[j] = p.mean[ng];
        r[j] = p.rstd[ng];
        w[j] = p.weight ? p.weight[c] : 1.f;
        b[j] = p.bias ? p.bias[c] : 0.f;
        sh[j] = su[j] = 0.f;
    }
    if (in) {
        Vec<Tin, VEC> v[kRows], dv[kRows], zv[kRows];
        for (int l = at.l0 + at.rl; l < at.l1; l += kRows * at.lanes) {
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                const int r = l + q * at.lanes;
                if (r >= at.l1) break;
                const long long o = base + (long long)r * p.C;
                v[q].load(static_cast<const Tin *>(p.x) + o);
                dv[q].load(static_cast<const Tin *>(p.dy) + o);
                if (GATED) zv[q].load(static_cast<const Tin *>(p.gate) + o);
            }
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                if (l + q * at.lanes >= at.l1) break;
                float f[VEC], g[VEC], z[VEC];
                v[q].get(f);
                dv[q].get(g);
                if (GATED) zv[q].get(z);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float h = (f[j] - m[j]) * r[j];
                    float a, d;
                    act_fd<Tin, true>(p.act, GATED ? z[j] : fmaf(h, w[j], b[j]), a, d);
                    const float du = g[j] * (GATED ? a : d);
                    su[j] += du;
                    sh[j] = fmaf(du, h, sh[j]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        lane_sum2(sh[j], su[j], at, pl.cvb);
        if (at.rl == 0 && in) {
            float *o = p.ws + (size_t)blockIdx.x * 2 * p.C + (size_t)at.cv * VEC + j;
            o[0] = sh[j];
            o[p.C] = su[j];
        }
    }
}

// Blocks up to N * G: mean(dh), mean(dh h) of one (n, g), behind the partial sums
// in ws; the blocks behind them: dweight and dbias of 32 channels each.
__global__ void __launch_bounds__(kSumThreads)
gn_tile_gsum_kernel(const GroupNormParams p, const GroupNormPlan pl, float *out) {
    if ((long long)blockIdx.x >= (long long)p.N * p.G) {
        sum_rows(p.ws, p.N * pl.tiles, p.C, p.dweight, p.dbias, (int)(blockIdx.x - (unsigned)(p.N * p.G)));
        return;
    }
    const int n = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const float *ws = p.ws + (size_t)n * pl.tiles * 2 * p.C + (size_t)g * p.D;
    const int items = pl.tiles * p.D;
    LongSum t1, t2;
#pragma unroll 4
    for (int i = threadIdx.x; i < items; i += kSumThreads) {
        const int t = i / p.D, d = i - t * p.D;
        const float w = p.weight ? p.weight[g * p.D + d] : 1.f;
        t2.add(w * ws[(size_t)t * 2 * p.C + d]);
        t1.add(w * ws[((size_t)t * 2 + 1) * p.C + d]);
    }
    float s1 = t1.value(), s2 = t2.value();
    slab_sum2(s1, s2, kSumThreads);
    if (threadIdx.x == 0) {
        const float inv = 1.f / ((float)p.L * (float)p.D);
        out[2 * ((size_t)n * p.G + g)] = s1 * inv;
        out[2 * ((size_t)n * p.G + g) + 1] = s2 * inv;
    }
}

template <typename Tin, int VEC, bool GATED>
__global__ void __launch_bounds__(kThreads)
gn_tile_bwd_kernel(const GroupNormParams p, const GroupNormPlan pl, const float *gsum) {
    const TilePlace at(p, pl, true);
    if (at.cv * VEC >= p.C) return;
    const long long base = (long long)at.n * p.L * p.C + (long long)at.cv * VEC;
    float w[VEC], b[VEC], m[VEC], r[VEC], s1[VEC], s2[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int c = at.cv * VEC + j;
        const size_t ng = (size_t)at.n * p.G + c / p.D;
        m[j] = p.mean[ng];
        r[j] = p.rstd[ng];
        w[j] = p.weight ? p.weight[c] : 1.f;
        b[j] = p.bias ? p.bias[c] : 0.f;
        s1[j] = gsum[2 * ng];
        s2[j] = gsum[2 * ng + 1];
    }
    Vec<Tin, VEC> v[kRows], dv[kRows], zv[kRows];
    for (int l = at.l0 + at.rl; l < at.l1; l += kRows * at.lanes) {
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            const int row = l + q * at.lanes;
            if (row >= at.l1) break;
            const long long o = base + (long long)row * p.C;
            v[q].load(static_cast<const Tin *>(p.x) + o);
            dv[q].load(static_cast<const Tin *>(p.dy) + o);
            if (GATED) zv[q].load(static_cast<const Tin *>(p.gate) + o);
        }
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            const int row = l + q * at.lanes;
            if (row >= at.l1) break;
            const long long o = base + (long long)row * p.C;
            float f[VEC], g[VEC], z[VEC];
            v[q].get(f);
            dv[q].get(g);
            if (GATED) zv[q].get(z);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float h = (f[j] - m[j]) * r[j], u = fmaf(h, w[j], b[j]);
                float a, d;
                act_fd<Tin, false>(p.act, GATED ? z[j] : u, a, d);
                const float du = g[j] * (GATED ? a : d);
                if (GATED) z[j] = g[j] * u * d;
                f[j] = r[j] * (fmaf(du, w[j], -s1[j]) - h * s2[j]);
            }
            if (p.dx) Vec<Tin, VEC>::put(static_cast<Tin *>(p.dx) + o, f);
            if (GATED && p.dgate) Vec<Tin, VEC>::put(static_cast<Tin *>(p.dgate) + o, z);
        }
    }
}

constexpr size_t kHeldSmem = (64 + 2 * kThreads) * sizeof(float);
constexpr size_t kTileSmem = 3 * kThreads * sizeof(float);
constexpr size_t kSumSmem = 2 * kSumThreads * sizeof(float);

template <typename Tin, int VEC, int VPT>
cudaError_t launch_held_fwd(const GroupNormParams &p, const GroupNormPlan &pl, cudaStream_t s) {
    const dim3 grid((unsigned)pl.gx, (unsigned)pl.gy);
    if (p.gate) gn_held_fwd_kernel<Tin, VEC, VPT, true><<<grid, kThreads, kHeldSmem, s>>>(p, pl);
    else gn_held_fwd_kernel<Tin, VEC, VPT, false><<<grid, kThreads, kHeldSmem, s>>>(p, pl);
    return cudaGetLastError();
}

template <typename Tin, int VEC, int VPT>
cudaError_t launch_held(const GroupNormParams &p, const GroupNormPlan &pl, bool backward, cudaStream_t s) {
    if (!backward) return launch_held_fwd<Tin, VEC, VPT>(p, pl, s);
    const dim3 grid((unsigned)pl.gx, (unsigned)pl.gy);
    if (p.gate) gn_held_bwd_kernel<Tin, VEC, VPT, true><<<grid, kThreads, kHeldSmem, s>>>(p, pl);
    else gn_held_bwd_kernel<Tin, VEC, VPT, false><<<grid, kThreads, kHeldSmem, s>>>(p, pl);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p.dweight || p.dbias) {
        gn_sum_kernel<<<(p.C + 31) / 32, kSumThreads, kSumSmem, s>>>(p.ws, pl.gy, p.C, p.dweight, p.dbias);
        e = cudaGetLastError();
    }
    return e;
}

template <typename Tin, int VEC>
cudaError_t launch_tiled(const GroupNormParams &p, const GroupNormPlan &pl, bool backward, cudaStream_t s) {
    const dim3 grid((unsigned)pl.gx, (unsigned)pl.gy);
    if (!backward) {
        gn_tile_stats_kernel<Tin, VEC><<<grid, kThreads, kTileSmem, s>>>(p, pl);
        gn_tile_mean_kernel<<<p.N * p.G, kThreads, kTileSmem, s>>>(p, pl);
        if (p.gate) gn_tile_fwd_kernel<Tin, VEC, true><<<grid, kThreads, 0, s>>>(p, pl);
        else gn_tile_fwd_kernel<Tin, VEC, false><<<grid, kThreads, 0, s>>>(p, pl);
        return cudaGetLastError();
    }
    float *gsum = p.ws + (size_t)p.N * pl.tiles * 2 * p.C;
    if (p.gate) gn_tile_dsum_kernel<Tin, VEC, true><<<grid, kThreads, kTileSmem, s>>>(p, pl);
    else gn_tile_dsum_kernel<Tin, VEC, false><<<grid, kThreads, kTileSmem, s>>>(p, pl);
    const unsigned sums = p.dweight || p.dbias ? (unsigned)((p.C + 31) / 32) : 0u;
    gn_tile_gsum_kernel<<<(unsigned)(p.N * p.G) + sums, kSumThreads, kSumSmem, s>>>(p, pl, gsum);
    if (p.dx || p.dgate) {
        if (p.gate) gn_tile_bwd_kernel<Tin, VEC, true><<<grid, kThreads, 0, s>>>(p, pl, gsum);
        else gn_tile_bwd_kernel<Tin, VEC, false><<<grid, kThreads, 0, s>>>(p, pl, gsum);
    }
    return cudaGetLastError();
}

template <typename Tin, int VEC>
cudaError_t launch_vec(const GroupNormParams &p, const GroupNormPlan &pl, bool backward, cudaStream_t s) {
    if (!pl.held) return launch_tiled<Tin, VEC>(p, pl, backward, s);
    switch (pl.vpt) {
        case 1: return launch_held<Tin, VEC, 1>(p, pl, backward, s);
        case 2: return launch_held<Tin, VEC, 2>(p, pl, backward, s);
    }
    // a forward slab only: the backward's sums of four vectors would not stay in registers
    return launch_held_fwd<Tin, VEC, 4>(p, pl, s);
}

cudaError_t launch(const GroupNormParams &p, const GroupNormPlan &pl, bool bf16, bool backward, cudaStream_t s) {
    if (bf16)
        return pl.vec == 8 ? launch_vec<__nv_bfloat16, 8>(p, pl, backward, s)
                           : launch_vec<__nv_bfloat16, 1>(p, pl, backward, s);
    return pl.vec == 4 ? launch_vec<float, 4>(p, pl, backward, s) : launch_vec<float, 1>(p, pl, backward, s);
}

int pow2_at_least(int x) {
    int r = 1;
    while (r < x) r *= 2;
    return r;
}

}  // namespace

GroupNormPlan group_norm_plan(int N, int L, int C, int G, bool bf16, bool backward, bool aligned) {
    GroupNormPlan pl = {};
    const int D = C / G, full = bf16 ? 8 : 4;
    // blocks of 256 threads that are resident at once (registers allow four of the
    // forward, two of the backward) on the 148 SMs of the one device this is built for
    // -- a count asked of the current device could differ between the workspace's
    // query and the call: more blocks would only be more partial rows
    const long long slots = 148ll * (backward ? 2 : 4);
    // held: vectors lie inside a group
    const int hv = aligned && D % full == 0 ? full : 1;
    const long long nvec = (long long)L * D / hv;
    if (backward ? L == 1 && nvec <= 2 * kThreads : nvec <= 4 * kThreads) {
        pl.held = true;
        pl.vec = hv;
        pl.tps = pow2_at_least((int)nvec);
        if (pl.tps > kThreads) pl.tps = kThreads;
        pl.vpt = pow2_at_least((int)((nvec + pl.tps - 1) / pl.tps));
        const int spc = kThreads / pl.tps;
        pl.gx = (G + spc - 1) / spc;
        pl.gpc = (G + pl.gx - 1) / pl.gx;
        pl.nsub = spc / pl.gpc;
        const long long rows = ((long long)N + pl.nsub - 1) / pl.nsub;
        long long gy = slots / pl.gx;
        if (gy < 1) gy = 1;
        // no more than 4 kDepth rows one after another in the sums of dweight and dbias
        if (backward && gy < rows / (4 * kDepth)) gy = rows / (4 * kDepth);
        if (gy > 65535) gy = 65535;
        if (gy > rows) gy = rows;
        pl.gy = (int)gy;
        pl.ws_floats = backward ? (size_t)pl.gy * 2 * C : 0;
        return pl;
    }
    pl.vec = aligned && C % full == 0 ? full : 1;
    const int cv = (C + pl.vec - 1) / pl.vec;
    pl.cvb = cv < kThreads ? pow2_at_least(cv) : kThreads;
    pl.gy = (cv + pl.cvb - 1) / pl.cvb;
    const int lanes = kThreads / pl.cvb;
    // as many tiles as make one round of resident blocks, of 4 rows a thread or more;
    // no more than kDepth steps a thread (of kRows rows forward, of one backward)
    long long tiles = slots / ((long long)N * pl.gy);
    if (tiles > (L + 4 * lanes - 1) / (4 * lanes)) tiles = (L + 4 * lanes - 1) / (4 * lanes);
    const long long most = (long long)kDepth * (backward ? 1 : kRows) * lanes;
    if (tiles < (L + most - 1) / most) tiles = (L + most - 1) / most;
    pl.rt = (int)((L + tiles - 1) / tiles);
    pl.tiles = (L + pl.rt - 1) / pl.rt;
    pl.gx = N * pl.tiles;
    pl.ws_floats = (size_t)N * pl.tiles * 2 * C + (size_t)N * G * 2;
    return pl;
}

cudaError_t launch_group_norm_fwd(const GroupNormParams &p, const GroupNormPlan &pl, bool bf16, cudaStream_t s) {
    return launch(p, pl, bf16, false, s);
}
cudaError_t launch_group_norm_bwd(const GroupNormParams &p, const GroupNormPlan &pl, bool bf16, cudaStream_t s) {
    return launch(p, pl, bf16, true, s);
}

}  // namespace kda
