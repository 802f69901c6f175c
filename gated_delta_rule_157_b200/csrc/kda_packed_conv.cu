// kda_packed_conv: the layer prologue's causal short convolution over packed
// sequences, the window of each (its last K - 1 rows) in a pool of slots.
//
//     u[t] = bias + sum_j w[j] x[t - (K-1) + j],  y = u * sigmoid(u),  y / |y|_head
//
// A lane owns 8 channels and walks a run of rows with the window in registers,
// so every row of x is read once (and K - 1 rows again where a run begins); a
// warp covers 256 channels, 16 lanes a head of 128.  Rows before a sequence's
// first come from its slot.  The run that holds a sequence's first row also
// does the K - 2 rows behind it and writes the slot's new window, after its
// own read of the old one: nobody else reads the slot.
#include "kda_packed.cuh"

namespace kda {
namespace {

__device__ unsigned int g_packed_conv_error = 0;

constexpr int kThreads = 128;
constexpr int kAhead = 4;                  // rows requested ahead of the one computed

// Eight channels as they lie in memory, and in fp32.
template <typename Tin> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = r; }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const unsigned u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        unsigned u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&u[i], &b, 4);
        }
        r = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void store(float *p) const {
        *reinterpret_cast<float4 *>(p) = a;
        *reinterpret_cast<float4 *>(p + 4) = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// exp for SiLU: the library function in fp32; for bf16 rows the hardware
// approximation, whose error (below 2^-20 here) vanishes in the rounding.
__device__ __forceinline__ float exp_for(const float *, float x) { return expf(x); }
__device__ __forceinline__ float exp_for(const __nv_bfloat16 *, float x) { return __expf(x); }

template <typename Tin, int K>
__global__ void __launch_bounds__(kThreads)
packed_conv_kernel(const PackedConvParams p, int run) {
    constexpr int W = K - 1;
    const int lane = threadIdx.x & 31;
    const int nchunk = (p.C + 255) / 256;
    const long long wid = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int c = (int)(wid % nchunk) * 256 + 8 * lane;
    const bool c_ok = c < p.C;             // lanes behind the last channel still vote
    const long long r0l = wid / nchunk * run;

    if (wid == 0) {                        // bounds and slots of every sequence
        for (int s = lane; s < p.N; s += 32) {
            const PackedSeq sq = packed_seq(p.cu, p.slots, p.T, p.P, s);
            if (sq.bad) atomicOr(&g_packed_conv_error, kPackedRange);
        }
    }
    if (r0l >= p.T) return;
    const int r0 = (int)r0l, r1 = p.T - r0 < run ? p.T : r0 + run;

    const Tin *x = static_cast<const Tin *>(p.x) + c;
    Tin *y = static_cast<Tin *>(p.y) + c;
    float w[K][8], bias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = c_ok ? p.w[(size_t)(c + i) * K + j] : 0.f;
        bias[i] = c_ok && p.bias ? p.bias[c + i] : 0.f;
    }

    // the last sequence that begins at or before r0
    int lo = 0, hi = p.N - 1;
    while (p.cu && lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu[mid] <= r0) lo = mid; else hi = mid - 1;
    }
    if (!p.cu) lo = r0;
    for (int s = lo; s < p.N; ++s) {
        const PackedSeq sq = packed_seq(p.cu, p.slots, p.T, p.P, s);
        if (sq.bad || sq.len == 0) continue;
        const int b = sq.begin, e = b + sq.len;
        if (b >= r1) break;
        int row = b > r0 ? b : r0;
        if (row > b && row < b + W) row = b + W < e ? b + W : e;      // the run with row b does these
        const int own = b >= r0 && b + W > r1 ? b + W : r1;
        const int end = e < own ? e : own;
        if (row >= end) continue;
        const bool repeat = __any_sync(0xffffffffu, packed_repeat(p.slots, s, sq.slot, lane, 32));
        if (repeat) {
            if (row == b && lane == 0) atomicOr(&g_packed_conv_error, kPackedRange);
            continue;
        }
        if (sq.slot < 0) continue;

        // window before `row`
        Tin *slot = static_cast<Tin *>(p.pool) + (size_t)sq.slot * W * p.C + c;
        const bool zero = p.fresh && p.fresh[s];
        float win[W > 0 ? W : 1][8];
        Raw8<Tin> raw[W > 0 ? W : 1];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int t = row - W + j;
            raw[j].zero();
            if (c_ok) {
                if (t >= b) raw[j].load(x + (long long)t * p.ldx);
                else if (!zero) raw[j].load(slot + (size_t)(t - b + W) * p.C);
            }
            raw[j].get(win[j]);
        }
        if (row == b) {                    // raw holds the whole old window
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int at = sq.len - W + j;
                Raw8<Tin> n;
                n.zero();
                if (at >= 0) {
                    if (c_ok) n.load(x + (long long)(b + at) * p.ldx);
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        if (i == at + W) n = raw[i];
                }
                if (c_ok) n.store(slot + (size_t)j * p.C);
            }
        }

        Raw8<Tin> ahead[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            ahead[u].zero();
            if (c_ok && row + u < end) ahead[u].load(x + (long long)(row + u) * p.ldx);
        }
        for (; row < end; row += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                float cur[8], f[8];
                ahead[u].get(cur);
                if (c_ok && row + u + kAhead < end) ahead[u].load(x + (long long)(row + u + kAhead) * p.ldx);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float a = fmaf(w[K - 1][i], cur[i], bias[i]);
#pragma unroll
                    for (int j = 0; j < W; ++j) a = fmaf(w[j][i], win[j][i], a);
                    f[i] = a;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j) win[j][i] = win[j + 1][i];
                    if (W > 0) win[W > 0 ? W - 1 : 0][i] = cur[i];
                }
                if (p.silu) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = f[i] / (1.f + exp_for(static_cast<Tin *>(nullptr), -f[i]));
                }
                if (p.head_dim) {
                    float q = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) q = fmaf(f[i], f[i], q);
#pragma unroll
                    for (int off = 8; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
                    const float r = 1.f / sqrtf(q + p.l2_eps);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= r;
                }
                if (c_ok && row + u < end) {
                    Raw8<Tin> o;
                    o.set(f);
                    o.store(y + (long long)(row + u) * p.ldy);
                }
            }
        }
    }
}

template <typename Tin>
cudaError_t launch_type(const PackedConvParams &p, int run, cudaStream_t s) {
    const long long warps = ((long long)p.T + run - 1) / run * ((p.C + 255) / 256);
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    switch (p.K) {
        case 1: packed_conv_kernel<Tin, 1><<<grid, kThreads, 0, s>>>(p, run); break;
        case 2: packed_conv_kernel<Tin, 2><<<grid, kThreads, 0, s>>>(p, run); break;
        case 3: packed_conv_kernel<Tin, 3><<<grid, kThreads, 0, s>>>(p, run); break;
        default: packed_conv_kernel<Tin, 4><<<grid, kThreads, 0, s>>>(p, run); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_conv(const PackedConvParams &p, bool bf16, cudaStream_t s) {
    int run = 1;
    while (run < 32 && (long long)p.T / (2 * run) * ((p.C + 255) / 256) >= 148 * 16) run *= 2;
    return bf16 ? launch_type<__nv_bfloat16>(p, run, s) : launch_type<float>(p, run, s);
}

cudaError_t read_and_clear_packed_conv_error(unsigned int *out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_packed_conv_error, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_packed_conv_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
