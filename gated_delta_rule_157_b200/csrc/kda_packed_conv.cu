// kda_packed_conv: the layer prologue's causal short convolution over packed
// sequences, the window of each (its last K - 1 rows) in a pool of slots.
//
//     u[t] = bias + sum_j w[j] x[t - (K-1) + j],  y = u * sigmoid(u),  y / |y|_head
//
// A lane owns 8 channels and walks a run of rows with the last four in a ring of
// registers (four rows unrolled, so that no row is moved), so every row of x
// is read once (and K - 1 rows again where a run begins); a warp covers 256
// channels, 16 lanes a head of 128.  Rows before a sequence's first come from its
// slot.  The run that holds a sequence's first row also does the K - 2 rows behind
// it and writes the slot's new window, after its own read of the old one: nobody
// else reads the slot.
//
// 16391 rows of 4096 channels take 74 us on the device, 3.6 TB/s of 6.55: two special
// functions a value (that unit 46 % busy, issue slots 49 %) at the 16 warps an SM that
// 128 registers allow.  A run is as long as leaves 16 warps an SM (of the 148 of the
// one device this is built for), 32 rows at most: a short run reads K - 1 rows again.
#include "kda_packed.cuh"

namespace kda {
namespace {

__device__ unsigned int g_packed_conv_error = 0;

constexpr int kThreads = 128;

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

// u * sigmoid(u): library exp and division in fp32; for bf16 rows the hardware
// approximations, off by 2^-21 of the value near 0 and by 2^-18 at |u| = 88 (the product
// by log2 e is rounded), which vanishes in the output's rounding to 8 bits.
__device__ __forceinline__ float silu_for(const float *, float u) { return u / (1.f + expf(-u)); }
__device__ __forceinline__ float silu_for(const __nv_bfloat16 *, float u) { return u * rcpf_(1.f + ex2f_(-kLog2E * u)); }

// Where to begin looking for the sequences of `row` and of those behind it: the last
// that begins at or before it.  Where bounds run backwards that is no answer: all
// sequences are looked at then.  (Eight bounds a lane in one round; whatever a warp
// does for a sequence reads all slots once, so reading all bounds once costs little.)
__device__ __forceinline__ int find_sequence(const int *cu, int n, int row, int lane, bool &backwards) {
    int count = 0;
    bool down = false;
    for (int i0 = 0; i0 < n; i0 += 256) {
        int a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + 32 * k + lane;
            a[k] = i < n ? cu[i] : 0x7FFFFFFF;
            b[k] = i < n ? cu[i + 1] : 0x7FFFFFFF;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i0 + 32 * k < n) {
                count += __popc(__ballot_sync(0xffffffffu, a[k] <= row));
                down |= b[k] < a[k];
            }
    }
    backwards = __any_sync(0xffffffffu, down);
    return backwards || count == 0 ? 0 : count - 1;
}

// kAhead: rows done together, and requested ahead: 4, or 1 where runs are single rows.
template <typename Tin, int K, int kAhead>
__global__ void __launch_bounds__(kThreads, sizeof(Tin) == 2 ? 4 : 1)
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
    float2 w[K][4], bias[4];               // channel pairs
    {
        const float *wc = p.w + (size_t)c * K;
        float wf[8 * K];
        if (reinterpret_cast<uintptr_t>(p.w) % 16 == 0) {        // 8 K floats from a multiple of 8 K
#pragma unroll
            for (int i = 0; i < 2 * K; ++i) {
                const float4 f = c_ok ? *reinterpret_cast<const float4 *>(wc + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
                wf[4 * i] = f.x; wf[4 * i + 1] = f.y; wf[4 * i + 2] = f.z; wf[4 * i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8 * K; ++i) wf[i] = c_ok ? wc[i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][i] = make_float2(wf[2 * i * K + j], wf[(2 * i + 1) * K + j]);
            bias[i] = make_float2(0.f, 0.f);
        }
        if (c_ok && p.bias) {
            if (reinterpret_cast<uintptr_t>(p.bias) % 16 == 0) {
                const float4 b0 = *reinterpret_cast<const float4 *>(p.bias + c);
                const float4 b1 = *reinterpret_cast<const float4 *>(p.bias + c + 4);
                bias[0] = make_float2(b0.x, b0.y); bias[1] = make_float2(b0.z, b0.w);
                bias[2] = make_float2(b1.x, b1.y); bias[3] = make_float2(b1.z, b1.w);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) bias[i] = make_float2(p.bias[c + 2 * i], p.bias[c + 2 * i + 1]);
            }
        }
    }

    bool backwards = false;
    for (int s = p.cu ? find_sequence(p.cu, p.N, r0, lane, backwards) : r0; s < p.N; ++s) {
        const PackedSeq sq = packed_seq(p.cu, p.slots, p.T, p.P, s);
        if (sq.bad || sq.len == 0) continue;
        const int b = sq.begin, e = b + sq.len;
        if (b >= r1) {
            if (backwards) continue;
            break;
        }
        int row = b > r0 ? b : r0;
        if (row > b && row < b + W) row = b + W < e ? b + W : e;      // the run with row b does these
        const int own = b >= r0 && b + W > r1 ? b + W : r1;
        const int end = e < own ? e : own;
        if (row >= end) continue;
        Raw8<Tin> ahead[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            ahead[u].zero();
            if (c_ok && row + u < end) ahead[u].load(x + (long long)(row + u) * p.ldx);
        }
        const bool zero = p.fresh && p.fresh[s];
        const bool repeat = __any_sync(0xffffffffu, packed_repeat(p.cu, p.slots, s, sq.slot, lane, 32));
        if (repeat) {
            if (row == b && lane == 0) atomicOr(&g_packed_conv_error, kPackedRange);
            continue;
        }
        if (sq.slot < 0) continue;

        // ring[(u - i) & 3]: the row i before row u of a block of four; the window before `row`
        Tin *slot = static_cast<Tin *>(p.pool) + (size_t)sq.slot * W * p.C + c;
        float2 ring[4][4];
        Raw8<Tin> raw[W > 0 ? W : 1];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int t = row - W + j;
            raw[j].zero();
            if (c_ok) {
                if (t >= b) raw[j].load(x + (long long)t * p.ldx);
                else if (!zero) raw[j].load(slot + (size_t)(t - b + W) * p.C);
            }
            float f[8];
            raw[j].get(f);
#pragma unroll
            for (int i = 0; i < 4; ++i) ring[(4 - W + j) & 3][i] = make_float2(f[2 * i], f[2 * i + 1]);
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

        // Four rows at a time, step by step for all four: their chains of special
        // functions and shuffles overlap.
        for (; row < end; row += kAhead) {
            float2 f[kAhead][4];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                float cur[8];
                ahead[u].get(cur);
#pragma unroll
                for (int i = 0; i < 4; ++i) ring[u][i] = make_float2(cur[2 * i], cur[2 * i + 1]);
                if (c_ok && row + u + kAhead < end) ahead[u].load(x + (long long)(row + u + kAhead) * p.ldx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[u][i] = bias[i];
#pragma unroll
                    for (int j = 0; j < K; ++j) f[u][i] = __ffma2_rn(w[j][i], ring[(u + 4 - W + j) & 3][i], f[u][i]);
                }
            }
            if (p.silu) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[u][i].x = silu_for(static_cast<Tin *>(nullptr), f[u][i].x);
                        f[u][i].y = silu_for(static_cast<Tin *>(nullptr), f[u][i].y);
                    }
            }
            if (p.head_dim) {
                float ss[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    float2 q = __fmul2_rn(f[u][0], f[u][0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) q = __ffma2_rn(f[u][i], f[u][i], q);
                    ss[u] = q.x + q.y;
                }
#pragma unroll
                for (int off = 8; off > 0; off >>= 1)
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], off);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const float r = rsqrtf(ss[u] + p.l2_eps);
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[u][i] = __fmul2_rn(f[u][i], make_float2(r, r));
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (c_ok && row + u < end) {
                    const float out[8] = {f[u][0].x, f[u][0].y, f[u][1].x, f[u][1].y,
                                          f[u][2].x, f[u][2].y, f[u][3].x, f[u][3].y};
                    Raw8<Tin> o;
                    o.set(out);
                    o.store(y + (long long)(row + u) * p.ldy);
                }
            if (kAhead == 1) {             // no ring to come round: the rows move
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ring[1][i] = ring[2][i];
                    ring[2][i] = ring[3][i];
                    ring[3][i] = ring[0][i];
                }
            }
        }
    }
}

template <typename Tin, int K>
cudaError_t launch_taps(const PackedConvParams &p, int run, cudaStream_t s) {
    const long long warps = ((long long)p.T + run - 1) / run * ((p.C + 255) / 256);
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    if (run == 1) packed_conv_kernel<Tin, K, 1><<<grid, kThreads, 0, s>>>(p, run);
    else packed_conv_kernel<Tin, K, 4><<<grid, kThreads, 0, s>>>(p, run);
    return cudaGetLastError();
}
template <typename Tin>
cudaError_t launch_type(const PackedConvParams &p, int run, cudaStream_t s) {
    switch (p.K) {
        case 1: return launch_taps<Tin, 1>(p, run, s);
        case 2: return launch_taps<Tin, 2>(p, run, s);
        case 3: return launch_taps<Tin, 3>(p, run, s);
    }
    return launch_taps<Tin, 4>(p, run, s);
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
