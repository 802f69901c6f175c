// kda_packed_fwd, chunk form on the tensor cores (tcgen05): bf16 activations,
// Dk = Dv = 128, one decay per (token, head), any decay g <= 0.
//
// With G the running sum of g inside a chunk of 64 tokens, r the L2 norm
// factors and S the state entering the chunk,
//
//     A_ij = beta_i r_i r_j (k_i . k_j) exp(G_i - G_j)     (j < i)
//     B_ij = scale rq_i r_j (q_i . k_j) exp(G_i - G_j)     (j <= i)
//     T = (I + A)^-1
//     P = [K ; Q] S
//     R_i = v_i - exp(G_i) r_i Pk_i,    U = T Diag(beta) R
//     O_i = scale exp(G_i) rq_i Pq_i + (B U)_i
//     S  <- exp(G_C) S + K^T Diag(r_j exp(G_C - G_j)) U
//
// Every exponent is a difference G_i - G_j <= 0 of one number per token, taken
// in two floats (head and tail of the running sum), so no decay is too strong:
// there is no anchor and no bound on g.
//
// Precision.  K and Q enter the products as they are given (bf16, unscaled:
// norms and decays are applied to rows of the fp32 results), so K K^T, Q K^T
// are exact products.  What is fp32 -- S, R, U and T Diag(beta) -- enters as
// three bf16 terms (head, middle, tail: 24 bits), six products of (order of
// magnitude) terms where both sides are split and three where K or Q is the
// other side; B and its U, which only reach the bf16 output, as two terms and
// three products.  The state therefore keeps fp32 accuracy over any number of
// chunks: it lives in fp32 registers, S = gamma S + dS with dS from the MMA.
//
// One CTA per SM walks (sequence, head) chains: 8 state warps (thread = value
// channel and half of the key channels; TMEM lane = value channel) run the
// serial part, 8 prep warps build T Diag(beta), B and the row factors of the
// next chunk meanwhile.  All MMAs are transposed (D = value channels x tokens
// or key channels), so S^T, R^T, U^T are A operands in TMEM and K, Q, T, B are
// B operands in shared memory; the K tile, loaded once by TMA with the 128-byte
// swizzle, serves K-major (P, K K^T) and MN-major (dS).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_packed.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int C = 64, D = 128;
constexpr int kStateThreads = 256, kPrepThreads = 256, kThreads = kStateThreads + kPrepThreads;
constexpr int LDA = 68;                    // row of the fp32 solve tiles
constexpr int kPage = 512;                 // sequences scheduled at a time

// Shared memory.
constexpr uint32_t KQ_BYTES = 32768;       // two blocks of 64 channels x [64 K rows | 64 Q rows] x 128 B
constexpr uint32_t OFF_KQ = 0;                                   // 2 stages
constexpr uint32_t OFF_V = OFF_KQ + 2 * KQ_BYTES;                // 2 x [64][128] bf16
constexpr uint32_t OFF_TB = OFF_V + 2 * 16384;                   // 2 x 3 terms of T Diag(beta), 64 x 64
constexpr uint32_t OFF_AQK = OFF_TB + 2 * 3 * 8192;              // 2 x 2 terms of B
constexpr uint32_t OFF_AKK = OFF_AQK + 2 * 2 * 8192;             // A, fp32
constexpr uint32_t OFF_T = OFF_AKK + C * LDA * 4;                // T and the solve's intermediates, fp32
constexpr uint32_t OFF_VEC = OFF_T + C * LDA * 4;                // 2 x {fk[64], fq[64], c[64], gamma}
constexpr uint32_t VEC_BYTES = 1024;
constexpr uint32_t OFF_PREP = OFF_VEC + 2 * VEC_BYTES;           // G head, G tail, r, rq, beta, norm parts
constexpr uint32_t OFF_SCHED = OFF_PREP + (5 * 64 + 256) * 4;    // begin, len, slot, order of a page
constexpr uint32_t OFF_MISC = OFF_SCHED + kPage * 16;
constexpr uint32_t SMEM_USED = OFF_MISC + 256;
constexpr uint32_t SMEM_BYTES = SMEM_USED + 1024;                // the base is rounded up to 1024
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");

enum { MB_KQ = 0, MB_V = 2, MB_READY = 4, MB_FREE = 6, MB_KK = 8, MB_S = 9, MB_O = 10, MB_DRAIN = 11, kNumBars = 12 };
constexpr uint32_t MISC_ABORT = 128, MISC_TMEM = 132, MISC_COUNT = 136;

// TMEM columns.
constexpr uint32_t COL_S = 0;              // S^T: 3 terms x 64; dS overwrites the first 128 once P is done,
constexpr uint32_t COL_U2 = 128;           // the two terms of U for O the rest
constexpr uint32_t COL_PK = 192;           // Pk^T, then U^T
constexpr uint32_t COL_PQ = 256;           // Pq^T, scaled in place, then O^T
constexpr uint32_t COL_R = 320;            // R^T: 3 terms x 32, then U'^T
constexpr uint32_t COL_KK = 416;           // [K ; Q] K^T of the next chunk
constexpr uint32_t TMEM_COLS = 512;

enum { BAR_STATE = 1, BAR_PREP = 2 };

__device__ unsigned int g_packed_chunk_error = 0;

struct PackedTcParams {
    PackedParams p;
    CUtensorMap tm[3];                     // k, q ([64][1][64], swizzled), v ([64][1][128])
};

extern __shared__ uint8_t smem_raw[];

struct Ctx {
    uint8_t *sm;
    uint32_t sbase, tm;
    volatile int *abort_flag;
};

__device__ __forceinline__ uint32_t bar_addr(const Ctx &x, int i) { return x.sbase + OFF_MISC + 8u * (uint32_t)i; }

// Waits are bounded in time; one that runs out sets the CTA's abort flag, which
// ends every other wait.
constexpr long long kWaitCycles = 4000000000ll;     // about two seconds
constexpr uint32_t kSuspendNs = 500000, kWaitTries = 4000;
__device__ __forceinline__ bool wait_bar(const Ctx &x, uint32_t mbar, uint32_t parity) {
    if (mbar_try_wait(mbar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(mbar, parity)) {
        if (*x.abort_flag) return false;
        if (clock64() - t0 > kWaitCycles) {
            *x.abort_flag = 1;
            return false;
        }
    }
    return true;
}

// ---- descriptors ------------------------------------------------------------
// MN-major operand in the 128-byte swizzle with `lbo` bytes from one block of
// 64 MN-elements to the next; k-step s (16 rows) starts 2048 s bytes in.
__device__ __forceinline__ uint64_t mn_desc(uint32_t base, uint32_t lbo, int s) {
    uint64_t d = mnmaj_desc(base, s);
    d &= ~((uint64_t)0x3FFFu << 16);
    return d | (uint64_t)(lbo >> 4) << 16;
}

// ---- splits -----------------------------------------------------------------
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// a, b as N bf16 terms each, rounded to nearest one after another: N = 3 leaves
// at most 2^-27 of the value, N = 2 2^-18.
template <int N>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&w)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w[i] = pack_bf16x2(a, b);
        if (i + 1 < N) {
            a -= bf_lo(w[i]);
            b -= bf_hi(w[i]);
        }
    }
}
// 32 consecutive columns of an operand row (v0, v1) as N terms at TMEM columns
// col, col + stride, ...
template <int N>
__device__ __forceinline__ void put_split(uint32_t taddr, uint32_t stride, const float (&v)[32]) {
    float w[N][16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        uint32_t t[N];
        split2<N>(v[2 * u], v[2 * u + 1], t);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i][u] = __uint_as_float(t[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) tmem_st16(taddr + (uint32_t)i * stride, w[i]);
}
__device__ __forceinline__ void get32(uint32_t taddr, float (&v)[32]) {
    float a[16], b[16];
    tmem_ld16x2(taddr, taddr + 16, a, b);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = a[i];
        v[16 + i] = b[i];
    }
}

// ---- schedule ---------------------------------------------------------------
// A page of sequences in shared memory: bounds and slot of each long live one,
// sorted by length, longest first.  Chains (rank, head) are dealt to the CTAs
// in rounds, every second round backwards, so that a CTA with a long chain gets
// a short one next.
struct Sched {
    int *begin, *len, *slot, *order;
    volatile int *count;
};
__device__ __forceinline__ Sched sched_of(uint8_t *sm) {
    Sched s;
    s.begin = reinterpret_cast<int *>(sm + OFF_SCHED);
    s.len = s.begin + kPage;
    s.slot = s.len + kPage;
    s.order = s.slot + kPage;
    s.count = reinterpret_cast<volatile int *>(sm + OFF_MISC + MISC_COUNT);
    return s;
}

// Fills the page that starts at sequence s0 (all threads of the CTA).
__device__ void fill_page(const PackedParams &p, const Sched &sc, int s0, int tid) {
    const int n = min(kPage, p.N - s0);
    for (int i = tid; i < n; i += kThreads) {
        const PackedSeq sq = packed_seq(p.cu, p.slots, p.T, p.P, s0 + i);
        if (sq.bad && blockIdx.x == 0) atomicOr(&g_packed_chunk_error, kPackedRange);
        sc.begin[i] = sq.begin;
        sc.len[i] = sq.bad ? 0 : sq.len;
        sc.slot[i] = sq.slot;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        bool live = sc.len[i] > p.split && sc.slot[i] >= 0;
        if (sc.slot[i] >= 0 && p.slots) {
            bool repeat = packed_repeat(p.slots, s0, sc.slot[i], 0, 1);
            for (int k = 0; k < i; ++k) repeat |= sc.slot[k] == sc.slot[i];
            if (repeat && blockIdx.x == 0) atomicOr(&g_packed_chunk_error, kPackedRange);
            live = live && !repeat;
        }
        sc.order[i] = live ? 1 : 0;
    }
    __syncthreads();
    // rank among the live ones: longer, or as long and earlier
    static_assert(kPage <= kThreads, "a thread ranks one sequence");
    const bool live = tid < n && sc.order[tid];
    int rank = 0, count = 0;
    if (live || tid == 0) {
        const int len = sc.len[tid];
        for (int k = 0; k < n; ++k) {
            if (!sc.order[k]) continue;
            ++count;
            rank += sc.len[k] > len || (sc.len[k] == len && k < tid);
        }
    }
    __syncthreads();
    if (live) sc.order[rank] = tid;
    if (tid == 0) *sc.count = count;
    __syncthreads();
}

// Walks the chunks of this CTA's chains of one page.
struct Cursor {
    int items, round;                      // chains of the page; next round to look at
    int n, chunks;                         // chunk of the chain
    int seq, begin, len, slot, hv;
    __device__ __forceinline__ void start(const PackedParams &p, const Sched &sc) {
        items = *sc.count * p.HV;
        round = 0;
        n = chunks = 0;
        next_chain(p, sc);
    }
    __device__ __forceinline__ bool valid() const { return n < chunks; }
    __device__ __forceinline__ void next_chain(const PackedParams &p, const Sched &sc) {
        n = chunks = 0;
        for (;; ++round) {
            const long long base = (long long)round * gridDim.x;
            if (base >= items) return;
            const long long i = base + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            if (i >= items) continue;
            ++round;
            seq = sc.order[(int)i / p.HV];
            hv = (int)i % p.HV;
            begin = sc.begin[seq];
            len = sc.len[seq];
            slot = sc.slot[seq];
            chunks = (len + C - 1) / C;
            return;
        }
    }
    __device__ __forceinline__ void next(const PackedParams &p, const Sched &sc) {
        if (++n >= chunks) next_chain(p, sc);
    }
};

// Loads of one chunk into its stage (one thread).
__device__ __forceinline__ void request(const PackedParams &p, const CUtensorMap *tm, const Ctx &x, const Cursor &c,
                                        int stage) {
    const int row = c.begin + c.n * C, h = c.hv / p.group;
    const uint32_t kq = x.sbase + OFF_KQ + (uint32_t)stage * KQ_BYTES, mb = bar_addr(x, MB_KQ + stage);
    mbar_arrive_expect_tx(mb, KQ_BYTES);
    tma_load_3d(kq, &tm[0], 0, h, row, mb);
    tma_load_3d(kq + 16384, &tm[0], 64, h, row, mb);
    tma_load_3d(kq + 8192, &tm[1], 0, h, row, mb);
    tma_load_3d(kq + 16384 + 8192, &tm[1], 64, h, row, mb);
    const uint32_t mv = bar_addr(x, MB_V + stage);
    mbar_arrive_expect_tx(mv, 16384);
    tma_load_3d(x.sbase + OFF_V + (uint32_t)stage * 16384u, &tm[2], 0, c.hv, row, mv);
}

// =====================================================================
// Prep role: warps 8-15.
// =====================================================================
__device__ __forceinline__ uint32_t tile_off(int r, int i) {      // 64 x 64 bf16, K-major, swizzled
    return (uint32_t)(r * 128 + (((i >> 3) ^ (r & 7)) << 4) + (i & 7) * 2);
}
// D (16 x 8) += A (16 x 8 KS) B (8 KS x 8), fp32 tiles in shared memory, each
// operand as tf32 head and tail: three products, the error of an fp32 product.
template <int KS>
__device__ __forceinline__ void warp_mm(float d[4], const float *A, const float *B, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        const float *a = A + g * LDA + 8 * kk + t;
        const float *b = B + (8 * kk + t) * LDA + g;
        const float av[4] = {a[0], a[8 * LDA], a[4], a[8 * LDA + 4]}, bv[2] = {b[0], b[4 * LDA]};
        uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ah[i] = to_tf32(av[i]);
            al[i] = to_tf32(av[i] - __uint_as_float(ah[i]));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bh[i] = to_tf32(bv[i]);
            bl[i] = to_tf32(bv[i] - __uint_as_float(bh[i]));
        }
        mma_tf32_16x8x8(d, al, bh);
        mma_tf32_16x8x8(d, ah, bl);
        mma_tf32_16x8x8(d, ah, bh);
    }
}
__device__ __forceinline__ void warp_put(float *Dst, const float d[4], float sgn, bool accumulate, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float2 *p0 = reinterpret_cast<float2 *>(Dst + g * LDA + 2 * t);
    float2 *p1 = reinterpret_cast<float2 *>(Dst + (g + 8) * LDA + 2 * t);
    float2 v0 = make_float2(sgn * d[0], sgn * d[1]), v1 = make_float2(sgn * d[2], sgn * d[3]);
    if (accumulate) {
        const float2 o0 = *p0, o1 = *p1;
        v0.x += o0.x; v0.y += o0.y; v1.x += o1.x; v1.y += o1.y;
    }
    *p0 = v0;
    *p1 = v1;
}
// -d (16 x 8, rows row0.., columns col0..) Diag(beta) as the three terms of T Diag(beta).
__device__ __forceinline__ void warp_tb(uint8_t *tb, int row0, int col0, const float d[4], const float *beta, int lane) {
    const int g = lane >> 2, t = lane & 3, c = col0 + 2 * t;
    const float b0 = -beta[c], b1 = -beta[c + 1];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t w[3];
        split2<3>(d[2 * half] * b0, d[2 * half + 1] * b1, w);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            *reinterpret_cast<uint32_t *>(tb + i * 8192 + tile_off(row0 + g + 8 * half, c)) = w[i];
    }
}

// One token's log-decay in log2 units, and its beta.
__device__ __forceinline__ void load_gate(const PackedParams &p, const Cursor &c, int t, float &z, float &b) {
    z = b = 0.f;
    if (c.n * C + t < c.len) {
        const long long row = c.begin + c.n * C + t;
        z = ld_act(static_cast<const __nv_bfloat16 *>(p.g) + row * p.ldg, c.hv);
        b = ld_act(static_cast<const __nv_bfloat16 *>(p.beta) + row * p.ldb, c.hv);
    }
}

__device__ __forceinline__ void prep_page(const PackedParams &p, const Ctx &x, const Sched &sc, int tid, int &gc) {
    uint8_t *sm = x.sm;
    const int lane = tid & 31, warp = tid >> 5;
    float *gh = reinterpret_cast<float *>(sm + OFF_PREP), *gl = gh + 64, *rk = gl + 64, *rq = rk + 64, *beta = rq + 64;
    float *part = beta + 64;               // [2][128]
    float *Akk = reinterpret_cast<float *>(sm + OFF_AKK), *Tm = reinterpret_cast<float *>(sm + OFF_T);

    Cursor cur;
    cur.start(p, sc);
    float z[2], b[2];                      // gate warp: tokens lane, lane + 32 of the next chunk
    if (warp == 7 && cur.valid())
        for (int u = 0; u < 2; ++u) load_gate(p, cur, lane + 32 * u, z[u], b[u]);
    for (; cur.valid(); ++gc) {
        const int stage = gc & 1, phase = (gc >> 1) & 1;
        const int Cc = min(C, cur.len - cur.n * C);
        uint8_t *kq = sm + OFF_KQ + (uint32_t)stage * KQ_BYTES;
        uint8_t *tb = sm + OFF_TB + (uint32_t)stage * 3 * 8192, *aqk = sm + OFF_AQK + (uint32_t)stage * 2 * 8192;
        float *vec = reinterpret_cast<float *>(sm + OFF_VEC + (uint32_t)stage * VEC_BYTES);
        // A wait that gives up leaves its thread running to the chunk's one vote,
        // where all return together; until then it issues nothing.
        bool ok = wait_bar(x, bar_addr(x, MB_KQ + stage), (uint32_t)phase);
        if (ok && gc >= 2) ok = wait_bar(x, bar_addr(x, MB_FREE + stage), (uint32_t)(((gc - 2) >> 1) & 1));
        if (Cc < C) {                      // rows behind the sequence: another's, or none
            for (int i = tid; i < (C - Cc) * 32; i += kPrepThreads) {
                const int r = Cc + i / 32, q = i % 32;           // 16 chunks of the K row, 16 of the Q row
                *reinterpret_cast<uint4 *>(kq + ((q >> 3) & 1) * 16384 + (q >> 4) * 8192 + r * 128 + (q & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            named_bar(BAR_PREP, kPrepThreads);
        }
        if (tid == 0 && ok) {              // [K ; Q] K^T
            const uint32_t kqa = x.sbase + OFF_KQ + (uint32_t)stage * KQ_BYTES;
            fence_after_sync();
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                mma_bf16(x.tm + COL_KK, kmaj_desc(kqa, 128, s), kmaj_desc(kqa, 128, s), idesc_bf16(128, 64), s > 0);
            mma_commit(bar_addr(x, MB_KK));
        }
        // Norms: thread = (row of [K ; Q], block of 64 channels).
        {
            const int r = tid & 127, blk = tid >> 7;
            float s0 = 0.f, s1 = 0.f;
            if (p.l2norm) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(kq + blk * 16384 + r * 128 + ((j ^ (r & 7)) << 4));
                    s0 = fmaf(bf_lo(w.x), bf_lo(w.x), s0);
                    s1 = fmaf(bf_hi(w.x), bf_hi(w.x), s1);
                    s0 = fmaf(bf_lo(w.y), bf_lo(w.y), s0);
                    s1 = fmaf(bf_hi(w.y), bf_hi(w.y), s1);
                    s0 = fmaf(bf_lo(w.z), bf_lo(w.z), s0);
                    s1 = fmaf(bf_hi(w.z), bf_hi(w.z), s1);
                    s0 = fmaf(bf_lo(w.w), bf_lo(w.w), s0);
                    s1 = fmaf(bf_hi(w.w), bf_hi(w.w), s1);
                }
            }
            part[blk * 128 + r] = s0 + s1;
        }
        // Gate warp: log-decays in log2 units, their running sum as head + tail.
        if (warp == 7) {
            const float ea = p.gate_in ? expf(p.A_log[cur.hv]) : 0.f;
            const float bias = p.gate_in && p.dt_bias ? p.dt_bias[cur.hv] : 0.f;
            float h[2], l[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = lane + 32 * u;
                float g = p.gate_in ? kda_gate(p.gate_in, z[u], bias, ea, p.g_min) : z[u];
                g *= kLog2E;
                // below 2^-150 a factor is 0 in fp32: a floor keeps the sums finite
                g = g < -1e4f ? -1e4f : g;
                h[u] = t < Cc ? g : 0.f;
                l[u] = 0.f;
                beta[t] = t < Cc ? (p.beta_sigmoid ? sigmoidf_(b[u]) : b[u]) : 0.f;
            }
            auto add = [](float &ah, float &al, float bh, float bl) {     // (ah, al) += (bh, bl)
                const float s = ah + bh, v = s - ah;
                const float e = (ah - (s - v)) + (bh - v) + al + bl;
                ah = s + e;
                al = e - (ah - s);
            };
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float oh = __shfl_up_sync(0xffffffffu, h[u], off), ol = __shfl_up_sync(0xffffffffu, l[u], off);
                    if (lane >= off) add(h[u], l[u], oh, ol);
                }
            }
            const float th = __shfl_sync(0xffffffffu, h[0], 31), tl = __shfl_sync(0xffffffffu, l[0], 31);
            add(h[1], l[1], th, tl);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                gh[lane + 32 * u] = h[u];
                gl[lane + 32 * u] = l[u];
            }
        }
        named_bar(BAR_PREP, kPrepThreads);
        if (tid < 128) {                   // row factors
            const int t = tid & 63;
            const float ss = part[tid] + part[128 + tid];
            const float r = p.l2norm ? (t < Cc ? 1.f / sqrtf(ss + p.l2_eps) : 0.f) : 1.f;
            const float e = ex2f_(gh[t] + gl[t]);
            if (tid < 64) {
                rk[t] = r;
                vec[t] = r * e;
                vec[128 + t] = r * ex2f_((gh[63] - gh[t]) + (gl[63] - gl[t]));
                if (t == 0) vec[192] = ex2f_(gh[63] + gl[63]);
            } else {
                rq[t] = r * p.scale;
                vec[64 + t] = r * p.scale * e;
            }
        }
        if (ok) ok = wait_bar(x, bar_addr(x, MB_KK), (uint32_t)(gc & 1));
        if (named_bar_any(BAR_PREP, kPrepThreads, !ok)) return;
        fence_after_sync();
        // A and B from the TMEM product: lane = row of [K ; Q], 32 columns per warp.
        {
            const int quad = warp & 3, half = warp >> 2, row = (quad & 1) * 32 + lane, j0 = 32 * half;
            if (!(half == 1 && (quad & 1) == 0)) {               // else wholly above the diagonal
                float v[32];
                get32(x.tm + ((uint32_t)(quad * 32) << 16) + COL_KK + (uint32_t)j0, v);
                const bool is_q = quad >= 2;
                const float hi = gh[row], lo = gl[row];
                const float f = is_q ? rq[row] : beta[row] * rk[row];
                const int last = is_q ? row : row - 1;           // last column that counts
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float e = ex2f_((hi - gh[j0 + j]) + (lo - gl[j0 + j]));
                    v[j] = j0 + j <= last ? v[j] * (f * rk[j0 + j]) * e : 0.f;
                }
                if (is_q) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        uint32_t w[4][2];
#pragma unroll
                        for (int i = 0; i < 4; ++i) split2<2>(v[j + 2 * i], v[j + 2 * i + 1], w[i]);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            *reinterpret_cast<uint4 *>(aqk + i * 8192 + tile_off(row, j0 + j)) =
                                make_uint4(w[0][i], w[1][i], w[2][i], w[3][i]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4 *>(Akk + row * LDA + j0 + j) =
                            make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                }
            }
        }
        fence_before_sync();
        named_bar(BAR_PREP, kPrepThreads);

        cur.next(p, sc);
        if (warp == 7 && cur.valid())      // in flight during the solve
            for (int u = 0; u < 2; ++u) load_gate(p, cur, lane + 32 * u, z[u], b[u]);

        // T = (I + A)^-1 by 16 x 16 blocks: the diagonal blocks first, the rest from
        // T_IJ = -T_II sum_{J<=K<I} A_IK T_KJ in three steps:
        //   (1) X10 = A10 T00, X32 = A32 T22, Xc = A_{23,01} T_{01,01} without its T10 term;
        //   (2) T10 = -T11 X10, T32 = -T33 X32, Xc[:, 0:16] -= Xc[:, 16:32] X10
        //       (the missing term A_{23,1} T10 equals -(A_{23,1} T11) X10);
        //   (3) T_{23,01} = -T_{23,23} Xc.
        // X10, X32 and Xc live above the diagonal of Tm.  (Substitution by blocks,
        // not powers of A: with keys alike the powers grow and cancel.)
        if (warp < 2) {
            const int blk = 2 * warp + (lane >> 4), j = lane & 15;
            const float *Ab = Akk + 16 * blk * LDA + 16 * blk;
            float xs[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) xs[r] = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                xs[i] = i == j ? 1.f : xs[i];                    // rows above j stay 0
#pragma unroll
                for (int r = i + 1; r < 16; ++r) xs[r] = fmaf(-Ab[r * LDA + i], xs[i], xs[r]);
            }
            const int col = 16 * blk + j;
            const float bj = beta[col];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                Tm[(16 * blk + r) * LDA + col] = xs[r];
                uint32_t w[3];
                split2<3>(xs[r] * bj, 0.f, w);
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    *reinterpret_cast<uint16_t *>(tb + i * 8192 + tile_off(16 * blk + r, col)) = (uint16_t)(w[i] & 0xFFFFu);
            }
        }
        named_bar(BAR_PREP, kPrepThreads);
        for (int task = warp; task < 12; task += 8) {
            const int blk = task >> 1, nh = (task & 1) * 8;
            const int arow = blk == 0 ? 16 : blk == 1 ? 48 : (blk == 2 || blk == 4) ? 32 : 48;
            const int kc = blk == 1 ? 32 : (blk == 2 || blk == 3) ? 16 : 0;
            const int drow = blk == 1 ? 32 : (blk == 3 || blk == 5) ? 16 : 0;
            const int dcol = blk == 0 ? 16 : (blk == 4 || blk == 5) ? 32 : 48;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            warp_mm<2>(d, Akk + arow * LDA + kc, Tm + kc * LDA + kc + nh, lane);
            warp_put(Tm + drow * LDA + dcol + nh, d, 1.f, false, lane);
        }
        named_bar(BAR_PREP, kPrepThreads);
        {
            const int task = warp >> 1, nh = (warp & 1) * 8;
            const int arow = task == 0 ? 16 : task == 1 ? 48 : 16 * (task - 2);
            const int acol = task == 0 ? 16 : 48;
            const int brow = task == 1 ? 32 : 0, bcol = task == 1 ? 48 : 16;
            const int drow = task == 0 ? 16 : task == 1 ? 48 : 16 * (task - 2);
            const int dcol = task == 0 ? 0 : 32;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            warp_mm<2>(d, Tm + arow * LDA + acol, Tm + brow * LDA + bcol + nh, lane);
            if (task != 0) warp_put(Tm + drow * LDA + dcol + nh, d, -1.f, task >= 2, lane);
            if (task < 2) warp_tb(tb, drow, dcol + nh, d, beta, lane);       // T10, T32
        }
        named_bar(BAR_PREP, kPrepThreads);
        {
            const int mt = warp >> 2, n0 = 8 * (warp & 3);
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            const float *A = Tm + (32 + 16 * mt) * LDA + 32, *B = Tm + 32 + n0;
            if (mt == 0) warp_mm<2>(d, A, B, lane);
            else warp_mm<4>(d, A, B, lane);
            warp_tb(tb, 32 + 16 * mt, n0, d, beta, lane);
        }
        fence_async_smem();
        named_bar(BAR_PREP, kPrepThreads);
        if (tid == 0) mbar_arrive(bar_addr(x, MB_READY + stage));
    }
}

// =====================================================================
// State role: warps 0-7.  Thread = (TMEM lane = value channel j, half hf).
// =====================================================================
struct StateRole {
    float S[64];                           // S[64 hf + i][j]
    uint32_t o[16];                        // the last chunk's outputs, token pairs, as bf16
    long long o_row;                       // their first row, and how many of the 64 count
    int o_count, o_hv;
};

__device__ __forceinline__ void store_o(const PackedParams &p, const StateRole &st, int hf, int j) {
    if (st.o_count == 0) return;
    // lanes exchange so that each writes two channels of one token of the pair
    const bool odd = j & 1;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + st.o_row * p.ldo + (long long)st.o_hv * D + (j & ~1);
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        const uint32_t mine = st.o[u];
        const uint32_t other = __float_as_uint(__shfl_xor_sync(0xffffffffu, __uint_as_float(mine), 1));
        const uint32_t w = odd ? (other >> 16) | (mine & 0xFFFF0000u) : (mine & 0xFFFFu) | (other << 16);
        const int t = 32 * hf + 2 * u + (odd ? 1 : 0);
        if (t < st.o_count) *reinterpret_cast<uint32_t *>(o + (long long)t * p.ldo) = w;
    }
}

__device__ __forceinline__ void load_state(const PackedParams &p, const Cursor &c, int s0, int hf, int j, float (&S)[64]) {
    const bool zero = p.fresh && p.fresh[s0 + c.seq];
    const float *src = p.pool + (((size_t)c.slot * p.HV + c.hv) * D + 64 * hf) * D + j;
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = zero ? 0.f : src[(size_t)i * D];
}
__device__ __forceinline__ void put_state(uint32_t tl, int hf, const float (&S)[64]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = S[32 * q + i];
        put_split<3>(tl + COL_S + (uint32_t)(32 * hf + 16 * q), 64, v);
    }
}

// Runs the page's chunks; `ph` counts the phases of MB_S, `requested` (thread 0)
// the chunks loaded.
__device__ __forceinline__ void state_page(const PackedParams &p, const CUtensorMap *tmaps, const Ctx &x,
                                           const Sched &sc, int s0, int tid, int &gc, uint32_t &ph, int &requested) {
    uint8_t *sm = x.sm;
    const int warp = tid >> 5, hf = warp >> 2, j = (warp & 3) * 32 + (tid & 31);
    const uint32_t tl = x.tm + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t id_p = idesc_bf16(128, 128), id_u = idesc_bf16(128, 64);
    const uint32_t id_s = idesc_bf16(128, 128, false, /*b_mn_major=*/true);

    Cursor cur, ahead;
    cur.start(p, sc);
    if (!cur.valid()) return;
    ahead = cur;
    if (tid == 0) {                        // two chunks in flight from the start
        for (int i = 0; i < 2 && ahead.valid(); ++i) {
            request(p, tmaps, x, ahead, (gc + i) & 1);
            ++requested;
            ahead.next(p, sc);
        }
    }
    StateRole st;
    st.o_count = 0;
    load_state(p, cur, s0, hf, j, st.S);
    put_state(tl, hf, st.S);
    tmem_st_wait();
    fence_before_sync();
    named_bar(BAR_STATE, kStateThreads);

    for (; cur.valid(); ++gc) {
        const int stage = gc & 1;
        const uint32_t phase = (uint32_t)((gc >> 1) & 1);
        const int Cc = min(C, cur.len - cur.n * C);
        const uint32_t kq = x.sbase + OFF_KQ + (uint32_t)stage * KQ_BYTES;
        const float *vec = reinterpret_cast<const float *>(sm + OFF_VEC + (uint32_t)stage * VEC_BYTES);
        // (waits that give up: as in prep_page)
        bool ok = wait_bar(x, bar_addr(x, MB_READY + stage), phase);
        if (tid == 0 && ok) {              // P^T = S^T [K ; Q]^T, small terms first
            fence_after_sync();
#pragma unroll
            for (int t = 2; t >= 0; --t)
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    mma_bf16_tmem_a(x.tm + COL_PK, x.tm + COL_S + (uint32_t)(64 * t + 8 * s), kmaj_desc(kq, 128, s), id_p,
                                    t < 2 || s > 0);
            mma_commit(bar_addr(x, MB_S));
        }
        store_o(p, st, hf, j);             // the previous chunk's
        if (ok) ok = wait_bar(x, bar_addr(x, MB_V + stage), phase);
        uint32_t vv[16];
        {
            const uint8_t *vt = sm + OFF_V + (uint32_t)stage * 16384u + (uint32_t)(32 * hf) * 256u + 2u * (uint32_t)j;
#pragma unroll
            for (int u = 0; u < 16; ++u)
                vv[u] = (uint32_t)*reinterpret_cast<const uint16_t *>(vt + 512 * u) |
                        (uint32_t)*reinterpret_cast<const uint16_t *>(vt + 512 * u + 256) << 16;
        }
        if (ok) ok = wait_bar(x, bar_addr(x, MB_S), ph);
        ph ^= 1u;
        fence_after_sync();
        {                                  // R^T = V^T - Pk^T Diag(fk)
            float v[32];
            get32(tl + COL_PK + (uint32_t)(32 * hf), v);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float vi = (i & 1) ? bf_hi(vv[i >> 1]) : bf_lo(vv[i >> 1]);
                v[i] = 32 * hf + i < Cc ? fmaf(-vec[32 * hf + i], v[i], vi) : 0.f;
            }
            put_split<3>(tl + COL_R + (uint32_t)(16 * hf), 32, v);
        }
        tmem_st_wait();
        fence_before_sync();
        named_bar(BAR_STATE, kStateThreads);
        if (tid == 0 && ok) {              // U^T = R^T (T Diag(beta))^T
            fence_after_sync();
            const uint32_t tb = x.sbase + OFF_TB + (uint32_t)stage * 3 * 8192;
            const int ra[6] = {2, 1, 0, 1, 0, 0}, ta[6] = {0, 1, 2, 0, 1, 0};
#pragma unroll
            for (int t = 0; t < 6; ++t)
#pragma unroll
                for (int s = 0; s < C / 16; ++s)
                    mma_bf16_tmem_a(x.tm + COL_PK, x.tm + COL_R + (uint32_t)(32 * ra[t] + 8 * s),
                                    kmaj_desc(tb + (uint32_t)ta[t] * 8192u, 64, s), id_u, t > 0 || s > 0);
            mma_commit(bar_addr(x, MB_S));
        }
        {                                  // meanwhile Pq^T Diag(fq), in place
            float v[32];
            get32(tl + COL_PQ + (uint32_t)(32 * hf), v);
            float a[16], b[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                a[i] = v[i] * vec[64 + 32 * hf + i];
                b[i] = v[16 + i] * vec[64 + 32 * hf + 16 + i];
            }
            tmem_st16(tl + COL_PQ + (uint32_t)(32 * hf), a);
            tmem_st16(tl + COL_PQ + (uint32_t)(32 * hf + 16), b);
        }
        if (ok) ok = wait_bar(x, bar_addr(x, MB_S), ph);
        ph ^= 1u;
        fence_after_sync();
        {                                  // U as two terms for O, Diag(c) U as three for dS
            float v[32];
            get32(tl + COL_PK + (uint32_t)(32 * hf), v);
            put_split<2>(tl + COL_U2 + (uint32_t)(16 * hf), 32, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= vec[128 + 32 * hf + i];
            put_split<3>(tl + COL_R + (uint32_t)(16 * hf), 32, v);
        }
        const float gamma = vec[192];
        tmem_st_wait();
        fence_before_sync();
        named_bar(BAR_STATE, kStateThreads);
        if (tid == 0 && ok) {              // dS^T = U'^T K, then O^T += U^T B^T
            fence_after_sync();
#pragma unroll
            for (int t = 2; t >= 0; --t)
#pragma unroll
                for (int s = 0; s < C / 16; ++s)
                    mma_bf16_tmem_a(x.tm + COL_S, x.tm + COL_R + (uint32_t)(32 * t + 8 * s), mn_desc(kq, 16384, s), id_s,
                                    t < 2 || s > 0);
            mma_commit(bar_addr(x, MB_S));
            const uint32_t aq = x.sbase + OFF_AQK + (uint32_t)stage * 2 * 8192;
            const int ua[3] = {1, 0, 0}, ba[3] = {0, 1, 0};
#pragma unroll
            for (int t = 0; t < 3; ++t)
#pragma unroll
                for (int s = 0; s < C / 16; ++s)
                    mma_bf16_tmem_a(x.tm + COL_PQ, x.tm + COL_U2 + (uint32_t)(32 * ua[t] + 8 * s),
                                    kmaj_desc(aq + (uint32_t)ba[t] * 8192u, 64, s), id_u, 1u);
            mma_commit(bar_addr(x, MB_O));
        }
        if (ok) ok = wait_bar(x, bar_addr(x, MB_S), ph);
        ph ^= 1u;
        fence_after_sync();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v[32];
            get32(tl + COL_S + (uint32_t)(64 * hf + 32 * q), v);
#pragma unroll
            for (int i = 0; i < 32; ++i) st.S[32 * q + i] = fmaf(gamma, st.S[32 * q + i], v[i]);
        }
        if (ok) ok = wait_bar(x, bar_addr(x, MB_O), (uint32_t)(gc & 1));
        fence_after_sync();
        {
            float v[32];
            get32(tl + COL_PQ + (uint32_t)(32 * hf), v);
#pragma unroll
            for (int u = 0; u < 16; ++u) st.o[u] = pack_bf16x2(v[2 * u], v[2 * u + 1]);
        }
        st.o_row = cur.begin + cur.n * C;
        st.o_count = Cc;
        st.o_hv = cur.hv;
        fence_before_sync();
        if (named_bar_any(BAR_STATE, kStateThreads, !ok)) return;
        if (tid == 0) {                    // every operand of this chunk has been read
            mbar_arrive(bar_addr(x, MB_FREE + stage));
            if (ahead.valid()) {
                request(p, tmaps, x, ahead, stage);
                ++requested;
                ahead.next(p, sc);
            }
        }
        const bool last = cur.n + 1 == cur.chunks;
        if (last) {
            float *dst = p.pool + (((size_t)cur.slot * p.HV + cur.hv) * D + 64 * hf) * D + j;
#pragma unroll
            for (int i = 0; i < 64; ++i) dst[(size_t)i * D] = st.S[i];
        }
        cur.next(p, sc);
        if (cur.valid()) {
            if (last) load_state(p, cur, s0, hf, j, st.S);
            fence_after_sync();
            put_state(tl, hf, st.S);
            tmem_st_wait();
            fence_before_sync();
            named_bar(BAR_STATE, kStateThreads);
        }
    }
    store_o(p, st, hf, j);
}

__global__ void __launch_bounds__(kThreads, 1)
packed_chunk_kernel(const __grid_constant__ PackedTcParams tp) {
    const PackedParams &p = tp.p;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5;
    Ctx x;
    x.sm = sm;
    x.sbase = smem_addr(sm);
    x.abort_flag = reinterpret_cast<volatile int *>(sm + OFF_MISC + MISC_ABORT);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_MISC + MISC_TMEM);
    if (warp == 0) {
        tmem_alloc(smem_addr(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) mbar_init(bar_addr(x, i), i == MB_DRAIN ? 2 : 1);
        *x.abort_flag = 0;
        fence_mbar_init();
    }
    // what lies above the diagonal of T Diag(beta) and B is never written again
    for (uint32_t i = tid; i < (OFF_AKK - OFF_TB) / 16; i += kThreads)
        *reinterpret_cast<uint4 *>(sm + OFF_TB + 16 * i) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    x.tm = *tmem_slot;

    const Sched sc = sched_of(sm);
    int gc = 0, requested = 0;             // chunks of this CTA so far: stages and phases go on over pages
    uint32_t ph = 0;
    for (int s0 = 0; s0 < p.N; s0 += kPage) {
        fill_page(p, sc, s0, tid);
        if (warp < kStateThreads / 32) state_page(p, tp.tm, x, sc, s0, tid, gc, ph, requested);
        else prep_page(p, x, sc, tid - kStateThreads, gc);
        __syncthreads();
        if (*x.abort_flag) break;
    }

    // TMEM is freed once every MMA issued is complete, and shared memory is left
    // once every load requested has landed, after an abort too (bounded).
    if (tid == 0 || tid == kStateThreads) {
        mma_commit(bar_addr(x, MB_DRAIN));
        for (uint32_t i = 0; i < kWaitTries; ++i)
            if (mbar_try_wait_suspend(bar_addr(x, MB_DRAIN), 0u, kSuspendNs)) break;
        for (int r = requested - 1; r >= 0 && r >= requested - 2; --r)
            for (int b : {MB_KQ, MB_V})
                for (uint32_t i = 0; i < kWaitTries; ++i)
                    if (mbar_try_wait_suspend(bar_addr(x, b + (r & 1)), (uint32_t)((r >> 1) & 1), kSuspendNs)) break;
    }
    fence_before_sync();
    __syncthreads();
    if (tid == 0 && *x.abort_flag) atomicOr(&g_packed_chunk_error, 1u);
    if (warp == 0) {
        fence_after_sync();
        tmem_dealloc(x.tm, TMEM_COLS);
    }
}

}  // namespace

bool packed_chunk_shape(const PackedParams &p, bool bf16) { return bf16 && p.Dk == D && p.Dv == D && p.g_per_head; }

bool packed_chunk_aligned(const PackedParams &p) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                        reinterpret_cast<uintptr_t>(p.v) | reinterpret_cast<uintptr_t>(p.o);
    return a % 16 == 0 && (p.ldq | p.ldk | p.ldv | p.ldo) % 8 == 0;
}

// Tensor map of [T][heads][128] bf16 rows `ld` elements apart, boxes of 64 rows
// of one head: 128 channels, or 64 in the 128-byte swizzle (MMA operand layout).
static cudaError_t make_map(CUtensorMap *map, const void *base, int heads, long long rows, long long ld, bool swizzle) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    if (!encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {(cuuint32_t)(swizzle ? 64 : D), 1, (cuuint32_t)C};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_packed_chunk(const PackedParams &p, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(packed_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    if (e != cudaSuccess) return e;
    PackedTcParams tp;
    tp.p = p;
    if ((e = make_map(&tp.tm[0], p.k, p.H, p.T, p.ldk, true)) != cudaSuccess) return e;
    if ((e = make_map(&tp.tm[1], p.q, p.H, p.T, p.ldq, true)) != cudaSuccess) return e;
    if ((e = make_map(&tp.tm[2], p.v, p.HV, p.T, p.ldv, false)) != cudaSuccess) return e;
    const long long chains = (long long)p.N * p.HV;
    packed_chunk_kernel<<<(unsigned)(chains < sms ? chains : sms), kThreads, SMEM_BYTES, s>>>(tp);
    return cudaGetLastError();
}

cudaError_t read_and_clear_packed_chunk_error(unsigned int *out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_packed_chunk_error, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_packed_chunk_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
