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
// are exact products.  What is fp32 -- S, R, U, U' = Diag(c) U, T Diag(beta), B --
// enters as the sum of three bf16 terms (head, middle, tail: 24 bits).  S and U' meet
// K or Q, which have one term: theirs are cut off one after another, and nothing is
// left over.  Where both sides are split the terms are rounded, which leaves the
// smallest middle and tail, and the six products of the larger orders are taken; what
// is left out is 2^-26 of a product.  The state itself lives in fp32 registers, S =
// gamma S + dS with dS from the MMA.  Simulated over 16 chunks the splits leave the
// state off by 5e-8 to 7e-8 of its norm (an fp32 recurrence on the same inputs by
// 5e-7), and 1 in 10^4 of the bf16 outputs differs from the rounded exact one.  Two
// terms of S would leave 1.3e-6 with hardly any decay, two of S, B and the U of O 3
// outputs in 10^3, for 0.75 ms instead of 0.81 on 32768 rows x 32 heads.
//
// One CTA per SM walks (sequence, head) chains, longest first.  8 state warps
// (thread = value channel = TMEM lane, and half of the key channels) run the
// serial part; two groups of 4 prep warps build T Diag(beta), B and the row
// factors of the chunks ahead, one the even, the other the odd chunks, so that
// each has two chunks' time for its chain of small dependent steps; a warp each
// evaluates their gates; one warp, the oldest, issues every load and MMA.  All
// MMAs are transposed (D = value channels x tokens or key channels), so S^T,
// R^T, U^T are A operands in TMEM and K, Q, T, B are B operands in shared memory;
// the K tile, loaded once by TMA with the 128-byte swizzle, serves K-major (P,
// K K^T) and MN-major (dS).  Operand terms replace the accumulator columns that
// the same thread has just read, so the state warps meet only at the mbarriers
// of the issuing warp.
//
// What bounds it: the chain of one chunk, about 11,500 cycles: what is left of P 700,
// O of the chunk before 800 and its stores 1,000, R 1,900, U 1,700, its terms for dS
// 1,100, dS 1,500, S and its terms 1,300, their stores 1,300 (the MMAs and the warps'
// TMEM accesses slow each other).  The tensor pipe is 35 % busy, issue slots 47 %, DRAM
// 12 %.  32768 rows x 32 heads in 4 sequences: 0.76 to 0.82 ms, 1.0 TB/s.  What shortened it: shared-memory addresses formed without a
// trip through an integer (accesses had become generic ones, and registers
// spilled), a warp that only issues, gates off the prep groups' path, no barrier
// among the state warps, U' before U.  Measured and not kept: 4 state warps of whole
// rows, 32-column TMEM accesses (registers spill), P for Q beside the split of U,
// the next K and Q requested behind P instead of ahead of it.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_packed.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int C = 64, D = 128;
constexpr int kStateThreads = 256, kPrepThreads = 256, kThreads = kStateThreads + kPrepThreads + 128;
constexpr int kStateWarps = kStateThreads / 32;
constexpr int kFirstState = 128, kFirstPrep = kFirstState + kStateThreads;     // threads below: the issuing warpgroup
constexpr int kGroup = 128;                // threads of a prep group
constexpr int LDA = 68;                    // row of the fp32 solve tiles
constexpr int kPage = 128;                 // sequences scheduled at a time

// Shared memory.
constexpr uint32_t KQ_BYTES = 32768;       // two blocks of 64 channels x [64 K rows | 64 Q rows] x 128 B
constexpr int kStages = 3;                 // of K, Q; of B and the row factors
constexpr uint32_t OFF_KQ = 0;
constexpr uint32_t OFF_V = OFF_KQ + kStages * KQ_BYTES;        // [64][128] bf16
constexpr uint32_t OFF_TB = OFF_V + 16384;                       // 3 terms of T Diag(beta), 64 x 64
constexpr uint32_t OFF_AQK = OFF_TB + 3 * 8192;                  // stages x 3 terms of B, lower blocks only
constexpr uint32_t B_BYTES = 16384;
constexpr uint32_t OFF_A = OFF_AQK + kStages * B_BYTES;          // per group: A, then T, fp32
constexpr uint32_t A_BYTES = C * LDA * 4;
constexpr uint32_t OFF_VEC = OFF_A + 2 * A_BYTES;                // stages x {-fk[64], fq[64], c[64], gamma}
constexpr uint32_t VEC_BYTES = 1024;
constexpr uint32_t OFF_PREP = OFF_VEC + kStages * VEC_BYTES;           // per group: G head, G tail, beta, rk, rq
constexpr uint32_t PREP_BYTES = 5 * 64 * 4;
constexpr uint32_t OFF_SCHED = OFF_PREP + 2 * PREP_BYTES;        // begin, len, slot, order of a page
constexpr uint32_t OFF_MISC = OFF_SCHED + kPage * 16;
constexpr uint32_t SMEM_USED = OFF_MISC + 256;
constexpr uint32_t SMEM_BYTES = SMEM_USED + 1024;                // the base is rounded up to 1024
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");

// Barriers.  KQ, V: loads landed.  GATE: gates of a chunk written, GFREE: the
// prep group done with them; READY: prep of a chunk done;
// FREE: its B and row factors used; TBFREE: its T used.  KK: [K ; Q] K^T done;
// KKFREE: read.  S: P, U, dS done, in turn; Q: Pq done; O: O done.  From the state
// warps, one arrival each: ST terms of S written, RT of R, UD of U', UT of U; OT the
// O before taken.
enum {
    MB_KQ = 0, MB_V = 3, MB_READY = 4, MB_FREE = 6, MB_KK = 9, MB_KKFREE = 11, MB_S = 13, MB_O = 14,
    MB_ST = 15, MB_OT = 16, MB_RT = 17, MB_UD = 18, MB_DRAIN = 19, MB_GATE = 20, MB_GFREE = 22, MB_TBFREE = 24, MB_Q = 26,
    MB_UT = 27, kNumBars = 28
};
__device__ __forceinline__ uint32_t bar_count(int i) {
    return (i >= MB_FREE && i < MB_KK) || (i >= MB_ST && i <= MB_UD) || i == MB_UT ? (uint32_t)kStateWarps : 1u;
}
static_assert(kNumBars * 8 <= 224, "room for the barriers");
constexpr uint32_t MISC_ABORT = 224, MISC_TMEM = 228, MISC_COUNT = 232;

// TMEM columns.  16 columns of an fp32 row become 8 + 8 columns of its first two
// terms; the third ones lie apart.
constexpr uint32_t COL_S = 0;              // S^T: term t < 2 of k-step s at 16 s + 8 t; dS
// Two tiles swap roles from chunk to chunk: X takes Pk^T, then two terms of R^T, then
// U^T B^T; Y (the X of the chunk before, its O taken) U^T, then two terms of it.
constexpr uint32_t COL_XY = 128;
__device__ __forceinline__ uint32_t col_x(int chunk) { return COL_XY + 64u * (uint32_t)(chunk & 1); }
__device__ __forceinline__ uint32_t col_y(int chunk) { return COL_XY + 64u * (uint32_t)(~chunk & 1); }
constexpr uint32_t COL_PQ = 256;           // Pq^T
constexpr uint32_t COL_S2 = 320;           // the third term of S^T, 8 s; then
constexpr uint32_t COL_UD = 320;           // U'^T: 3 terms x 32
constexpr uint32_t COL_KK = 416;           // [K ; Q] K^T of a chunk ahead
constexpr uint32_t COL_RU2 = 480;          // the third term of R^T, then of U^T, 8 s
constexpr uint32_t TMEM_COLS = 512;

enum { BAR_PREP = 1 };                     // + group

// Registers per thread: the state warps hold 64 values of S and a tile with its
// terms, the prep warps a tile, the issuing warpgroup little.  The shares add up
// to no more than the block is launched with (640 x 96: the kernel's launch
// bounds leave 102, allocated in eights) -- an increase beyond that would wait
// for ever.
constexpr int kLaunchRegs = 96, kStateRegs = 144, kPrepRegs = 72, kIssueRegs = 48;
static_assert(kStateThreads * kStateRegs + kPrepThreads * kPrepRegs + 128 * kIssueRegs <= kThreads * kLaunchRegs,
              "register shares");
template <int N>
__device__ __forceinline__ void regs_up() {
#ifdef __CUDA_ARCH__
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
#endif
}
template <int N>
__device__ __forceinline__ void regs_down() {
#ifdef __CUDA_ARCH__
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
#endif
}

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

// Steps of a descriptor's start address (its low field counts 16 bytes): k-step
// s of a K-major operand of `rows` rows, and of an MN-major one.
__host__ __device__ constexpr uint64_t kstep(int rows, int s) { return (uint64_t)(((s >> 2) * rows * 128 + (s & 3) * 32) >> 4); }
__host__ __device__ constexpr uint64_t mnstep(int s) { return (uint64_t)(s * 2048 >> 4); }

// ---- splits -----------------------------------------------------------------
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// The pair v as N bf16 terms each, rounded to nearest one after another: N = 3
// leaves at most 2^-27 of the value, N = 2 2^-18.
template <int N>
__device__ __forceinline__ void split2(float2 v, uint32_t (&w)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w[i] = pack_bf16x2(v.x, v.y);
        if (i + 1 < N) v = __ffma2_rn(make_float2(bf_lo(w[i]), bf_hi(w[i])), make_float2(-1.f, -1.f), v);
    }
}
// The leading 8 bits of both values, and what they leave.
__device__ __forceinline__ uint32_t top2(float2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632u); }
__device__ __forceinline__ float2 rest2(float2 v) {
    return __ffma2_rn(make_float2(bf_hi(__float_as_uint(v.x)), bf_hi(__float_as_uint(v.y))), make_float2(-1.f, -1.f), v);
}
// 16 consecutive columns of an operand row as three terms at TMEM columns, term by
// term (eight words live at a time).  Cut off one after another: exact.
__device__ __forceinline__ void put_cut(uint32_t at0, uint32_t at1, uint32_t at2, const float2 (&v)[8]) {
    float2 r[8];
    uint32_t w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        w[u] = top2(v[u]);
        r[u] = rest2(v[u]);
    }
    tmem_st8(at0, w);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        w[u] = top2(r[u]);
        r[u] = rest2(r[u]);
    }
    tmem_st8(at1, w);
#pragma unroll
    for (int u = 0; u < 8; ++u) w[u] = top2(r[u]);
    tmem_st8(at2, w);
}
// The same with rounded terms, two over the 16 columns themselves and a third at `third`.
__device__ __forceinline__ void put_three(uint32_t taddr, uint32_t third, const float2 (&v)[8]) {
    float2 r[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) r[u] = v[u];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            w[u] = pack_bf16x2(r[u].x, r[u].y);
            if (i < 2) r[u] = __ffma2_rn(make_float2(bf_lo(w[u]), bf_hi(w[u])), make_float2(-1.f, -1.f), r[u]);
        }
        tmem_st8(i < 2 ? taddr + 8u * (uint32_t)i : third, w);
    }
}
__device__ __forceinline__ void get16(uint32_t taddr, float2 (&v)[8]) {
    float a[16];
    tmem_ld16(taddr, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = make_float2(a[2 * i], a[2 * i + 1]);
}
// v (.) f, f from shared memory
__device__ __forceinline__ void scale16(float2 (&v)[8], const float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(f + 4 * i);
        v[2 * i] = __fmul2_rn(v[2 * i], make_float2(x.x, x.y));
        v[2 * i + 1] = __fmul2_rn(v[2 * i + 1], make_float2(x.z, x.w));
    }
}

// One lane of the (converged) warp issues; values it needs are made
// warp-uniform first, so that descriptors are computed on the uniform path.
__device__ __forceinline__ bool elect_one() {
#ifdef __CUDA_ARCH__
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r != 0;
#else
    return (threadIdx.x & 31) == 0;
#endif
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
#ifdef __CUDA_ARCH__
    return __shfl_sync(0xffffffffu, v, 0);
#else
    return v;
#endif
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
        if (live && p.slots) {             // (the recurrence looks at the short ones)
            bool repeat = packed_repeat(p.cu, p.slots, s0, sc.slot[i], 0, 1);
            for (int k = 0; k < i; ++k)
                if (sc.slot[k] == sc.slot[i]) repeat |= packed_has_rows(p.cu, s0 + k);
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
    int round;                             // next round to look at
    int n, chunks, len;                    // chunk of the chain; chunks and rows of the chain
    int chain;                             // rank * HV + head
    __device__ __forceinline__ void start(const PackedParams &p, const Sched &sc) {
        round = 0;
        next_chain(p, sc);
    }
    __device__ __forceinline__ bool valid() const { return n < chunks; }
    __device__ __forceinline__ int seq(const PackedParams &p, const Sched &sc) const { return sc.order[chain / p.HV]; }
    __device__ __forceinline__ int head(const PackedParams &p) const { return chain % p.HV; }
    __device__ __forceinline__ int rows() const { return min(C, len - n * C); }
    __device__ __forceinline__ void next_chain(const PackedParams &p, const Sched &sc) {
        n = chunks = len = 0;
        const int items = *sc.count * p.HV, ctas = (int)gridDim.x;
        while (round < (items + ctas - 1) / ctas) {
            chain = round * ctas + ((round & 1) ? ctas - 1 - (int)blockIdx.x : (int)blockIdx.x);
            ++round;
            if (chain >= items) continue;
            len = sc.len[seq(p, sc)];
            chunks = (len + C - 1) / C;
            return;
        }
    }
    __device__ __forceinline__ void next(const PackedParams &p, const Sched &sc) {
        if (++n >= chunks) next_chain(p, sc);
    }
};

// A cursor of loads: with the first row and the head of its chunk at hand, so that
// the issuing warp divides once a chain only (its next MMAs wait behind a load).
struct Feed {
    Cursor c;
    int row, head, khead;
    __device__ __forceinline__ void place(const PackedParams &p, const Sched &sc) {
        if (!c.valid()) return;
        row = sc.begin[c.seq(p, sc)];
        head = c.head(p);
        khead = head / p.group;
    }
    __device__ __forceinline__ void next(const PackedParams &p, const Sched &sc) {
        row += C;
        if (++c.n < c.chunks) return;
        c.next_chain(p, sc);
        place(p, sc);
    }
};
// Loads of one chunk (one thread).
__device__ __forceinline__ void request_kq(const CUtensorMap *tm, const Ctx &x, int row, int h, int stage) {
    const uint32_t kq = x.sbase + OFF_KQ + (uint32_t)stage * KQ_BYTES, mb = bar_addr(x, MB_KQ + stage);
    mbar_arrive_expect_tx(mb, KQ_BYTES);
    tma_load_3d(kq, &tm[0], 0, h, row, mb);
    tma_load_3d(kq + 16384, &tm[0], 64, h, row, mb);
    tma_load_3d(kq + 8192, &tm[1], 0, h, row, mb);
    tma_load_3d(kq + 16384 + 8192, &tm[1], 64, h, row, mb);
}
__device__ __forceinline__ void request_v(const CUtensorMap *tm, const Ctx &x, int row, int h) {
    const uint32_t mb = bar_addr(x, MB_V);
    mbar_arrive_expect_tx(mb, 16384);
    tma_load_3d(x.sbase + OFF_V, &tm[2], 0, h, row, mb);
}

// =====================================================================
// Prep role: one group of four warps for the even chunks, one for the odd.
// =====================================================================
__device__ __forceinline__ uint32_t tile_off(int r, int i) {      // 64 x 64 bf16, K-major, swizzled
    return (uint32_t)(r * 128 + (((i >> 3) ^ (r & 7)) << 4) + (i & 7) * 2);
}
// B has values in its lower 16 x 16 blocks only: k-step s (columns 16 s ..) is a strip
// of the 4 - s blocks from rows 16 s on, an MMA of 64 - 16 s tokens.  The strips of all
// three terms fill the room of two whole tiles: a strip stands in one of the four
// 32-byte columns of the 128-byte rows, its first block b blocks of 16 rows down.
//     column 0: (term 0, s 0), (1, 0)            column 1: (2, 0), (0, 1), (0, 3)
//     column 2: (1, 1), (2, 1), (0, 2)           column 3: (1, 2), (2, 2), (1, 3), (2, 3)
// 4 b + column of the strips s = 0 .. 3 of a term, a byte each.
__host__ __device__ constexpr uint32_t strip_code(int term, int s) {
    return ((term == 0 ? 0x1D1A1100u : term == 1 ? 0x13030210u : 0x170B0E01u) >> (8 * s)) & 31u;
}
// Offset of the strip's first row, and of 8 values of a row (16 bytes) in it.
__device__ __forceinline__ uint32_t strip_off(int term, int s) {
    const uint32_t c = strip_code(term, s);
    return (c >> 2) * 2048u + (c & 3u) * 32u;
}
__device__ __forceinline__ uint32_t strip_at(int term, int r, int i) {
    const int s = i >> 4;
    const uint32_t c = strip_code(term, s);
    return (c >> 2) * 2048u + (uint32_t)(r - 16 * s) * 128u + ((((c & 3u) * 2u + ((uint32_t)(i >> 3) & 1u)) ^ (uint32_t)(r & 7)) << 4);
}
// D (16 x 8 NB) = A (16 x 16) B (16 x 8 NB), fp32 tiles in shared memory, each
// operand as tf32 head and tail: three products, the error of an fp32 product.
// Head times head and the cross terms run as chains of their own.
template <int NB>
__device__ __forceinline__ void warp_block(float (&d)[NB][4], const float *A, const float *B, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float e[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) e[n][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        const float *a = A + g * LDA + 8 * kk + t;
        const float av[4] = {a[0], a[8 * LDA], a[4], a[8 * LDA + 4]};
        uint32_t ah[4], al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ah[i] = to_tf32(av[i]);
            al[i] = to_tf32(av[i] - __uint_as_float(ah[i]));
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const float *b = B + (8 * kk + t) * LDA + 8 * n + g;
            const float bv[2] = {b[0], b[4 * LDA]};
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                bh[i] = to_tf32(bv[i]);
                bl[i] = to_tf32(bv[i] - __uint_as_float(bh[i]));
            }
            mma_tf32_16x8x8(e[n], al, bh);
            mma_tf32_16x8x8(d[n], ah, bh);
            mma_tf32_16x8x8(e[n], ah, bl);
        }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[n][i] += e[n][i];
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
// One chunk's gate inputs for the tokens lane, lane + 32, kept as loaded (a
// conversion would wait for them).
struct Gate {
    __nv_bfloat16 z[2], b[2];
    float A, bias;
    __device__ __forceinline__ void load(const PackedParams &p, const Sched &sc, const Cursor &c, int lane) {
        A = bias = 0.f;
        if (!c.valid()) return;
        const int count = c.rows(), hv = c.head(p), row0 = sc.begin[c.seq(p, sc)] + c.n * C;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = lane + 32 * u;
            if (t < count) {
                const long long row = row0 + t;
                z[u] = static_cast<const __nv_bfloat16 *>(p.g)[row * p.ldg + hv];
                b[u] = static_cast<const __nv_bfloat16 *>(p.beta)[row * p.ldb + hv];
            }
        }
        if (p.gate_in) {
            A = p.A_log[hv];
            if (p.dt_bias) bias = p.dt_bias[hv];
        }
    }
};
// (ah, al) += (bh, bl), head and tail
__device__ __forceinline__ void add_two(float &ah, float &al, float bh, float bl) {
    const float s = ah + bh, v = s - ah;
    const float e = (ah - (s - v)) + (bh - v) + al + bl;
    ah = s + e;
    al = e - (ah - s);
}
__device__ __forceinline__ float *group_vectors(uint8_t *sm, int grp) {       // G head, G tail, beta, rk, rq
    return reinterpret_cast<float *>(sm + OFF_PREP + (uint32_t)grp * PREP_BYTES);
}

// =====================================================================
// Gate warps, one per prep group: log-decays of a chunk in log2 units, their
// running sum as head + tail, and beta, written when the group is done with
// those of its last chunk.
// =====================================================================
__device__ __forceinline__ void gate_page(const PackedParams &p, const Ctx &x, const Sched &sc, int grp, int lane, int &gc) {
    float *gh = group_vectors(x.sm, grp), *gl = gh + 64, *beta = gl + 64;
    Cursor cur;
    cur.start(p, sc);
    if ((gc & 1) != grp && cur.valid()) {  // the other group's chunk
        cur.next(p, sc);
        ++gc;
    }
    Gate gate;
    gate.load(p, sc, cur, lane);
    while (cur.valid()) {
        const int mine = gc, Cc = cur.rows();
        const float ea = p.gate_in ? expf(gate.A) : 0.f;
        float h[2], l[2] = {0.f, 0.f}, be[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = lane + 32 * u;
            const float zu = __bfloat162float(gate.z[u]), bu = __bfloat162float(gate.b[u]);
            float g = p.gate_in ? kda_gate(p.gate_in, zu, gate.bias, ea, p.g_min) : zu;
            g *= kLog2E;
            // below 2^-150 a factor is 0 in fp32: a floor keeps the sums finite
            g = g < -1e4f ? -1e4f : g;
            h[u] = t < Cc ? g : 0.f;
            be[u] = t < Cc ? (p.beta_sigmoid ? sigmoidf_(bu) : bu) : 0.f;
        }
        cur.next(p, sc);                   // the group's next chunk is two on
        ++gc;
        if (cur.valid()) {
            cur.next(p, sc);
            ++gc;
        }
        gate.load(p, sc, cur, lane);
#pragma unroll 1
        for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float oh = __shfl_up_sync(0xffffffffu, h[u], off), ol = __shfl_up_sync(0xffffffffu, l[u], off);
                if (lane >= off) add_two(h[u], l[u], oh, ol);
            }
        }
        add_two(h[1], l[1], __shfl_sync(0xffffffffu, h[0], 31), __shfl_sync(0xffffffffu, l[0], 31));
        if (mine >= 2 && !wait_bar(x, bar_addr(x, MB_GFREE + grp), (uint32_t)(((mine >> 1) - 1) & 1))) return;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            gh[lane + 32 * u] = h[u];
            gl[lane + 32 * u] = l[u];
            beta[lane + 32 * u] = be[u];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_addr(x, MB_GATE + grp));
    }
}

__device__ __forceinline__ void prep_page(const PackedParams &p, const Ctx &x, const Sched &sc, int grp, int tid, int &gc) {
    uint8_t *sm = x.sm;
    const int lane = tid & 31, warp = tid >> 5, bar = BAR_PREP + grp;
    const float *gh = group_vectors(sm, grp), *gl = gh + 64, *beta = gl + 64;
    float *rk = group_vectors(sm, grp) + 192, *rq = rk + 64;
    float *Am = reinterpret_cast<float *>(sm + OFF_A + (uint32_t)grp * A_BYTES);
    uint8_t *tb = sm + OFF_TB;

    Cursor cur;
    cur.start(p, sc);
    if ((gc & 1) != grp && cur.valid()) {  // the other group's chunk
        cur.next(p, sc);
        ++gc;
    }
    for (; cur.valid(); ++gc) {
        const int stage = gc % kStages, Cc = cur.rows();
        uint8_t *aqk = sm + OFF_AQK + (uint32_t)stage * B_BYTES;
        float *vec = reinterpret_cast<float *>(sm + OFF_VEC + (uint32_t)stage * VEC_BYTES);
        cur.next(p, sc);                   // two on: the group's next chunk
        int step = 1;
        if (cur.valid()) {
            cur.next(p, sc);
            step = 2;
        }
        // A wait that gives up leaves its thread running to the chunk's one vote,
        // where all return together.
        //
        // A wait for a phase needs the phase before complete.  Of KQ that is the load of
        // chunk gc - 3, which the issuing warp saw landed before FREE of gc - 5, and that
        // these threads waited for two chunks ago; the first chunks wait for FREE here.
        auto freed = [&]() { return wait_bar(x, bar_addr(x, MB_FREE + stage), (uint32_t)((gc / kStages - 1) & 1)); };
        bool ok = gc < kStages || gc >= kStages + 2 || freed();
        if (ok) ok = wait_bar(x, bar_addr(x, MB_KQ + stage), (uint32_t)((gc / kStages) & 1));
        // Norms: thread = row of [K ; Q].
        float ss;
        {
            const uint8_t *kq = sm + OFF_KQ + (uint32_t)stage * KQ_BYTES + tid * 128;
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
            if (p.l2norm) {
#pragma unroll 4
                for (int j = 0; j < 16; ++j) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(kq + (j >> 3) * 16384 + (((j & 7) ^ (tid & 7)) << 4));
                    const float2 f0 = make_float2(bf_lo(w.x), bf_hi(w.x)), f1 = make_float2(bf_lo(w.y), bf_hi(w.y));
                    const float2 f2 = make_float2(bf_lo(w.z), bf_hi(w.z)), f3 = make_float2(bf_lo(w.w), bf_hi(w.w));
                    s0 = __ffma2_rn(f0, f0, s0);
                    s1 = __ffma2_rn(f1, f1, s1);
                    s0 = __ffma2_rn(f2, f2, s0);
                    s1 = __ffma2_rn(f3, f3, s1);
                }
            }
            ss = (s0.x + s1.x) + (s0.y + s1.y);
        }
        if (ok) ok = wait_bar(x, bar_addr(x, MB_GATE + grp), (uint32_t)((gc >> 1) & 1));
        if (ok && gc >= kStages + 2) ok = freed();
        {                                  // row factors (0 behind the sequence's end)
            const int t = tid & 63;
            const float r = t < Cc ? (p.l2norm ? rsqrtf(ss + p.l2_eps) : 1.f) : 0.f;
            const float e = ex2f_(gh[t] + gl[t]);
            if (tid < 64) {
                rk[t] = r;
                vec[t] = -r * e;
                vec[128 + t] = r * ex2f_((gh[63] - gh[t]) + (gl[63] - gl[t]));
                if (t == 0) vec[192] = ex2f_(gh[63] + gl[63]);
            } else {
                rq[t] = r * p.scale;
                vec[64 + t] = r * p.scale * e;
            }
        }
        if (ok) ok = wait_bar(x, bar_addr(x, MB_KK + grp), (uint32_t)((gc >> 1) & 1));
        if (named_bar_any(bar, kGroup, !ok)) return;
        fence_after_sync();
        // A and B from the TMEM product: lane = row of [K ; Q].
        {
            const int row = (warp & 1) * 32 + lane;
            const bool is_q = warp >= 2;
            const float hi = gh[row], lo = gl[row];
            const float f = is_q ? rq[row] : beta[row] * rk[row];
            // the last column that counts; none in rows behind the end, whose products are another's rows
            const int last = row < Cc ? (is_q ? row : row - 1) : -1;
#pragma unroll 1
            for (int j0 = 0; j0 < 32 * (warp & 1) + 32; j0 += 16) {
                float v[16];
                tmem_ld16(x.tm + ((uint32_t)(warp * 32) << 16) + COL_KK + (uint32_t)j0, v);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 h4 = *reinterpret_cast<const float4 *>(gh + j0 + j);
                    const float4 l4 = *reinterpret_cast<const float4 *>(gl + j0 + j);
                    const float4 r4 = *reinterpret_cast<const float4 *>(rk + j0 + j);
                    const float2 m = make_float2(-1.f, -1.f);
                    const float2 d0 = __fadd2_rn(__ffma2_rn(make_float2(h4.x, h4.y), m, make_float2(hi, hi)),
                                                 __ffma2_rn(make_float2(l4.x, l4.y), m, make_float2(lo, lo)));
                    const float2 d1 = __fadd2_rn(__ffma2_rn(make_float2(h4.z, h4.w), m, make_float2(hi, hi)),
                                                 __ffma2_rn(make_float2(l4.z, l4.w), m, make_float2(lo, lo)));
                    const float2 w0 = __fmul2_rn(make_float2(v[j], v[j + 1]),
                                                 __fmul2_rn(make_float2(r4.x, r4.y), make_float2(f, f)));
                    const float2 w1 = __fmul2_rn(make_float2(v[j + 2], v[j + 3]),
                                                 __fmul2_rn(make_float2(r4.z, r4.w), make_float2(f, f)));
                    v[j] = j0 + j <= last ? w0.x * ex2f_(d0.x) : 0.f;
                    v[j + 1] = j0 + j + 1 <= last ? w0.y * ex2f_(d0.y) : 0.f;
                    v[j + 2] = j0 + j + 2 <= last ? w1.x * ex2f_(d1.x) : 0.f;
                    v[j + 3] = j0 + j + 3 <= last ? w1.y * ex2f_(d1.y) : 0.f;
                }
                if (is_q) {
#pragma unroll
                    for (int j = 0; j < 16; j += 8) {
                        uint32_t w[4][3];
#pragma unroll
                        for (int i = 0; i < 4; ++i) split2<3>(make_float2(v[j + 2 * i], v[j + 2 * i + 1]), w[i]);
                        if (j0 <= row) {               // (no room for blocks above the diagonal)
#pragma unroll
                            for (int i = 0; i < 3; ++i)
                                *reinterpret_cast<uint4 *>(aqk + strip_at(i, row, j0 + j)) =
                                    make_uint4(w[0][i], w[1][i], w[2][i], w[3][i]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(Am + row * LDA + j0 + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                }
            }
        }
        fence_before_sync();
        named_bar(bar, kGroup);
        if (tid == 0) mbar_arrive(bar_addr(x, MB_KKFREE));
        if (Cc < C) {                      // K and Q rows behind the sequence, another's or none: zero
            uint8_t *z = sm + OFF_KQ + (uint32_t)stage * KQ_BYTES;
            for (int i = tid; i < (C - Cc) * 32; i += kGroup) {
                const int r = Cc + i / 32, q = i % 32;
                *reinterpret_cast<uint4 *>(z + ((q >> 3) & 1) * 16384 + (q >> 4) * 8192 + r * 128 + (q & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
        }

        // T = (I + A)^-1 by 16 x 16 blocks, in place: the diagonal blocks first, the
        // rest from T_IJ = -T_II sum_{J<=K<I} A_IK T_KJ in three steps:
        //   (1) X10 = A10 T00, X32 = A32 T22, Xc = A_{23,01} T_{01,01} without its T10 term;
        //   (2) T10 = -T11 X10, T32 = -T33 X32, Xc[:, 0:16] -= Xc[:, 16:32] X10
        //       (the missing term A_{23,1} T10 equals -(A_{23,1} T11) X10);
        //   (3) T_{23,01} = -T_{23,23} Xc.
        // X10, X32 and Xc live above the diagonal.  (Substitution by blocks, not powers
        // of A: with keys alike the powers grow and cancel.)
        {
            // block `warp`, column j = lane % 16 (both half-warps alike), row by row
            const int j = lane & 15;
            float *Ab = Am + 16 * warp * LDA + 16 * warp;
            float xs[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float s0 = r == j ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                for (int i = 0; i < r; i += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(Ab + r * LDA + i);
                    s0 = fmaf(-a.x, xs[i], s0);
                    if (i + 1 < r) s1 = fmaf(-a.y, xs[i + 1], s1);
                    if (i + 2 < r) s0 = fmaf(-a.z, xs[i + 2], s0);
                    if (i + 3 < r) s1 = fmaf(-a.w, xs[i + 3], s1);
                }
                xs[r] = s0 + s1;
            }
            __syncwarp();                  // every row of the block has been read
            if (lane < 16) {
#pragma unroll
                for (int r = 0; r < 16; ++r) Ab[r * LDA + j] = xs[r];
            }
        }
        named_bar(bar, kGroup);
        {                                  // (1): a whole product and half of one per warp
            const int arow = warp == 0 ? 16 : warp == 2 ? 32 : 48, kc = warp < 2 ? 0 : 16;
            float *to = Am + (warp & 1 ? 16 : 0) * LDA + (warp == 0 ? 16 : warp == 1 ? 32 : 48);
            const int nh = 8 * (warp & 1);
            float d[2][4] = {}, h[1][4] = {};
            warp_block<2>(d, Am + arow * LDA + kc, Am + kc * LDA + kc, lane);
            if (warp < 2) warp_block<1>(h, Am + 32 * LDA, Am + nh, lane);
            else warp_block<1>(h, Am + 48 * LDA + 32, Am + 32 * LDA + 32 + nh, lane);
            warp_put(to, d[0], 1.f, false, lane);
            warp_put(to + 8, d[1], 1.f, false, lane);
            warp_put(Am + (warp < 2 ? 32 : 32 * LDA + 48) + nh, h[0], 1.f, false, lane);
        }
        named_bar(bar, kGroup);
        {                                  // (2)
            const int arow = warp == 0 ? 16 : warp == 1 ? 48 : 16 * (warp - 2);
            const int acol = warp == 0 ? 16 : 48;
            const int brow = warp == 1 ? 32 : 0, bcol = warp == 1 ? 48 : 16;
            float *to = Am + arow * LDA + (warp == 0 ? 0 : 32);
            float d[2][4] = {};
            warp_block<2>(d, Am + arow * LDA + acol, Am + brow * LDA + bcol, lane);
            warp_put(to, d[0], -1.f, warp >= 2, lane);
            warp_put(to + 8, d[1], -1.f, warp >= 2, lane);
        }
        named_bar(bar, kGroup);
        {                                  // (3): warp = (block row, block column)
            const int mt = warp & 1, cb = warp >> 1;
            const float *A = Am + (32 + 16 * mt) * LDA + 32, *B = Am + 32 + 16 * cb;
            float *to = Am + (32 + 16 * mt) * LDA + 16 * cb;
            float d[2][4] = {};
            warp_block<2>(d, A, B, lane);
            if (mt == 1) warp_block<2>(d, A + 16, B + 16 * LDA, lane);
            warp_put(to, d[0], -1.f, false, lane);
            warp_put(to + 8, d[1], -1.f, false, lane);
        }
        // (of chunk gc - 1; a barrier per parity, whose phase before is chunk gc - 3's)
        if (ok && gc > 0) ok = wait_bar(x, bar_addr(x, MB_TBFREE + ((gc - 1) & 1)), (uint32_t)(((gc - 1) >> 1) & 1));
        named_bar(bar, kGroup);
        {                                  // T Diag(beta) as three terms: warp = block row, lane pair = row
            const int r = tid >> 1;
#pragma unroll 1
            for (int c0 = 8 * (tid & 1); c0 < 16 * warp + 16; c0 += 16) {
                const float4 t0 = *reinterpret_cast<const float4 *>(Am + r * LDA + c0);
                const float4 t1 = *reinterpret_cast<const float4 *>(Am + r * LDA + c0 + 4);
                const float4 b0 = *reinterpret_cast<const float4 *>(beta + c0);
                const float4 b1 = *reinterpret_cast<const float4 *>(beta + c0 + 4);
                uint32_t w[4][3];
                split2<3>(__fmul2_rn(make_float2(t0.x, t0.y), make_float2(b0.x, b0.y)), w[0]);
                split2<3>(__fmul2_rn(make_float2(t0.z, t0.w), make_float2(b0.z, b0.w)), w[1]);
                split2<3>(__fmul2_rn(make_float2(t1.x, t1.y), make_float2(b1.x, b1.y)), w[2]);
                split2<3>(__fmul2_rn(make_float2(t1.z, t1.w), make_float2(b1.z, b1.w)), w[3]);
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    *reinterpret_cast<uint4 *>(tb + i * 8192 + tile_off(r, c0)) =
                        make_uint4(w[0][i], w[1][i], w[2][i], w[3][i]);
            }
        }
        if (Cc < C) {                      // V rows behind the sequence
            if (ok) ok = wait_bar(x, bar_addr(x, MB_V), (uint32_t)(gc & 1));
            for (int i = tid; i < (C - Cc) * 16; i += kGroup)
                *reinterpret_cast<uint4 *>(sm + OFF_V + (Cc + i / 16) * 256 + (i % 16) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        named_bar(bar, kGroup);
        if (tid == 0 && ok) {
            mbar_arrive(bar_addr(x, MB_READY + grp));
            mbar_arrive(bar_addr(x, MB_GFREE + grp));
        }
        gc += step - 1;
    }
}

// =====================================================================
// State role.  Thread = (TMEM lane = value channel j, half hf).
// =====================================================================
// One chain's S and where its outputs go.
struct Chain {
    float *pool;                           // S[64 hf][j] of the slot
    __nv_bfloat16 *o;                      // of this lane: row 32 hf + (lane & 1), channels j & ~1 and the next
    bool zero;
    __device__ __forceinline__ void at(const PackedParams &p, const Sched &sc, const Cursor &c, int s0, int hf, int j) {
        const int seq = c.seq(p, sc), hv = c.head(p);
        pool = p.pool + (((size_t)sc.slot[seq] * p.HV + hv) * D + 64 * hf) * D + j;
        o = static_cast<__nv_bfloat16 *>(p.o) + ((long long)sc.begin[seq] + 32 * hf + (j & 1)) * p.ldo +
            (long long)hv * D + (j & ~1);
        zero = p.fresh && p.fresh[s0 + seq];
    }
};
__device__ __forceinline__ void load_state(const Chain &ch, float2 (&S)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        S[i] = ch.zero ? make_float2(0.f, 0.f) : make_float2(ch.pool[(2 * i) * D], ch.pool[(2 * i + 1) * D]);
}
__device__ __forceinline__ void put_state(uint32_t tl, int hf, const float2 (&S)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float2 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = S[8 * q + i];
        const uint32_t at = tl + COL_S + (uint32_t)(64 * hf + 16 * q);
        put_cut(at, at + 8u, tl + COL_S2 + (uint32_t)(32 * hf + 8 * q), v);
    }
}

// O^T = Pq^T Diag(fq) + U^T B^T of a chunk, as bf16 pairs of tokens.
__device__ __forceinline__ void take_o(uint32_t tl, int chunk, int hf, const float *fq, uint32_t (&o)[16]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float a[16], b[16];
        tmem_ld16x2(tl + COL_PQ + (uint32_t)(32 * hf + 16 * q), tl + col_x(chunk) + (uint32_t)(32 * hf + 16 * q), a, b);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float4 f = *reinterpret_cast<const float4 *>(fq + 16 * q + 4 * u);
            const float2 o0 = __ffma2_rn(make_float2(a[4 * u], a[4 * u + 1]), make_float2(f.x, f.y),
                                         make_float2(b[4 * u], b[4 * u + 1]));
            const float2 o1 = __ffma2_rn(make_float2(a[4 * u + 2], a[4 * u + 3]), make_float2(f.z, f.w),
                                         make_float2(b[4 * u + 2], b[4 * u + 3]));
            o[8 * q + 2 * u] = pack_bf16x2(o0.x, o0.y);
            o[8 * q + 2 * u + 1] = pack_bf16x2(o1.x, o1.y);
        }
    }
}
// Lanes exchange so that each writes two channels of one token of a pair;
// `count` of the 32 tokens are rows.
__device__ __forceinline__ void store_o(const PackedParams &p, __nv_bfloat16 *at, int count, int lane,
                                        const uint32_t (&o)[16]) {
    if (count <= 0) return;
    const uint32_t sel = (lane & 1) ? 0x3276u : 0x5410u;         // odd: other's upper, mine; even: mine, other's lower
    const int first = lane & 1;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        const uint32_t other = __float_as_uint(__shfl_xor_sync(0xffffffffu, __uint_as_float(o[u]), 1));
        const uint32_t w = __byte_perm(o[u], other, sel);
        if (2 * u + first < count) *reinterpret_cast<uint32_t *>(at) = w;
        at += 2 * p.ldo;
    }
}

// One arrival of the (converged) warp, after what its lanes wrote to TMEM.
__device__ __forceinline__ void warp_arrive(const Ctx &x, int bar, int lane) {
    tmem_st_wait();
    fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_addr(x, bar));
}

// Runs the page's chunks; `gc` counts this CTA's chunks, `ph` the phases of MB_S.
// The warps do not wait for one another: what one lane reads of TMEM it wrote
// itself or an MMA did.  A warp whose wait gives up returns; the abort flag ends
// the others' waits.
__device__ __forceinline__ void state_page(const PackedParams &p, const Ctx &x, const Sched &sc, int s0, int tid, int &gc,
                                           uint32_t &ph) {
    uint8_t *sm = x.sm;
    const int warp = tid >> 5, lane = tid & 31, hf = warp >> 2, j = (warp & 3) * 32 + lane;
    const uint32_t tl = x.tm + ((uint32_t)((warp & 3) * 32) << 16);    // (roles begin at multiples of four warps)

    Cursor cur;
    cur.start(p, sc);
    if (!cur.valid()) return;
    float2 S[32];                          // S[64 hf + 2 i .. + 1][j]
    Chain ch;
    ch.at(p, sc, cur, s0, hf, j);
    load_state(ch, S);
    put_state(tl, hf, S);
    warp_arrive(x, MB_ST, lane);
    __nv_bfloat16 *o_at = nullptr;         // of the chunk before, and its rows of this half
    int o_count = 0;

    bool first = true;
    for (; cur.valid(); ++gc) {
        const int stage = gc % kStages, before = (gc + kStages - 1) % kStages;
        const float *vec = reinterpret_cast<const float *>(sm + OFF_VEC + (uint32_t)stage * VEC_BYTES) + 32 * hf;
        if (!first) {                      // O of the chunk before, while P is computed
            uint32_t o[16];
            if (!wait_bar(x, bar_addr(x, MB_O), (uint32_t)((gc - 1) & 1))) return;
            fence_after_sync();
            take_o(tl, gc - 1, hf, reinterpret_cast<const float *>(sm + OFF_VEC + (uint32_t)before * VEC_BYTES) + 64 + 32 * hf, o);
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar_addr(x, MB_OT));
                mbar_arrive(bar_addr(x, MB_FREE + before));
            }
            store_o(p, o_at, o_count, lane, o);
        } else if (lane == 0) {
            mbar_arrive(bar_addr(x, MB_OT));
        }
        if (!wait_bar(x, bar_addr(x, MB_READY + (gc & 1)), (uint32_t)((gc >> 1) & 1))) return;
        if (!wait_bar(x, bar_addr(x, MB_V), (uint32_t)(gc & 1))) return;
        if (!wait_bar(x, bar_addr(x, MB_S), ph)) return;
        ph ^= 1u;
        fence_after_sync();
        // R^T = V^T - Pk^T Diag(fk)  (vec holds -fk)
        const uint8_t *vt = sm + OFF_V + (uint32_t)(32 * hf) * 256u + 2u * (uint32_t)j;
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
            float2 v[8], pk[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = make_float2(bf_lo(*reinterpret_cast<const uint16_t *>(vt + 4096 * q + 512 * u)),
                                   bf_lo(*reinterpret_cast<const uint16_t *>(vt + 4096 * q + 512 * u + 256)));
            const uint32_t at = tl + col_x(gc) + (uint32_t)(32 * hf + 16 * q);
            get16(at, pk);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 f = *reinterpret_cast<const float4 *>(vec + 16 * q + 4 * u);
                v[2 * u] = __ffma2_rn(make_float2(f.x, f.y), pk[2 * u], v[2 * u]);
                v[2 * u + 1] = __ffma2_rn(make_float2(f.z, f.w), pk[2 * u + 1], v[2 * u + 1]);
            }
            put_three(at, tl + COL_RU2 + (uint32_t)(16 * hf + 8 * q), v);
        }
        warp_arrive(x, MB_RT, lane);
        if (!wait_bar(x, bar_addr(x, MB_S), ph)) return;
        ph ^= 1u;
        fence_after_sync();
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {      // Diag(c) U for dS
            float2 v[8];
            get16(tl + col_y(gc) + (uint32_t)(32 * hf + 16 * q), v);
            scale16(v, vec + 128 + 16 * q);
            const uint32_t at = tl + COL_UD + (uint32_t)(16 * hf + 8 * q);
            put_cut(at, at + 32u, at + 64u, v);
        }
        const float gamma = vec[192 - 32 * hf];
        warp_arrive(x, MB_UD, lane);
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {      // U for O, while dS is computed
            float2 v[8];
            const uint32_t at = tl + col_y(gc) + (uint32_t)(32 * hf + 16 * q);
            get16(at, v);
            put_three(at, tl + COL_RU2 + (uint32_t)(16 * hf + 8 * q), v);
        }
        warp_arrive(x, MB_UT, lane);
        o_at = ch.o + (long long)cur.n * C * p.ldo;
        o_count = cur.rows() - 32 * hf;
        if (!wait_bar(x, bar_addr(x, MB_S), ph)) return;
        ph ^= 1u;
        fence_after_sync();
        // S = gamma S + dS, and its terms over the columns of dS and of the U' that made it
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float2 v[8];
            const uint32_t at = tl + COL_S + (uint32_t)(64 * hf + 16 * q);
            get16(at, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                S[8 * q + i] = __ffma2_rn(make_float2(gamma, gamma), S[8 * q + i], v[i]);
                v[i] = S[8 * q + i];
            }
            put_cut(at, at + 8u, tl + COL_S2 + (uint32_t)(32 * hf + 8 * q), v);
        }
        const bool last = cur.n + 1 == cur.chunks;
        if (last) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                ch.pool[(2 * i) * D] = S[i].x;
                ch.pool[(2 * i + 1) * D] = S[i].y;
            }
        }
        cur.next(p, sc);
        first = false;
        if (cur.valid()) {
            if (last) {
                ch.at(p, sc, cur, s0, hf, j);
                load_state(ch, S);
                put_state(tl, hf, S);
            }
            warp_arrive(x, MB_ST, lane);
        }
    }
    if (!wait_bar(x, bar_addr(x, MB_O), (uint32_t)((gc - 1) & 1))) return;
    fence_after_sync();
    uint32_t o[16];                        // the last chunk's
    take_o(tl, gc - 1, hf, reinterpret_cast<const float *>(sm + OFF_VEC + (uint32_t)((gc - 1) % kStages) * VEC_BYTES) + 64 + 32 * hf, o);
    fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_addr(x, MB_FREE + (gc - 1) % kStages));
    store_o(p, o_at, o_count, lane, o);
}

// =====================================================================
// Issuing warp: loads and MMAs, one elected lane, in the order the chunks need
// them.
// =====================================================================
struct Issue {
    int kq_n, v_n, kk_n;                   // chunks of this CTA requested, and multiplied for the prep warps
    uint32_t ph;                           // phases of MB_S
};

// Column of term t of S^T for k-step s.
__device__ __forceinline__ uint32_t s_col(int t, int s) { return t < 2 ? COL_S + 16u * s + 8u * t : COL_S2 + 8u * s; }

// [K ; Q] K^T of chunk n, once its rows have landed and the product before it has been read.
__device__ __forceinline__ bool issue_kk(const Ctx &x, Issue &is) {
    const int n = is.kk_n++;
    if (!wait_bar(x, bar_addr(x, MB_KQ + n % kStages), (uint32_t)((n / kStages) & 1))) return false;
    if (n > 0 && !wait_bar(x, bar_addr(x, MB_KKFREE), (uint32_t)((n - 1) & 1))) return false;
    const uint32_t a = uniform(x.sbase + OFF_KQ + (uint32_t)(n % kStages) * KQ_BYTES), d = uniform(x.tm + COL_KK);
    const uint32_t mb = uniform(bar_addr(x, MB_KK + (n & 1)));
    if (elect_one()) {
        fence_after_sync();
        const uint64_t dk = kmaj_desc(a, 128, 0);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
            mma_bf16(d, dk + kstep(128, s), dk + kstep(128, s), idesc_bf16(128, 64), s > 0);
        mma_commit(mb);
    }
    __syncwarp();
    return true;
}

__device__ __forceinline__ void issue_page(const PackedParams &p, const CUtensorMap *tmaps, const Ctx &x, const Sched &sc,
                                           int &gc, Issue &is) {
    const uint32_t id_u = idesc_bf16(128, 64), id_s = idesc_bf16(128, 128, false, /*b_mn_major=*/true);
    const uint32_t tm = uniform(x.tm), mb = uniform(bar_addr(x, MB_S)), mo = uniform(bar_addr(x, MB_O));
    const uint32_t mt = uniform(bar_addr(x, MB_TBFREE)), mq = uniform(bar_addr(x, MB_Q)), tb = uniform(x.sbase + OFF_TB);
    Cursor cur;                            // the chunk at hand
    Feed kq, v;                            // the next K and Q, the next V to load
    cur.start(p, sc);
    if (!cur.valid()) return;
    kq.c = cur;
    kq.place(p, sc);
    v = kq;
    int left = 0;                          // chunks of the page whose product is not issued yet
    for (Cursor c = cur; c.valid(); c.next_chain(p, sc)) left += c.chunks;
    auto load_kq = [&]() {
        if (!kq.c.valid()) return;
        if (elect_one()) request_kq(tmaps, x, kq.row, kq.khead, is.kq_n % kStages);
        __syncwarp();
        ++is.kq_n;
        kq.next(p, sc);
    };
    auto load_v = [&]() {
        if (!v.c.valid()) return;
        if (elect_one()) request_v(tmaps, x, v.row, v.head);
        __syncwarp();
        ++is.v_n;
        v.next(p, sc);
    };
    for (int i = 0; i < kStages; ++i) load_kq();
    load_v();
    for (int i = 0; i < 2 && left > 0; ++i, --left)
        if (!issue_kk(x, is)) return;
    for (bool first = true; cur.valid(); first = false, ++gc, cur.next(p, sc)) {
        const uint32_t par = (uint32_t)(gc & 1);
        const uint32_t a = uniform(x.sbase + OFF_KQ + (uint32_t)(gc % kStages) * KQ_BYTES);
        const uint32_t aq = uniform(x.sbase + OFF_AQK + (uint32_t)(gc % kStages) * B_BYTES);
        const uint32_t cx = uniform(x.tm + col_x(gc)), cy = uniform(x.tm + col_y(gc));
        // Pk^T = S^T K^T, small terms first; its columns still hold the U of the O before
        if (!wait_bar(x, bar_addr(x, MB_READY + (gc & 1)), (uint32_t)((gc >> 1) & 1))) return;
        if (!first && !wait_bar(x, bar_addr(x, MB_O), par ^ 1u)) return;
        if (!wait_bar(x, bar_addr(x, MB_ST), par)) return;
        const uint64_t dk = kmaj_desc(a, 128, 0);
        if (elect_one()) {
            fence_after_sync();
#pragma unroll 1
            for (int t = 2; t >= 0; --t)
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    mma_bf16_tmem_a(cx, tm + s_col(t, s), dk + kstep(128, s), id_u, t < 2 || s > 0);
            mma_commit(mb);
        }
        __syncwarp();
        is.ph ^= 1u;
        // Pq^T = S^T Q^T and a product for the prep warps, while the state warps work on R
        if (!wait_bar(x, bar_addr(x, MB_OT), par)) return;
        if (elect_one()) {
            fence_after_sync();
#pragma unroll 1
            for (int t = 2; t >= 0; --t)
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    mma_bf16_tmem_a(tm + COL_PQ, tm + s_col(t, s), dk + 512 + kstep(128, s), id_u, t < 2 || s > 0);
            mma_commit(mq);
        }
        __syncwarp();
        if (left > 0) {
            --left;
            if (!issue_kk(x, is)) return;
        }
        // U^T = R^T (T Diag(beta))^T
        if (!wait_bar(x, bar_addr(x, MB_RT), par)) return;
        if (elect_one()) {
            fence_after_sync();
            const uint64_t dt = kmaj_desc(tb, 64, 0);
            // terms (2,0), (1,1), (0,2), (1,0), (0,1), (0,0) of R and T Diag(beta)
#pragma unroll 1
            for (int t = 0; t < 6; ++t) {
                const uint32_t ra = (0x001012u >> (4 * t)) & 3u, ta = (0x010210u >> (4 * t)) & 3u;
                const uint32_t r0 = ra < 2 ? cx + 8u * ra : tm + COL_RU2, rs = ra < 2 ? 16u : 8u;
#pragma unroll
                for (int s = 0; s < C / 16; ++s)
                    mma_bf16_tmem_a(cy, r0 + rs * s, dt + ta * 512u + kstep(64, s), id_u, t > 0 || s > 0);
            }
            mma_commit(mb);
            mma_commit(mt + 8u * par);
        }
        __syncwarp();
        is.ph ^= 1u;
        load_v();                          // every state warp has read this chunk's
        // dS^T = U'^T K over the columns of S, then U^T B^T
        if (!wait_bar(x, bar_addr(x, MB_UD), par)) return;
        if (!wait_bar(x, bar_addr(x, MB_Q), par)) return;
        if (elect_one()) {
            fence_after_sync();
            const uint64_t dm = mn_desc(a, 16384, 0);
#pragma unroll 1
            for (int t = 2; t >= 0; --t)
#pragma unroll
                for (int s = 0; s < C / 16; ++s)
                    mma_bf16_tmem_a(tm + COL_S, tm + COL_UD + 32u * t + 8u * s, dm + mnstep(s), id_s, t < 2 || s > 0);
            mma_commit(mb);
        }
        __syncwarp();
        if (!wait_bar(x, bar_addr(x, MB_UT), par)) return;
        if (elect_one()) {
            fence_after_sync();
            const uint64_t da = kmaj_desc(aq, 64, 0);
            // terms (2,0), (1,1), (0,2), (1,0), (0,1), (0,0) of U and B, B by strips
#pragma unroll 1
            for (int t = 0; t < 6; ++t) {
                const int ua = (0x001012 >> (4 * t)) & 3, ba = (0x010210 >> (4 * t)) & 3;
                const uint32_t u0 = ua < 2 ? cy + 8u * (uint32_t)ua : tm + COL_RU2, us = ua < 2 ? 16u : 8u;
#pragma unroll
                for (int s = 0; s < C / 16; ++s)
                    mma_bf16_tmem_a(cx + 16u * s, u0 + us * s, da + (strip_off(ba, s) >> 4),
                                    idesc_bf16(128, 64 - 16 * s), t > 0 || s > 0);
            }
            mma_commit(mo);
        }
        __syncwarp();
        // dS is done: so are all readers of this chunk's K and Q
        if (!wait_bar(x, bar_addr(x, MB_S), is.ph)) return;
        is.ph ^= 1u;
        load_kq();
    }
}

__global__ void __launch_bounds__(kThreads, 1)
packed_chunk_kernel(const __grid_constant__ PackedTcParams tp) {
    const PackedParams &p = tp.p;
    // rounded up by an offset, not through an integer, so that accesses stay shared-memory ones
    uint8_t *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
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
        for (int i = 0; i < kNumBars; ++i) mbar_init(bar_addr(x, i), bar_count(i));
        *x.abort_flag = 0;
        fence_mbar_init();
    }
    // what lies above the diagonal blocks of T Diag(beta) is never written again
    for (uint32_t i = tid; i < (OFF_AQK - OFF_TB) / 16; i += kThreads)
        *reinterpret_cast<uint4 *>(sm + OFF_TB + 16 * i) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    x.tm = *tmem_slot;

    const Sched sc = sched_of(sm);
    int gc = 0;                            // chunks of this CTA so far: stages and phases go on over pages
    Issue is = {0, 0, 0, 0u};
    if (tid >= kFirstState && tid < kFirstPrep) {
        regs_up<kStateRegs>();
        uint32_t ph = 0;
        for (int s0 = 0; s0 < p.N; s0 += kPage) {
            fill_page(p, sc, s0, tid);
            state_page(p, x, sc, s0, tid - kFirstState, gc, ph);
            __syncthreads();
            if (*x.abort_flag) break;
        }
    } else if (tid >= kFirstPrep) {
        regs_down<kPrepRegs>();
        for (int s0 = 0; s0 < p.N; s0 += kPage) {
            fill_page(p, sc, s0, tid);
            prep_page(p, x, sc, (tid - kFirstPrep) / kGroup, (tid - kFirstPrep) % kGroup, gc);
            __syncthreads();
            if (*x.abort_flag) break;
        }
    } else {                               // one warp issues, one serves each prep group, one has nothing to do
        regs_down<kIssueRegs>();
        const bool issuer = warp == 0;     // the oldest warp, so that it is not kept waiting for a slot
        for (int s0 = 0; s0 < p.N; s0 += kPage) {
            fill_page(p, sc, s0, tid);
            if (issuer) issue_page(p, tp.tm, x, sc, gc, is);
            else if (warp < 3) gate_page(p, x, sc, warp - 1, tid & 31, gc);
            __syncthreads();
            if (*x.abort_flag) break;
        }
        // TMEM is freed once every MMA issued is complete, and shared memory is left
        // once every load requested has landed, after an abort too (bounded).
        const uint32_t mb = uniform(bar_addr(x, MB_DRAIN));
        if (issuer && elect_one()) mma_commit(mb);
        __syncwarp();
        auto done = [&](int bar, int phase) {
            for (uint32_t i = 0; i < kWaitTries; ++i)
                if (mbar_try_wait_suspend(bar_addr(x, bar), (uint32_t)(phase & 1), kSuspendNs)) break;
        };
        if (issuer) done(MB_DRAIN, 0);
        for (int n = is.kq_n - 1; n >= 0 && n >= is.kq_n - kStages; --n) done(MB_KQ + n % kStages, n / kStages);
        if (is.v_n > 0) done(MB_V, is.v_n - 1);
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
    // The roles' registers add up to kLaunchRegs a thread: a build that launches with
    // fewer would wait for ever for the increase.
    static const int regs = []() {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, packed_chunk_kernel) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
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
