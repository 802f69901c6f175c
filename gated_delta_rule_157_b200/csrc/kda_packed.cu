// kda_packed_fwd, recurrent form: every (sequence, value head) token by token
// in fp32, state in registers from its load to its store.
//
// With ka = k (.) a, qa = q (.) a (a the decay of the token), both inner
// products read the state as it was before the token,
//
//     e = v - S^T ka,    o = S^T qa + (q . k) beta e,    S <- a (.) S + k (beta e)^T,
//
// so one pass over the registers and one reduction serve both.  State columns
// are independent: a warp owns CW = 4 * 32 / RG columns of all Dk rows, lane =
// (row group, quad of columns); only the RG row groups meet, in seven
// exchanges and four broadcasts a token, and no warp waits for another inside a
// tile of tokens.  What depends on the token alone (norms, gates, ka, qa) is prepared by the block
// for a tile of TPW tokens per warp.  Long sequences (LOOP) prepare two tokens
// a warp into a double shared buffer, the next tile's rows requested while one is
// computed: one block barrier per tile.  Where the caller knows that sequences fit
// one tile of a token per warp (decode, verification) nothing is kept for a next tile, which
// leaves registers for more blocks: there it is the traffic that counts.
//
// A decode step of 256 x 32 chains (1.08 GB) takes 238 us on the device, 4.5 TB/s: the
// traffic, with the wait for a block's first rows on top (24 % of the warps active,
// issue slots 33 %).  A ragged prefill of 6 x 16 chains is bound by the longest chain,
// 0.63 us a token: 283 instructions of each warp, most of them dependent.
#include "kda_packed.cuh"

namespace kda {
namespace {

__device__ unsigned int g_packed_error = 0;

constexpr int kRG = 8;                     // row groups (lanes along a column)
constexpr int kCW = 4 * 32 / kRG;          // state columns per warp

extern __shared__ float smem[];

// Floats of one prepared token: ka, qa, k, a (one decay per channel) or k, q
// (one per head), the row of v, and {beta, q . k, a}.
__host__ __device__ constexpr int token_floats(int dkp, bool per_head) { return (per_head ? 2 : 4) * dkp + 128 + 4; }

template <typename Tin, int RPL, bool PER_HEAD>
struct TokenPrep {
    static constexpr int DKP = RPL * kRG;
    static constexpr int NC = (DKP + 31) / 32;
    Tin q0[NC], k0[NC], g0[NC], v0[4], beta0;      // as loaded: a conversion would wait for the load

    __device__ __forceinline__ void load(const PackedParams &p, long long row, int h, int hv, int lane) {
        const Tin *qr = static_cast<const Tin *>(p.q) + row * p.ldq + (long long)h * p.Dk;
        const Tin *kr = static_cast<const Tin *>(p.k) + row * p.ldk + (long long)h * p.Dk;
        const Tin *vr = static_cast<const Tin *>(p.v) + row * p.ldv + (long long)hv * p.Dv;
        const Tin *gr = static_cast<const Tin *>(p.g) + row * p.ldg + (long long)hv * (PER_HEAD ? 1 : p.Dk);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + 32 * i;
            if (c < p.Dk) {
                q0[i] = qr[c];
                k0[i] = kr[c];
                if (!PER_HEAD) g0[i] = gr[c];
            }
        }
        if (PER_HEAD) g0[0] = gr[0];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < p.Dv) v0[i] = vr[lane + 32 * i];
        beta0 = static_cast<const Tin *>(p.beta)[row * p.ldb + hv];
    }

    // `bias`: dt_bias of this lane's channels, 0 beyond them.
    __device__ __forceinline__ void store(const PackedParams &p, const float (&bias)[NC], float ea, int lane, float *out) {
        float q[NC], k[NC], g[NC], v[4];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const bool in = lane + 32 * i < p.Dk;
            q[i] = in ? ld_act(&q0[i], 0) : 0.f;
            k[i] = in ? ld_act(&k0[i], 0) : 0.f;
            g[i] = in && !PER_HEAD ? ld_act(&g0[i], 0) : 0.f;
        }
        if (PER_HEAD) g[0] = ld_act(&g0[0], 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lane + 32 * i < p.Dv ? ld_act(&v0[i], 0) : 0.f;
        const float beta = ld_act(&beta0, 0);
        float sq = 0.f, sk = 0.f, qk = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            sq = fmaf(q[i], q[i], sq);
            sk = fmaf(k[i], k[i], sk);
            qk = fmaf(q[i], k[i], qk);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            sq += __shfl_xor_sync(0xffffffffu, sq, off);
            sk += __shfl_xor_sync(0xffffffffu, sk, off);
            qk += __shfl_xor_sync(0xffffffffu, qk, off);
        }
        const float rq = p.l2norm ? p.scale / sqrtf(sq + p.l2_eps) : p.scale;
        const float rk = p.l2norm ? 1.f / sqrtf(sk + p.l2_eps) : 1.f;
        float a_head = 0.f;
        if (PER_HEAD) {
            a_head = expf(p.gate_in ? kda_gate(p.gate_in, g[0], bias[0], ea, p.g_min) : g[0]);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + 32 * i;
            if (c >= DKP) break;
            const float kn = k[i] * rk, qn = q[i] * rq;
            if (PER_HEAD) {
                out[c] = kn;
                out[DKP + c] = qn;
            } else {
                const bool in = c < p.Dk;
                const float a = in ? expf(p.gate_in ? kda_gate(p.gate_in, g[i], bias[i], ea, p.g_min) : g[i]) : 0.f;
                out[c] = kn * a;
                out[DKP + c] = qn * a;
                out[2 * DKP + c] = kn;
                out[3 * DKP + c] = a;
            }
        }
        float *vo = out + (PER_HEAD ? 2 : 4) * DKP;
#pragma unroll
        for (int i = 0; i < 4; ++i) vo[lane + 32 * i] = v[i];
        if (lane == 0) {
            vo[128] = p.beta_sigmoid ? sigmoidf_(beta) : beta;
            vo[129] = qk * rq * rk;
            vo[130] = a_head;
        }
    }
};

template <typename Tin, int RPL, bool PER_HEAD, int TPW, bool LOOP>
__global__ void __launch_bounds__(256, LOOP ? 1 : 2)
packed_recurrent_kernel(const PackedParams p) {
    constexpr int DKP = RPL * kRG;
    constexpr int TF = token_floats(DKP, PER_HEAD);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int s = blockIdx.x / p.HV, hv = blockIdx.x % p.HV, h = hv / p.group;
    const int rg = lane / (32 / kRG), quad = lane % (32 / kRG);
    const int col = (blockIdx.y * warps + warp) * kCW + 4 * quad;
    const bool col_ok = col < p.Dv;

    const PackedSeq sq = packed_seq(p.cu, p.slots, p.T, p.P, s);
    // a sequence without rows changes nothing
    const bool mine = !sq.bad && sq.slot >= 0 && sq.len > 0 && sq.len <= p.split;

    // The first rows before the state, so that they are prepared while it is on its way.
    const int tile = TPW * warps;
    TokenPrep<Tin, RPL, PER_HEAD> raw[TPW];
#pragma unroll
    for (int u = 0; u < TPW; ++u) {
        const int t = warp * TPW + u;
        if (mine && t < sq.len) raw[u].load(p, (long long)sq.begin + t, h, hv, lane);
    }
    constexpr int NC = TokenPrep<Tin, RPL, PER_HEAD>::NC;
    const float A = p.gate_in ? p.A_log[hv] : 0.f;
    float bias[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + 32 * i;
        bias[i] = 0.f;
        if (p.gate_in && p.dt_bias && (PER_HEAD ? i == 0 : c < p.Dk)) bias[i] = p.dt_bias[PER_HEAD ? hv : (size_t)hv * p.Dk + c];
    }

    // The state: rows (i / 4) * 4 RG + 4 rg + i % 4 of this lane's four columns,
    // kept as row pairs so that the prepared vectors feed packed FMAs directly.
    float *S = p.pool + ((size_t)(mine ? sq.slot : 0) * p.HV + hv) * p.Dk * p.Dv + col;
    float2 st[RPL / 2][4];
    const bool zero = !mine || (p.fresh && p.fresh[s]);
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        const int r = (i >> 2) * (4 * kRG) + 4 * rg + (i & 3);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!zero && col_ok && r < p.Dk) x = __ldcs(reinterpret_cast<const float4 *>(S + (size_t)r * p.Dv));
        if ((i & 1) == 0) {
            st[i >> 1][0].x = x.x; st[i >> 1][1].x = x.y; st[i >> 1][2].x = x.z; st[i >> 1][3].x = x.w;
        } else {
            st[i >> 1][0].y = x.x; st[i >> 1][1].y = x.y; st[i >> 1][2].y = x.z; st[i >> 1][3].y = x.w;
        }
    }

    const bool repeat = __syncthreads_or(packed_repeat(p.cu, p.slots, s, sq.slot, tid, blockDim.x));
    if ((sq.bad || (repeat && sq.len > 0)) && tid == 0 && hv == 0 && blockIdx.y == 0) atomicOr(&g_packed_error, kPackedRange);
    if (!mine || repeat) return;
    const float ea = expf(A);
    for (int t0 = 0, buf = 0; t0 < sq.len; t0 += tile, buf ^= 1) {
        float *tok = smem + (LOOP ? buf * tile * TF : 0);
#pragma unroll
        for (int u = 0; u < TPW; ++u) {
            const int t = t0 + warp * TPW + u;
            if (t < sq.len) raw[u].store(p, bias, ea, lane, tok + (warp * TPW + u) * TF);
        }
        __syncthreads();
        if (LOOP) {
#pragma unroll
            for (int u = 0; u < TPW; ++u) {            // the next tile's rows, in flight meanwhile
                const int t = t0 + tile + warp * TPW + u;
                if (t < sq.len) raw[u].load(p, (long long)sq.begin + t, h, hv, lane);
            }
        }
        const int n = min(tile, sq.len - t0);
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            const float *x = tok + t * TF;
            const float *xk = x + 4 * rg, *xq = x + DKP + 4 * rg;      // ka, qa (or k, q)
            float2 ak[4], aq[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) ak[c] = aq[c] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < RPL / 4; ++i) {
                const float4 k4 = *reinterpret_cast<const float4 *>(xk + i * 4 * kRG);
                const float4 q4 = *reinterpret_cast<const float4 *>(xq + i * 4 * kRG);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    ak[c] = __ffma2_rn(make_float2(k4.x, k4.y), st[2 * i][c], ak[c]);
                    aq[c] = __ffma2_rn(make_float2(q4.x, q4.y), st[2 * i][c], aq[c]);
                    ak[c] = __ffma2_rn(make_float2(k4.z, k4.w), st[2 * i + 1][c], ak[c]);
                    aq[c] = __ffma2_rn(make_float2(q4.z, q4.w), st[2 * i + 1][c], aq[c]);
                }
            }
            // Sums over the row groups, scattered: of the eight (S^T ka, S^T qa per
            // column) each group ends with one -- group c with S^T ka of column c,
            // group 4 + c with S^T qa of it -- in 4 + 2 + 1 exchanges.
            float r[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                r[c] = ak[c].x + ak[c].y;
                r[4 + c] = aq[c].x + aq[c].y;
            }
#pragma unroll
            for (int half = 4; half > 0; half >>= 1) {
                const bool up = rg & half;
#pragma unroll
                for (int c = 0; c < half; ++c) {
                    const float send = up ? r[c] : r[half + c], keep = up ? r[half + c] : r[c];
                    r[c] = keep + __shfl_xor_sync(0xffffffffu, send, half * (32 / kRG));
                }
            }
            const float *xv = x + (PER_HEAD ? 2 : 4) * DKP;
            const float beta = xv[128], qk = xv[129], ah = xv[130];
            const int c = rg & 3;
            const float dot = PER_HEAD ? ah * r[0] : r[0];
            const float mine_u = beta * (xv[(col & 127) + c] - dot);       // of use in the groups below 4
            float u[4], uc = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                u[k] = __shfl_sync(0xffffffffu, mine_u, k * (32 / kRG) + quad);
                uc = c == k ? u[k] : uc;
            }
            if (rg >= 4 && col_ok)
                st_act(static_cast<Tin *>(p.o) + ((long long)sq.begin + t0 + t) * p.ldo + (long long)hv * p.Dv,
                       (size_t)(col + c), fmaf(qk, uc, dot));
#pragma unroll
            for (int i = 0; i < RPL / 4; ++i) {
                const float4 k4 = *reinterpret_cast<const float4 *>((PER_HEAD ? xk : xk + 2 * DKP) + i * 4 * kRG);
                float4 a4 = make_float4(ah, ah, ah, ah);
                if (!PER_HEAD) a4 = *reinterpret_cast<const float4 *>(xk + 3 * DKP + i * 4 * kRG);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 u2 = make_float2(u[c], u[c]);
                    st[2 * i][c] = __ffma2_rn(make_float2(k4.x, k4.y), u2,
                                              __fmul2_rn(make_float2(a4.x, a4.y), st[2 * i][c]));
                    st[2 * i + 1][c] = __ffma2_rn(make_float2(k4.z, k4.w), u2,
                                                  __fmul2_rn(make_float2(a4.z, a4.w), st[2 * i + 1][c]));
                }
            }
        }
        if (!LOOP && t0 + tile < sq.len) { // a sequence longer than the caller said
            __syncthreads();
#pragma unroll
            for (int u = 0; u < TPW; ++u) {
                const int t = t0 + tile + warp * TPW + u;
                if (t < sq.len) raw[u].load(p, (long long)sq.begin + t, h, hv, lane);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        const int r = (i >> 2) * (4 * kRG) + 4 * rg + (i & 3);
        float4 x;
        if ((i & 1) == 0)
            x = make_float4(st[i >> 1][0].x, st[i >> 1][1].x, st[i >> 1][2].x, st[i >> 1][3].x);
        else
            x = make_float4(st[i >> 1][0].y, st[i >> 1][1].y, st[i >> 1][2].y, st[i >> 1][3].y);
        if (col_ok && r < p.Dk) __stcs(reinterpret_cast<float4 *>(S + (size_t)r * p.Dv), x);
    }
}

template <typename Tin, int RPL, bool PER_HEAD, int TPW, bool LOOP>
cudaError_t launch_one(const PackedParams &p, int warps, cudaStream_t s) {
    const int all = (p.Dv + kCW - 1) / kCW;
    const dim3 grid((unsigned)p.N * (unsigned)p.HV, (unsigned)((all + warps - 1) / warps));
    const size_t bytes = (size_t)(LOOP ? 2 : 1) * TPW * warps * token_floats(RPL * kRG, PER_HEAD) * sizeof(float);
    auto kernel = packed_recurrent_kernel<Tin, RPL, PER_HEAD, TPW, LOOP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kernel<<<grid, 32 * warps, bytes, s>>>(p);
    return cudaGetLastError();
}

// One tile (max_len tokens fit a token per warp): four warps a block for up to
// four tokens (241 us for a step of 256 x 32 chains against 250 with eight), a
// block per chain for more, and for long sequences (453 us for a ragged prefill
// of 6 x 16 chains against 525 with two blocks a chain, which prepare every token
// twice).
template <typename Tin, int RPL, bool PER_HEAD>
cudaError_t launch_len(const PackedParams &p, int max_len, cudaStream_t s) {
    const int all = (p.Dv + kCW - 1) / kCW;
    if (max_len <= 4 && all > 4) return launch_one<Tin, RPL, PER_HEAD, 1, false>(p, 4, s);
    if (max_len <= all) return launch_one<Tin, RPL, PER_HEAD, 1, false>(p, all, s);
    return launch_one<Tin, RPL, PER_HEAD, 2, true>(p, all, s);
}

template <typename Tin>
cudaError_t launch_type(const PackedParams &p, int max_len, cudaStream_t s) {
    if (p.Dk <= 64) return p.g_per_head ? launch_len<Tin, 8, true>(p, max_len, s) : launch_len<Tin, 8, false>(p, max_len, s);
    return p.g_per_head ? launch_len<Tin, 16, true>(p, max_len, s) : launch_len<Tin, 16, false>(p, max_len, s);
}

}  // namespace

cudaError_t launch_packed_recurrent(const PackedParams &p, bool bf16, int max_len, cudaStream_t s) {
    return bf16 ? launch_type<__nv_bfloat16>(p, max_len, s) : launch_type<float>(p, max_len, s);
}

cudaError_t read_and_clear_packed_error(unsigned int *out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_packed_error, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_packed_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
