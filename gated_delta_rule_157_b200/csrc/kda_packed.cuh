// Packed batches: N sequences of T rows in all, one after another, each with a
// slot of a state pool.  What the packed kernels share.
#pragma once
#include "kda_internal.cuh"

namespace kda {

// Validated arguments of a packed forward of the delta rule.
struct PackedParams {
    int N, T, P, H, HV, Dk, Dv, group;
    float g_min, scale, l2_eps;
    int l2norm, beta_sigmoid, gate_in, g_per_head;
    int split;                       // the recurrent kernel takes sequences of at most this many rows,
                                     // the chunk kernel (where both are launched) the longer ones
    long long ldq, ldk, ldv, ldg, ldb, ldo;   // elements from one row to the next
    const void *q, *k, *v, *g, *beta;
    const float *A_log, *dt_bias;
    const int *cu;                   // [N + 1] row bounds, or NULL: sequence s is row s
    const int *slots;                // [N], or NULL: sequence s has slot s; negative: skipped
    const unsigned char *fresh;      // [N], or NULL: nonzero starts from a zero state
    float *pool;                     // [P, HV, Dk, Dv]
    void *o;
};

struct PackedConvParams {
    int N, T, P, C, K, head_dim, silu;
    float l2_eps;
    long long ldx, ldy;
    const void *x;
    const float *w, *bias;
    const int *cu, *slots;
    const unsigned char *fresh;
    void *pool;                      // [P, K - 1, C], of x's type
    void *y;
};

// Error word bit: a sequence with row bounds outside [0, T], a slot outside the
// pool, or (both with rows) a slot that an earlier sequence of the call has: skipped.
constexpr unsigned kPackedRange = 2u;

struct PackedSeq {
    int begin, len, slot;
    bool bad;                        // bounds or slot outside their range (the repeat is looked for separately)
};

__device__ __forceinline__ PackedSeq packed_seq(const int *cu, const int *slots, int T, int P, int s) {
    PackedSeq r;
    const int b = cu ? cu[s] : s, e = cu ? cu[s + 1] : s + 1;
    r.slot = slots ? slots[s] : s;
    r.bad = b < 0 || e < b || e > T || r.slot >= P;
    r.begin = r.bad ? 0 : b;
    r.len = r.bad ? 0 : e - b;
    return r;
}

// Whether an earlier sequence names the same slot (one without rows does not count):
// this thread's share of the search (threads tid, tid + step, ...); the caller ORs
// over the threads.
__device__ __forceinline__ bool packed_has_rows(const int *cu, int s) { return !cu || cu[s + 1] != cu[s]; }
__device__ __forceinline__ bool packed_repeat(const int *cu, const int *slots, int s, int slot, int tid, int step) {
    bool hit = false;
    if (slots && slot >= 0)
        for (int i = tid; i < s; i += 8 * step) {
            int v[8];                      // loads in flight together
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i + k * step < s ? slots[i + k * step] : -1;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (v[k] == slot) hit |= packed_has_rows(cu, i + k * step);
        }
    return hit;
}

cudaError_t launch_packed_recurrent(const PackedParams &p, bool bf16, int max_len, cudaStream_t s);
cudaError_t launch_packed_chunk(const PackedParams &p, cudaStream_t s);
// Whether the chunk kernel takes these types and widths, and these rows.
bool packed_chunk_shape(const PackedParams &p, bool bf16);
bool packed_chunk_aligned(const PackedParams &p);
// Sequences of more rows than this go to the chunk kernel where it applies
// (HV = 32, recurrence against chunks: 8 sequences of 8 rows 19 : 30 us, of 16
// 29 : 30, of 64 79 : 30; 64 sequences of 8 rows 87 : 161 us, of 16 204 : 161).
constexpr int kPackedSplit = 12;
cudaError_t launch_packed_conv(const PackedConvParams &p, bool bf16, cudaStream_t s);
// Error words of the packed kernels, read and cleared (after a synchronise).
cudaError_t read_and_clear_packed_error(unsigned int *out);
cudaError_t read_and_clear_packed_chunk_error(unsigned int *out);
cudaError_t read_and_clear_packed_conv_error(unsigned int *out);

}  // namespace kda
