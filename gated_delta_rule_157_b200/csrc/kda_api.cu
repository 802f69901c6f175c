// C ABI of the library (declared in include/kda.h): host-side validation,
// dispatch and launch.  Validation errors return before anything is enqueued.
#include <stdint.h>

#include "kda_group_norm.cuh"
#include "kda_internal.cuh"
#include "kda_packed.cuh"

namespace {

using kda::ChunkParams;
using kda::StepParams;

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

Range range_of(const void *p, size_t bytes) {
    uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + bytes};
}

bool overlaps(Range a, Range b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

kda_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

static kda_status chunk_fwd(const kda_chunk_args *a, void *stream, bool withhold_ready) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->B < 0 || a->T < 0 || a->H < 1 || a->HV < 1 || a->HV % a->H != 0)
        return KDA_ERR_INVALID_ARG;
    if (a->Dk < 1 || a->Dv < 1 || a->chunk < 1) return KDA_ERR_INVALID_ARG;
    if (a->dtype != KDA_DT_F32 && a->dtype != KDA_DT_BF16) return KDA_ERR_INVALID_ARG;
    if (a->algo != KDA_ALGO_AUTO && a->algo != KDA_ALGO_SIMT && a->algo != KDA_ALGO_TC)
        return KDA_ERR_INVALID_ARG;
    if (a->Dk > 128 || a->Dv > 128 || a->chunk > 64) return KDA_ERR_UNSUPPORTED;
    if (!(a->g_min < 0.f) || !(a->l2_eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (a->gate_in_kernel < 0 || a->gate_in_kernel > 2) return KDA_ERR_INVALID_ARG;
    const bool bf16 = a->dtype == KDA_DT_BF16;
    const size_t es = bf16 ? 2 : 4;
    const size_t ntok = (size_t)a->B * a->T;
    const size_t gk = a->g_per_head ? 1 : (size_t)a->Dk;   // gate values per (token, value head)
    if (a->B == 0) return KDA_OK;

    if (ntok > 0) {
        if (!a->q || !a->k || !a->v || !a->g || !a->beta) return KDA_ERR_INVALID_ARG;   // o may be NULL
        if (a->gate_in_kernel && !a->A_log) return KDA_ERR_INVALID_ARG;
        const void *acts[] = {a->q, a->k, a->v, a->g, a->beta, a->o};
        for (const void *p : acts)
            if (!aligned(p, es)) return KDA_ERR_ALIGNMENT;
    }
    const float *fl[] = {a->A_log, a->dt_bias, a->S0, a->S_T, a->M_T, a->S_chunks};
    for (const float *p : fl)
        if (p && !aligned(p, 4)) return KDA_ERR_ALIGNMENT;

    // Aliasing: o must not overlap inputs; S_T / M_T must not overlap o, inputs
    // (S_T == S0 exactly is allowed) or each other.
    const size_t nq = ntok * a->H * a->Dk * es, nv = ntok * a->HV * a->Dv * es;
    const size_t ng = ntok * a->HV * gk * es, nb = ntok * a->HV * es;
    const size_t ns = (size_t)a->B * a->HV * a->Dk * a->Dv * 4;
    const size_t nm = (size_t)a->B * a->HV * a->Dk * a->Dk * 4;
    Range r_in[] = {range_of(a->q, ntok ? nq : 0), range_of(a->k, ntok ? nq : 0),
                    range_of(a->v, ntok ? nv : 0), range_of(a->g, ntok ? ng : 0),
                    range_of(a->beta, ntok ? nb : 0),
                    range_of(a->A_log, a->A_log ? (size_t)a->HV * 4 : 0),
                    range_of(a->dt_bias, a->dt_bias ? (size_t)a->HV * gk * 4 : 0)};
    Range r_s0 = range_of(a->S0, a->S0 ? ns : 0);
    Range r_o = range_of(a->o, (ntok && a->o) ? nv : 0);
    Range r_st = range_of(a->S_T, a->S_T ? ns : 0);
    Range r_mt = range_of(a->M_T, a->M_T ? nm : 0);
    const size_t nchunks = a->T > 0 ? ((size_t)a->T + a->chunk - 1) / a->chunk : 0;
    Range r_sc = range_of(a->S_chunks, a->S_chunks ? ns * nchunks : 0);
    for (Range r : r_in) {
        if (overlaps(r_o, r) || overlaps(r_st, r) || overlaps(r_mt, r) || overlaps(r_sc, r))
            return KDA_ERR_ALIAS;
    }
    if (overlaps(r_o, r_s0) || overlaps(r_o, r_st) || overlaps(r_o, r_mt) || overlaps(r_st, r_mt) ||
        overlaps(r_mt, r_s0))
        return KDA_ERR_ALIAS;
    if (overlaps(r_sc, r_o) || overlaps(r_sc, r_s0) || overlaps(r_sc, r_st) || overlaps(r_sc, r_mt))
        return KDA_ERR_ALIAS;
    if (overlaps(r_st, r_s0) && a->S_T != a->S0) return KDA_ERR_ALIAS;

    ChunkParams p;
    p.B = a->B; p.T = a->T; p.H = a->H; p.HV = a->HV; p.Dk = a->Dk; p.Dv = a->Dv;
    p.C = a->chunk; p.group = a->HV / a->H;
    p.g_min = a->g_min; p.scale = a->scale; p.l2_eps = a->l2_eps;
    p.l2norm = a->qk_l2norm_in_kernel != 0;
    p.beta_sigmoid = a->beta_sigmoid_in_kernel != 0;
    p.gate_in = a->gate_in_kernel;
    p.g_per_head = a->g_per_head != 0;
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta;
    p.A_log = a->A_log; p.dt_bias = a->dt_bias; p.S0 = a->S0;
    p.o = a->o; p.S_T = a->S_T; p.M_T = a->M_T; p.S_chunks = a->S_chunks;
    p.withhold_ready = withhold_ready ? 1 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    if (a->T == 0) return cuda_status(kda::launch_chunk_empty(p, s));

    // The tensor-core kernel's exponent scheme needs g >= g_min: with a
    // caller-given decay or the (unbounded) softplus gate it clamps g there
    // and reports the clamp, so AUTO sends both to the exact SIMT kernel.
    const bool tc_ok = kda::chunk_tc_supported(p, bf16);
    if (withhold_ready && (a->algo != KDA_ALGO_TC || !tc_ok)) return KDA_ERR_UNSUPPORTED;
    if (a->algo == KDA_ALGO_TC) {
        if (!tc_ok) return KDA_ERR_UNSUPPORTED;
        const void *v16[] = {a->q, a->k, a->v, a->g, a->o};
        for (const void *ptr : v16)
            if (!aligned(ptr, 16)) return KDA_ERR_ALIGNMENT;
        return cuda_status(kda::launch_chunk_tc(p, s));
    }
    // A log-decay given directly (no in-kernel gate) may lie below g_min, where
    // the tensor-core kernel's exponent bound does not hold: AUTO takes the
    // SIMT kernel, which is exact for any g <= 0.
    if (a->algo == KDA_ALGO_AUTO && tc_ok && a->gate_in_kernel == 1) {
        bool al16 = true;
        const void *v16[] = {a->q, a->k, a->v, a->g, a->o};
        for (const void *ptr : v16) al16 = al16 && aligned(ptr, 16);
        if (al16) return cuda_status(kda::launch_chunk_tc(p, s));
    }
    return cuda_status(kda::launch_chunk_simt(p, bf16, s));
}

kda_status kda_chunk_fwd(const kda_chunk_args *a, void *stream) { return chunk_fwd(a, stream, false); }

kda_status kda_debug_chunk_stall(const kda_chunk_args *a, void *stream) { return chunk_fwd(a, stream, true); }

kda_status kda_chunk_bwd(const kda_chunk_bwd_args *a, void *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->B < 0 || a->T < 0 || a->H < 1 || a->HV < 1 || a->HV % a->H != 0)
        return KDA_ERR_INVALID_ARG;
    if (a->Dk < 1 || a->Dv < 1 || a->chunk < 1) return KDA_ERR_INVALID_ARG;
    if (a->dtype != KDA_DT_F32 && a->dtype != KDA_DT_BF16) return KDA_ERR_INVALID_ARG;
    if (a->algo != KDA_ALGO_AUTO && a->algo != KDA_ALGO_SIMT && a->algo != KDA_ALGO_TC)
        return KDA_ERR_INVALID_ARG;
    if (a->algo == KDA_ALGO_TC) return KDA_ERR_UNSUPPORTED;
    if (a->Dk > 128 || a->Dv > 128 || a->chunk > 64) return KDA_ERR_UNSUPPORTED;
    if (!(a->g_min < 0.f) || !(a->l2_eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (a->gate_in_kernel < 0 || a->gate_in_kernel > 2) return KDA_ERR_INVALID_ARG;
    if (a->B == 0) return KDA_OK;
    const bool bf16 = a->dtype == KDA_DT_BF16;
    const size_t es = bf16 ? 2 : 4;
    const size_t ntok = (size_t)a->B * a->T;
    const size_t gk = a->g_per_head ? 1 : (size_t)a->Dk;
    if (ntok > 0) {
        if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->S_chunks || !a->dout) return KDA_ERR_INVALID_ARG;
        if (!a->dq || !a->dk || !a->dv || !a->dg || !a->dbeta) return KDA_ERR_INVALID_ARG;
        if (a->gate_in_kernel && !a->A_log) return KDA_ERR_INVALID_ARG;
        const void *acts[] = {a->q, a->k, a->v, a->g, a->beta, a->dout};
        for (const void *p : acts)
            if (!aligned(p, es)) return KDA_ERR_ALIGNMENT;
    }
    const float *fl[] = {a->A_log, a->dt_bias, a->S_chunks, a->dS_T, a->dq, a->dk, a->dv,
                         a->dg, a->dbeta, a->dS0, a->dA_log, a->ddt_bias};
    for (const float *p : fl)
        if (p && !aligned(p, 4)) return KDA_ERR_ALIGNMENT;

    const size_t nq = ntok * a->H * a->Dk, nv = ntok * a->HV * a->Dv;
    const size_t ng = ntok * a->HV * gk, nb = ntok * a->HV;
    const size_t ns = (size_t)a->B * a->HV * a->Dk * a->Dv;
    const size_t nchunks = a->T > 0 ? ((size_t)a->T + a->chunk - 1) / a->chunk : 0;
    const bool gate = a->gate_in_kernel != 0;
    Range r_in[] = {range_of(a->q, ntok ? nq * es : 0), range_of(a->k, ntok ? nq * es : 0),
                    range_of(a->v, ntok ? nv * es : 0), range_of(a->g, ntok ? ng * es : 0),
                    range_of(a->beta, ntok ? nb * es : 0), range_of(a->dout, ntok ? nv * es : 0),
                    range_of(a->A_log, a->A_log ? (size_t)a->HV * 4 : 0),
                    range_of(a->dt_bias, a->dt_bias ? (size_t)a->HV * gk * 4 : 0),
                    range_of(a->S_chunks, a->S_chunks ? ns * nchunks * 4 : 0),
                    range_of(a->dS_T, a->dS_T ? ns * 4 : 0)};
    Range r_out[] = {range_of(a->dq, ntok ? nq * 4 : 0), range_of(a->dk, ntok ? nq * 4 : 0),
                     range_of(a->dv, ntok ? nv * 4 : 0), range_of(a->dg, ntok ? ng * 4 : 0),
                     range_of(a->dbeta, ntok ? nb * 4 : 0), range_of(a->dS0, a->dS0 ? ns * 4 : 0),
                     range_of(gate ? a->dA_log : nullptr, gate && a->dA_log ? (size_t)a->HV * 4 : 0),
                     range_of(gate ? a->ddt_bias : nullptr, gate && a->ddt_bias ? (size_t)a->HV * gk * 4 : 0)};
    const int n_out = sizeof(r_out) / sizeof(r_out[0]);
    for (int i = 0; i < n_out; ++i) {
        for (Range r : r_in)
            if (overlaps(r_out[i], r)) return KDA_ERR_ALIAS;
        for (int j = i + 1; j < n_out; ++j)
            if (overlaps(r_out[i], r_out[j])) return KDA_ERR_ALIAS;
    }

    kda::BwdParams p;
    p.B = a->B; p.T = a->T; p.H = a->H; p.HV = a->HV; p.Dk = a->Dk; p.Dv = a->Dv;
    p.C = a->chunk; p.group = a->HV / a->H;
    p.g_min = a->g_min; p.scale = a->scale; p.l2_eps = a->l2_eps;
    p.l2norm = a->qk_l2norm_in_kernel != 0;
    p.beta_sigmoid = a->beta_sigmoid_in_kernel != 0;
    p.gate_in = a->gate_in_kernel;
    p.g_per_head = a->g_per_head != 0;
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta;
    p.A_log = a->A_log; p.dt_bias = a->dt_bias; p.S_chunks = a->S_chunks;
    p.dout = a->dout; p.dS_T = a->dS_T;
    p.dq = a->dq; p.dk = a->dk; p.dv = a->dv; p.dg = a->dg; p.dbeta = a->dbeta; p.dS0 = a->dS0;
    p.dA_log = gate ? a->dA_log : nullptr;
    p.ddt_bias = gate ? a->ddt_bias : nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    // The q/k/g/beta (and parameter) gradients are accumulated with atomics.
    struct Zero { void *p; size_t bytes; } zeros[] = {
        {p.dq, ntok ? nq * 4 : 0}, {p.dk, ntok ? nq * 4 : 0}, {p.dg, ntok ? ng * 4 : 0},
        {p.dbeta, ntok ? nb * 4 : 0}, {p.dA_log, p.dA_log ? (size_t)a->HV * 4 : 0},
        {p.ddt_bias, p.ddt_bias ? (size_t)a->HV * gk * 4 : 0}};
    for (const Zero &z : zeros) {
        if (z.bytes && cudaMemsetAsync(z.p, 0, z.bytes, s) != cudaSuccess) return KDA_ERR_CUDA;
    }
    return cuda_status(kda::launch_chunk_bwd(p, bf16, s));
}

kda_status kda_step(const kda_step_args *a, void *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->B < 0 || a->H < 1 || a->HV < 1 || a->HV % a->H != 0) return KDA_ERR_INVALID_ARG;
    if (a->Dk < 1 || a->Dv < 1) return KDA_ERR_INVALID_ARG;
    if (a->dtype != KDA_DT_F32 && a->dtype != KDA_DT_BF16) return KDA_ERR_INVALID_ARG;
    if (a->Dk > 128 || a->Dv > 128 || a->Dv % 4 != 0) return KDA_ERR_UNSUPPORTED;
    if (!(a->g_min < 0.f) || !(a->l2_eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (a->gate_in_kernel < 0 || a->gate_in_kernel > 2) return KDA_ERR_INVALID_ARG;
    if (a->B == 0) return KDA_OK;
    const size_t gk = a->g_per_head ? 1 : (size_t)a->Dk;
    if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->S || !a->o) return KDA_ERR_INVALID_ARG;
    if (a->gate_in_kernel && !a->A_log) return KDA_ERR_INVALID_ARG;
    const bool bf16 = a->dtype == KDA_DT_BF16;
    const size_t es = bf16 ? 2 : 4;
    const void *acts[] = {a->q, a->k, a->v, a->g, a->beta, a->o};
    for (const void *p : acts)
        if (!aligned(p, es)) return KDA_ERR_ALIGNMENT;
    if (!aligned(a->S, 16)) return KDA_ERR_ALIGNMENT;
    if ((a->A_log && !aligned(a->A_log, 4)) || (a->dt_bias && !aligned(a->dt_bias, 4)))
        return KDA_ERR_ALIGNMENT;

    const size_t B = a->B;
    Range r_in[] = {range_of(a->q, B * a->H * a->Dk * es), range_of(a->k, B * a->H * a->Dk * es),
                    range_of(a->v, B * a->HV * a->Dv * es), range_of(a->g, B * a->HV * gk * es),
                    range_of(a->beta, B * a->HV * es),
                    range_of(a->A_log, a->A_log ? (size_t)a->HV * 4 : 0),
                    range_of(a->dt_bias, a->dt_bias ? (size_t)a->HV * gk * 4 : 0)};
    Range r_s = range_of(a->S, B * a->HV * a->Dk * a->Dv * 4);
    Range r_o = range_of(a->o, B * a->HV * a->Dv * es);
    for (Range r : r_in)
        if (overlaps(r_o, r) || overlaps(r_s, r)) return KDA_ERR_ALIAS;
    if (overlaps(r_o, r_s)) return KDA_ERR_ALIAS;

    StepParams p;
    p.B = a->B; p.H = a->H; p.HV = a->HV; p.Dk = a->Dk; p.Dv = a->Dv; p.group = a->HV / a->H;
    p.g_min = a->g_min; p.scale = a->scale; p.l2_eps = a->l2_eps;
    p.l2norm = a->qk_l2norm_in_kernel != 0;
    p.beta_sigmoid = a->beta_sigmoid_in_kernel != 0;
    p.gate_in = a->gate_in_kernel;
    p.g_per_head = a->g_per_head != 0;
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta;
    p.A_log = a->A_log; p.dt_bias = a->dt_bias; p.S = a->S; p.o = a->o;
    return cuda_status(kda::launch_step(p, bf16, static_cast<cudaStream_t>(stream)));
}

kda_status kda_compose(int n_seg, int BH, int Dk, int Dv, const float *M, const float *S_seg,
                       const float *S_init, float *S_in, void *stream) {
    if (n_seg < 0 || BH < 0 || Dk < 1 || Dv < 1) return KDA_ERR_INVALID_ARG;
    if (Dk > 128 || Dv > 128) return KDA_ERR_UNSUPPORTED;
    if (BH == 0) return KDA_OK;
    if (!S_in || (n_seg > 0 && (!M || !S_seg))) return KDA_ERR_INVALID_ARG;
    const float *ps[] = {M, S_seg, S_init, S_in};
    for (const float *p : ps)
        if (p && !aligned(p, 4)) return KDA_ERR_ALIGNMENT;
    const size_t st = (size_t)BH * Dk * Dv * 4, mt = (size_t)BH * Dk * Dk * 4;
    Range r_out = range_of(S_in, st * (n_seg + 1));
    if (overlaps(r_out, range_of(M, M ? mt * n_seg : 0)) ||
        overlaps(r_out, range_of(S_seg, S_seg ? st * n_seg : 0)) ||
        overlaps(r_out, range_of(S_init, S_init ? st : 0)))
        return KDA_ERR_ALIAS;
    return cuda_status(kda::launch_compose(n_seg, BH, Dk, Dv, M, S_seg, S_init, S_in,
                                           static_cast<cudaStream_t>(stream)));
}

kda_status kda_short_conv(const kda_conv_args *a, void *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->B < 0 || a->T < 0 || a->C < 1 || a->K < 1 || a->K > 4 || !(a->l2_eps >= 0.f))
        return KDA_ERR_INVALID_ARG;
    if (a->head_dim != 0 && a->head_dim != 128) return KDA_ERR_UNSUPPORTED;
    if (a->C % 128 != 0) return KDA_ERR_UNSUPPORTED;
    if (a->B == 0) return KDA_OK;
    const size_t ntok = (size_t)a->B * a->T, es = 2;
    if (!a->w || (ntok > 0 && (!a->x || !a->y))) return KDA_ERR_INVALID_ARG;
    // the kernels move 8 channels (16 bytes) per lane
    const void *p16[] = {a->x, a->y, a->state_in, a->state_out};
    for (const void *p : p16)
        if (p && !aligned(p, 16)) return KDA_ERR_ALIGNMENT;
    if (!aligned(a->w, 4) || (a->bias && !aligned(a->bias, 4))) return KDA_ERR_ALIGNMENT;
    const size_t nx = ntok * a->C * es, ns = (size_t)a->B * (a->K - 1) * a->C * es;
    Range r_y = range_of(a->y, ntok ? nx : 0), r_so = range_of(a->state_out, a->state_out ? ns : 0);
    Range r_in[] = {range_of(a->x, ntok ? nx : 0), range_of(a->state_in, a->state_in ? ns : 0),
                    range_of(a->w, (size_t)a->C * a->K * 4), range_of(a->bias, a->bias ? (size_t)a->C * 4 : 0)};
    for (Range r : r_in)
        if (overlaps(r_y, r) || overlaps(r_so, r)) return KDA_ERR_ALIAS;
    if (overlaps(r_y, r_so)) return KDA_ERR_ALIAS;
    kda::ConvParams p;
    p.B = a->B; p.T = a->T; p.C = a->C; p.K = a->K; p.head_dim = a->head_dim; p.silu = a->silu != 0;
    p.l2_eps = a->l2_eps;
    p.x = a->x; p.w = a->w; p.bias = a->bias; p.state_in = a->state_in; p.y = a->y; p.state_out = a->state_out;
    return cuda_status(kda::launch_short_conv(p, static_cast<cudaStream_t>(stream)));
}

kda_status kda_output_gate(const kda_gate_args *a, void *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->N < 0 || a->HV < 1 || a->D < 1 || !(a->eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (a->D != 128) return KDA_ERR_UNSUPPORTED;
    if (a->N == 0) return KDA_OK;
    if (!a->o || !a->gate || !a->y) return KDA_ERR_INVALID_ARG;
    const void *p8[] = {a->o, a->gate, a->y};
    for (const void *p : p8)
        if (!aligned(p, 8)) return KDA_ERR_ALIGNMENT;
    if (a->weight && !aligned(a->weight, 4)) return KDA_ERR_ALIGNMENT;
    const size_t n = (size_t)a->N * a->HV * a->D * 2;
    Range r_y = range_of(a->y, n);
    if (overlaps(r_y, range_of(a->o, n)) || overlaps(r_y, range_of(a->gate, n)) ||
        overlaps(r_y, range_of(a->weight, a->weight ? (size_t)a->D * 4 : 0)))
        return KDA_ERR_ALIAS;
    kda::GateParams p;
    p.N = a->N; p.HV = a->HV; p.D = a->D; p.eps = a->eps;
    p.o = a->o; p.gate = a->gate; p.weight = a->weight; p.y = a->y;
    return cuda_status(kda::launch_output_gate(p, static_cast<cudaStream_t>(stream)));
}

// Rows a strided activation spans: T rows of `row` elements, `ld` apart.
static size_t span_bytes(long long T, long long ld, size_t row, size_t es) {
    return T > 0 ? ((size_t)(T - 1) * (size_t)ld + row) * es : 0;
}

kda_status kda_packed_fwd(const kda_packed_args *a, void *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->N < 0 || a->T < 0 || a->P < 0 || a->H < 1 || a->HV < 1 || a->HV % a->H != 0) return KDA_ERR_INVALID_ARG;
    if (a->Dk < 1 || a->Dv < 1 || a->max_seqlen < 0 || a->T > 0x7FFFFFFF - 4096) return KDA_ERR_INVALID_ARG;
    if (a->dtype != KDA_DT_F32 && a->dtype != KDA_DT_BF16) return KDA_ERR_INVALID_ARG;
    if (a->algo != KDA_ALGO_AUTO && a->algo != KDA_ALGO_SIMT && a->algo != KDA_ALGO_TC) return KDA_ERR_INVALID_ARG;
    if (!(a->g_min < 0.f) || !(a->l2_eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (a->gate_in_kernel < 0 || a->gate_in_kernel > 2) return KDA_ERR_INVALID_ARG;
    if (a->Dk > 128 || a->Dv > 128 || a->Dv % 4 != 0) return KDA_ERR_UNSUPPORTED;
    if ((long long)a->N * a->HV > 0x7FFFFFFFll) return KDA_ERR_UNSUPPORTED;     // the grid
    if (!a->cu_seqlens && a->N != a->T) return KDA_ERR_INVALID_ARG;
    if (!a->slots && a->N > a->P) return KDA_ERR_INVALID_ARG;
    if (a->N == 0 || a->T == 0) return KDA_OK;
    if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->o) return KDA_ERR_INVALID_ARG;
    if (a->P > 0 && !a->pool) return KDA_ERR_INVALID_ARG;
    if (a->gate_in_kernel && !a->A_log) return KDA_ERR_INVALID_ARG;
    const bool bf16 = a->dtype == KDA_DT_BF16;
    const size_t es = bf16 ? 2 : 4, gk = a->g_per_head ? 1 : (size_t)a->Dk;
    const size_t rq = (size_t)a->H * a->Dk, rv = (size_t)a->HV * a->Dv, rg = a->HV * gk, rb = a->HV;
    if (a->ld_q < (long long)rq || a->ld_k < (long long)rq || a->ld_v < (long long)rv || a->ld_g < (long long)rg ||
        a->ld_beta < (long long)rb || a->ld_o < (long long)rv)
        return KDA_ERR_INVALID_ARG;
    const void *acts[] = {a->q, a->k, a->v, a->g, a->beta, a->o};
    for (const void *p : acts)
        if (!aligned(p, es)) return KDA_ERR_ALIGNMENT;
    const void *p4[] = {a->A_log, a->dt_bias, a->cu_seqlens, a->slots};
    for (const void *p : p4)
        if (p && !aligned(p, 4)) return KDA_ERR_ALIGNMENT;
    if (!aligned(a->pool, 16)) return KDA_ERR_ALIGNMENT;

    Range r_in[] = {range_of(a->q, span_bytes(a->T, a->ld_q, rq, es)),
                    range_of(a->k, span_bytes(a->T, a->ld_k, rq, es)),
                    range_of(a->v, span_bytes(a->T, a->ld_v, rv, es)),
                    range_of(a->g, span_bytes(a->T, a->ld_g, rg, es)),
                    range_of(a->beta, span_bytes(a->T, a->ld_beta, rb, es)),
                    range_of(a->A_log, a->A_log ? (size_t)a->HV * 4 : 0),
                    range_of(a->dt_bias, a->dt_bias ? a->HV * gk * 4 : 0),
                    range_of(a->cu_seqlens, a->cu_seqlens ? ((size_t)a->N + 1) * 4 : 0),
                    range_of(a->slots, a->slots ? (size_t)a->N * 4 : 0),
                    range_of(a->fresh, a->fresh ? (size_t)a->N : 0)};
    Range r_pool = range_of(a->pool, (size_t)a->P * a->HV * a->Dk * a->Dv * 4);
    Range r_o = range_of(a->o, span_bytes(a->T, a->ld_o, rv, es));
    for (Range r : r_in)
        if (overlaps(r_o, r) || overlaps(r_pool, r)) return KDA_ERR_ALIAS;
    if (overlaps(r_o, r_pool)) return KDA_ERR_ALIAS;

    kda::PackedParams p;
    p.N = a->N; p.T = a->T; p.P = a->P; p.H = a->H; p.HV = a->HV; p.Dk = a->Dk; p.Dv = a->Dv;
    p.group = a->HV / a->H;
    p.g_min = a->g_min; p.scale = a->scale; p.l2_eps = a->l2_eps;
    p.l2norm = a->qk_l2norm_in_kernel != 0;
    p.beta_sigmoid = a->beta_sigmoid_in_kernel != 0;
    p.gate_in = a->gate_in_kernel;
    p.g_per_head = a->g_per_head != 0;
    p.ldq = a->ld_q; p.ldk = a->ld_k; p.ldv = a->ld_v; p.ldg = a->ld_g; p.ldb = a->ld_beta; p.ldo = a->ld_o;
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta;
    p.A_log = a->A_log; p.dt_bias = a->dt_bias;
    p.cu = a->cu_seqlens; p.slots = a->slots; p.fresh = a->fresh;
    p.pool = a->pool; p.o = a->o;
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    // What the lengths can be: one row each without bounds, else the caller's bound or all rows.
    int max_len = a->cu_seqlens ? a->T : 1;
    if (a->cu_seqlens && a->max_seqlen > 0 && a->max_seqlen < max_len) max_len = a->max_seqlen;
    constexpr int kAll = 0x7FFFFFFF;
    if (a->algo == KDA_ALGO_TC) {
        if (!kda::packed_chunk_shape(p, bf16)) return KDA_ERR_UNSUPPORTED;
        if (!kda::packed_chunk_aligned(p)) return KDA_ERR_ALIGNMENT;
        p.split = 0;
        return cuda_status(kda::launch_packed_chunk(p, s));
    }
    const bool chunk = a->algo == KDA_ALGO_AUTO && max_len > kda::kPackedSplit && kda::packed_chunk_shape(p, bf16) &&
                       kda::packed_chunk_aligned(p);
    p.split = chunk ? kda::kPackedSplit : kAll;
    if (chunk) {
        const kda_status st = cuda_status(kda::launch_packed_chunk(p, s));
        if (st != KDA_OK) return st;
    }
    return cuda_status(kda::launch_packed_recurrent(p, bf16, max_len, s));
}

kda_status kda_packed_conv(const kda_packed_conv_args *a, void *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->N < 0 || a->T < 0 || a->P < 0 || a->C < 1 || a->K < 1 || a->K > 4 || !(a->l2_eps >= 0.f))
        return KDA_ERR_INVALID_ARG;
    if (a->dtype != KDA_DT_F32 && a->dtype != KDA_DT_BF16) return KDA_ERR_INVALID_ARG;
    if (a->T > 0x7FFFFFFF - 4096) return KDA_ERR_INVALID_ARG;
    if (a->head_dim != 0 && a->head_dim != 128) return KDA_ERR_UNSUPPORTED;
    if (a->C % 128 != 0) return KDA_ERR_UNSUPPORTED;
    if (!a->cu_seqlens && a->N != a->T) return KDA_ERR_INVALID_ARG;
    if (!a->slots && a->N > a->P && a->K > 1) return KDA_ERR_INVALID_ARG;
    if (a->N == 0 || a->T == 0) return KDA_OK;
    if (!a->x || !a->w || !a->y || (a->K > 1 && a->P > 0 && !a->pool)) return KDA_ERR_INVALID_ARG;
    if (a->ld_x < a->C || a->ld_y < a->C) return KDA_ERR_INVALID_ARG;
    const bool bf16 = a->dtype == KDA_DT_BF16;
    const size_t es = bf16 ? 2 : 4;
    const void *p16[] = {a->x, a->y, a->pool};
    for (const void *p : p16)
        if (p && !aligned(p, 16)) return KDA_ERR_ALIGNMENT;
    if (a->ld_x * es % 16 != 0 || a->ld_y * es % 16 != 0) return KDA_ERR_ALIGNMENT;
    const void *p4[] = {a->w, a->bias, a->cu_seqlens, a->slots};
    for (const void *p : p4)
        if (p && !aligned(p, 4)) return KDA_ERR_ALIGNMENT;
    Range r_in[] = {range_of(a->x, span_bytes(a->T, a->ld_x, a->C, es)), range_of(a->w, (size_t)a->C * a->K * 4),
                    range_of(a->bias, a->bias ? (size_t)a->C * 4 : 0),
                    range_of(a->cu_seqlens, a->cu_seqlens ? ((size_t)a->N + 1) * 4 : 0),
                    range_of(a->slots, a->slots ? (size_t)a->N * 4 : 0),
                    range_of(a->fresh, a->fresh ? (size_t)a->N : 0)};
    Range r_y = range_of(a->y, span_bytes(a->T, a->ld_y, a->C, es));
    Range r_pool = range_of(a->pool, a->pool ? (size_t)a->P * (a->K - 1) * a->C * es : 0);
    for (Range r : r_in)
        if (overlaps(r_y, r) || overlaps(r_pool, r)) return KDA_ERR_ALIAS;
    if (overlaps(r_y, r_pool)) return KDA_ERR_ALIAS;
    kda::PackedConvParams p;
    p.N = a->N; p.T = a->T; p.P = a->K > 1 || a->slots ? a->P : a->N;
    p.C = a->C; p.K = a->K; p.head_dim = a->head_dim; p.silu = a->silu != 0;
    p.l2_eps = a->l2_eps;
    p.ldx = a->ld_x; p.ldy = a->ld_y;
    p.x = a->x; p.w = a->w; p.bias = a->bias; p.cu = a->cu_seqlens; p.slots = a->slots; p.fresh = a->fresh;
    p.pool = a->pool; p.y = a->y;
    return cuda_status(kda::launch_packed_conv(p, bf16, static_cast<cudaStream_t>(stream)));
}

// The plan reads activations in vectors when every one of them starts on 16
// bytes; rows and groups keep that alignment where their sizes allow it.
static bool group_norm_sizes(int N, int L, int C, int G, int dtype) {
    return N >= 0 && L >= 1 && C >= 1 && G >= 1 && C % G == 0 && (dtype == KDA_DT_F32 || dtype == KDA_DT_BF16);
}

// What the kernels count in an int: rows, the values of a slab and channels, with room
// for a step beyond the last (at most 2 x 65535 x 256 rows); and the grid's limits.
static bool group_norm_supported(int N, int L, int C, int G, int dtype, bool backward) {
    constexpr long long most = 0x7FFFFFFFll - (1ll << 26);
    if ((long long)N * L > most || (long long)L * (C / G) > most || (long long)N * G + C > most) return false;
    for (int aligned = 0; N > 0 && aligned < 2; ++aligned)
        if (kda::group_norm_plan(N, L, C, G, dtype == KDA_DT_BF16, backward, aligned != 0).gy > 65535) return false;
    return true;
}

unsigned long long kda_group_norm_workspace(int N, int L, int C, int G, int dtype, int backward) {
    if (!group_norm_sizes(N, L, C, G, dtype) || N == 0 || !group_norm_supported(N, L, C, G, dtype, backward != 0)) return 0;
    const bool bf16 = dtype == KDA_DT_BF16;
    // the larger of the plans with and without 16-byte aligned pointers
    const size_t a = kda::group_norm_plan(N, L, C, G, bf16, backward != 0, true).ws_floats;
    const size_t b = kda::group_norm_plan(N, L, C, G, bf16, backward != 0, false).ws_floats;
    return (a > b ? a : b) * sizeof(float);
}

static kda_status group_norm(const kda_group_norm_args *a, void *stream, bool backward) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (!group_norm_sizes(a->N, a->L, a->C, a->G, a->dtype) || !(a->eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (a->act < KDA_ACT_NONE || a->act > KDA_ACT_SIGMOID) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = a->dtype == KDA_DT_BF16;
    const size_t es = bf16 ? 2 : 4;
    const size_t nx = (size_t)a->N * a->L * a->C * es, nc = (size_t)a->C * 4, ns = (size_t)a->N * a->G * 4;
    if (!group_norm_supported(a->N, a->L, a->C, a->G, a->dtype, backward)) return KDA_ERR_UNSUPPORTED;
    if (backward && a->dgate && !a->gate) return KDA_ERR_INVALID_ARG;
    const float *f4[] = {a->weight, a->bias, a->mean, a->rstd, a->dweight, a->dbias};
    for (const float *p : f4)
        if (p && !aligned(p, 4)) return KDA_ERR_ALIGNMENT;
    if (a->N == 0) {
        if (backward && a->dweight && cudaMemsetAsync(a->dweight, 0, nc, s) != cudaSuccess) return KDA_ERR_CUDA;
        if (backward && a->dbias && cudaMemsetAsync(a->dbias, 0, nc, s) != cudaSuccess) return KDA_ERR_CUDA;
        return KDA_OK;
    }
    if (!a->x || !a->mean || !a->rstd || (backward ? !a->dy : !a->y)) return KDA_ERR_INVALID_ARG;
    const unsigned long long need = kda_group_norm_workspace(a->N, a->L, a->C, a->G, a->dtype, backward);
    if (need && !a->workspace) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->workspace, 16)) return KDA_ERR_ALIGNMENT;
    const void *acts[] = {a->x, a->gate, backward ? a->dy : a->y, backward ? a->dx : nullptr,
                          backward ? a->dgate : nullptr};
    bool vec = true;
    for (const void *p : acts) {
        if (!aligned(p, es)) return KDA_ERR_ALIGNMENT;
        vec = vec && aligned(p, 16);
    }
    Range in[] = {range_of(a->x, nx), range_of(a->gate, a->gate ? nx : 0),
                  range_of(a->weight, a->weight ? nc : 0), range_of(a->bias, a->bias ? nc : 0),
                  range_of(a->dy, backward ? nx : 0), range_of(a->mean, backward ? ns : 0),
                  range_of(a->rstd, backward ? ns : 0)};
    Range out[] = {range_of(a->y, backward ? 0 : nx), range_of(a->mean, backward ? 0 : ns),
                   range_of(a->rstd, backward ? 0 : ns), range_of(a->dx, backward && a->dx ? nx : 0),
                   range_of(a->dgate, backward && a->dgate ? nx : 0),
                   range_of(a->dweight, backward && a->dweight ? nc : 0),
                   range_of(a->dbias, backward && a->dbias ? nc : 0),
                   range_of(a->workspace, need)};
    const int n_out = sizeof(out) / sizeof(out[0]);
    for (int i = 0; i < n_out; ++i) {
        for (Range r : in)
            if (overlaps(out[i], r)) return KDA_ERR_ALIAS;
        for (int j = i + 1; j < n_out; ++j)
            if (overlaps(out[i], out[j])) return KDA_ERR_ALIAS;
    }
    kda::GroupNormParams p;
    p.N = a->N; p.L = a->L; p.C = a->C; p.G = a->G; p.D = a->C / a->G;
    p.act = a->act; p.eps = a->eps;
    p.x = a->x; p.gate = a->gate; p.dy = a->dy; p.weight = a->weight; p.bias = a->bias;
    p.y = a->y; p.dx = a->dx; p.dgate = a->dgate; p.mean = a->mean; p.rstd = a->rstd;
    p.dweight = a->dweight; p.dbias = a->dbias; p.ws = static_cast<float *>(a->workspace);
    const kda::GroupNormPlan pl = kda::group_norm_plan(a->N, a->L, a->C, a->G, bf16, backward, vec);
    return cuda_status(backward ? kda::launch_group_norm_bwd(p, pl, bf16, s) : kda::launch_group_norm_fwd(p, pl, bf16, s));
}

kda_status kda_group_norm_fwd(const kda_group_norm_args *a, void *stream) { return group_norm(a, stream, false); }

kda_status kda_group_norm_bwd(const kda_group_norm_args *a, void *stream) { return group_norm(a, stream, true); }

kda_status kda_device_status(void *stream) {
    unsigned int word = 0, more[5] = {};
    cudaError_t e = kda::read_and_clear_device_error(static_cast<cudaStream_t>(stream), &word);
    if (e == cudaSuccess) e = kda::read_and_clear_step_error(&more[0]);
    if (e == cudaSuccess) e = kda::read_and_clear_conv_error(&more[1]);
    if (e == cudaSuccess) e = kda::read_and_clear_packed_error(&more[2]);
    if (e == cudaSuccess) e = kda::read_and_clear_packed_chunk_error(&more[3]);
    if (e == cudaSuccess) e = kda::read_and_clear_packed_conv_error(&more[4]);
    if (e != cudaSuccess) return KDA_ERR_CUDA;
    for (unsigned int w : more) word |= w;
    if (word & 1u) return KDA_ERR_TIMEOUT;
    return (word & 2u) ? KDA_ERR_RANGE : KDA_OK;
}

const char *kda_status_string(kda_status s) {
    switch (s) {
        case KDA_OK: return "KDA_OK";
        case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG";
        case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED";
        case KDA_ERR_ALIGNMENT: return "KDA_ERR_ALIGNMENT";
        case KDA_ERR_ALIAS: return "KDA_ERR_ALIAS";
        case KDA_ERR_CUDA: return "KDA_ERR_CUDA";
        case KDA_ERR_TIMEOUT: return "KDA_ERR_TIMEOUT";
        case KDA_ERR_RANGE: return "KDA_ERR_RANGE";
    }
    return "KDA_ERR_UNKNOWN";
}

int kda_version(void) { return 200; }

}  // extern "C"
