// Group norm over channels-last rows: arguments and launch plan.
#pragma once
#include "kda_internal.cuh"

namespace kda {

struct GroupNormParams {
    int N, L, C, G, D;               // D = C / G channels of a group
    int act;                         // 0 none, 1 SiLU, 2 sigmoid
    float eps;
    const void *x, *gate, *dy;
    const float *weight, *bias;
    void *y, *dx, *dgate;
    float *mean, *rstd;              // [N, G]: written by the forward, read by the backward
    float *dweight, *dbias;
    float *ws;                       // workspace of GroupNormPlan::ws_floats floats
};

// How a call is cut.  Slabs of L * D values that fit the registers of one block
// are done in one pass (`held`); longer ones in three (partial sums per tile of
// rows, their sum, the result).  Depends on sizes and alignment alone.
struct GroupNormPlan {
    bool held;
    int vec;                         // channels per vector access
    int tps, vpt;                    // held: threads per slab (a power of two), vectors per thread
    int gpc, nsub;                   // held: groups and rows n a block has side by side
    int gx, gy;                      // grid
    int cvb;                         // tiled: vectors of a row side by side in a block (a power of two)
    int tiles, rt;                   // tiled: tiles of a slab, rows of a tile
    size_t ws_floats;
};
// `aligned`: every activation pointer is 16-byte aligned.
GroupNormPlan group_norm_plan(int N, int L, int C, int G, bool bf16, bool backward, bool aligned);
cudaError_t launch_group_norm_fwd(const GroupNormParams &p, const GroupNormPlan &pl, bool bf16, cudaStream_t s);
cudaError_t launch_group_norm_bwd(const GroupNormParams &p, const GroupNormPlan &pl, bool bf16, cudaStream_t s);

}  // namespace kda
