// fp8_block.cuh -- shared by the FP8 block-128 product, its gradients and the
// token-block quantiser: the group table of a row matrix.
#pragma once

#include "grouped_common.cuh"
#include "launch.h"

namespace moe {

// Warp 0 fills the tile table of G row groups: group g owns rows offsets[g] ..
// offsets[g+1]-1 of M (one group of all rows when offsets is NULL).  The
// offsets are data on the device, so they are made harmless here: clamped to
// [0, M] and to a running maximum.  Offsets that are in order come out as
// they are; of others no row outside the matrix is touched, and the groups'
// rows still sum to at most M (the capacity of the padded layouts).
__device__ __forceinline__ void build_group_table(TileTable* tt, const int32_t* __restrict__ offsets,
                                                  int G, int M, int BM) {
    const int lane = threadIdx.x & 31;
    if (offsets == nullptr) {
        if (lane == 0) {
            tt->goff[0] = 0;
            tt->goff[1] = M;
            tt->mstart[0] = 0;
            tt->mstart[1] = (M + BM - 1) / BM;
        }
        __syncwarp();
        return;
    }
    // running maximum: each lane over a contiguous chunk, then over the lanes
    const int pero = (G + 1 + 31) / 32;
    const int o0 = min(G + 1, lane * pero), o1 = min(G + 1, o0 + pero);
    int top = 0;
    for (int g = o0; g < o1; ++g) top = max(top, min(M, max(0, offsets[g])));
    int before = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before = max(before, v);
    }
    before = __shfl_up_sync(0xffffffffu, before, 1);
    if (lane == 0) before = 0;
    for (int g = o0; g < o1; ++g) {
        before = max(before, min(M, max(0, offsets[g])));
        tt->goff[g] = before;
    }
    __syncwarp();
    const int per = (G + 31) / 32;
    const int g0 = min(G, lane * per), g1 = min(G, g0 + per);
    int sum = 0;
    for (int g = g0; g < g1; ++g) sum += (tt->goff[g + 1] - tt->goff[g] + BM - 1) / BM;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    int run = incl - sum;
    for (int g = g0; g < g1; ++g) {
        tt->mstart[g] = run;
        run += (tt->goff[g + 1] - tt->goff[g] + BM - 1) / BM;
    }
    if (lane == 31) tt->mstart[G] = incl;
    __syncwarp();
}

// The group that owns tile `tile` of a table with one n-tile per row tile
// (mstart[g] <= tile < mstart[g+1]); tile < mstart[G].
__device__ __forceinline__ int group_of(const TileTable* tt, int G, int tile) {
    int lo = 0, hi = G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tt->mstart[mid] <= tile) lo = mid; else hi = mid;
    }
    return lo;
}

// The output types of the products.
__device__ __forceinline__ void store_out(void* out, int64_t i, float v, int type) {
    if (type == MOE_OUT_F32) {
        static_cast<float*>(out)[i] = v;
    } else if (type == MOE_OUT_F16) {
        const uint32_t h = pack_f16x2_sat(v, 0.0f);
        static_cast<uint16_t*>(out)[i] = (uint16_t)h;
    } else {
        static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
    }
}

}  // namespace moe
