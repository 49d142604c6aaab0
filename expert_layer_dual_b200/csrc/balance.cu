// balance.cu -- the router's training side: the load-balance loss with its
// per-expert counts, and the gradient of the router logits.
//
// For logits l [T][E], the selected ids [T][k] and an optional token mask, with
// P[t] = softmax(l[t]) over all E experts and n the number of tokens that count:
//   c_e  = assignments of counted tokens to expert e,   f_e = E c_e / (k n),
//   m_e  = (1/n) sum_t P[t][e],                         loss = coef sum_e f_e m_e,
// and for upstream gradients dloss (of the loss) and dw [T][k] (of the top-k
// weights w), the gradient of the logits (the counts are constants):
//   g_e      = dloss coef / n * P_e ((f_e - 1) - sum_j (f_j - 1) P_j)
//            + renormalised weights:  sum_{j: id_j = e} w_j (dw_j - sum_i w_i dw_i)
//            | softmax over all E:    P_e (sum_{j: id_j = e} dw_j - sum_i w_i dw_i).
// f_e - 1 stands in the place of f_e because the P sum to one: near balance f_e is
// near 1, and the difference of two FP32 values near 1 would keep few bits; f_e - 1
// = (E c_e - k n) / (k n) has an exact integer numerator.
//
// Both kernels give a warp a row, its E <= 256 values in registers (eight per
// lane), and read and write each value once: bound by HBM for many tokens and by
// launch latency for few.  Sums are FP32 within a row and over a warp's rows
// (a few dozen to a few hundred), FP64 over blocks; no atomic on a float, so the
// results do not depend on scheduling.
#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr int kPer = 8;        // values of a row per lane (E <= 256)
constexpr int kWarps = 8;      // warps per block of the many-block kernels
constexpr int kOneWarps = 32;  // warps of the one-block kernel
constexpr int kColBlock = 8;   // experts per block of k_balance_finish

// The column of value i of this lane: VEC: two runs of four consecutive
// columns per lane (16-byte accesses, E % 4 == 0); else every 32nd column.
template <bool VEC>
__device__ __forceinline__ int col_of(int i, int lane) {
    return VEC ? (i >> 2) * 128 + lane * 4 + (i & 3) : i * 32 + lane;
}

template <bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float* v) {
    if (VEC) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int c = q * 128 + lane * 4;
            float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (c < E) f = *reinterpret_cast<const float4*>(row + c);
            v[4 * q] = f.x;
            v[4 * q + 1] = f.y;
            v[4 * q + 2] = f.z;
            v[4 * q + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = i * 32 + lane;
            v[i] = c < E ? row[c] : -INFINITY;
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store_row(float* __restrict__ row, int E, int lane, const float* v) {
    if (VEC) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int c = q * 128 + lane * 4;
            if (c < E)
                *reinterpret_cast<float4*>(row + c) =
                    make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = i * 32 + lane;
            if (c < E) row[c] = v[i];
        }
    }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// v <- softmax of the row held across the warp.  A row with no finite logit
// (every entry -inf) becomes zeros: it selects nothing.
__device__ __forceinline__ void softmax_row(float* v) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, v[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        v[i] = expf(v[i] - m);
        s += v[i];
    }
    s = warp_sum(s);
    const float inv = s > 0.0f ? 1.0f / s : (s == 0.0f ? 0.0f : s);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] *= inv;
}

__device__ __forceinline__ double balance_fraction(int count, int E, double kn) {
    return kn > 0.0 ? (double)count * E / kn : 0.0;
}

// ---------------------------------------------------------------------------
// Loss, first pass: each warp takes every (warps)th token, keeps the sums of
// its tokens' probabilities in registers (a lane always holds the same
// columns) and counts the assignments in shared memory (integers); the block's
// sums go to its row of the partials.  ONE: a single block, which finishes the
// result itself (few tokens: one launch).
// ---------------------------------------------------------------------------
template <int WARPS>
struct RowsSmem {
    float psum[WARPS][256];
    int cnt[256];
    int tokens, bad;
    double term[8];
};

template <bool VEC, bool ONE, int WARPS>
__global__ void __launch_bounds__(WARPS * 32)
    k_balance_rows(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                   const uint8_t* __restrict__ mask, int T, int E, int k, BalancePartials part,
                   BalanceOut out) {
    __shared__ RowsSmem<WARPS> sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < 256; e += WARPS * 32) sm.cnt[e] = 0;
    if (tid == 0) sm.tokens = sm.bad = 0;
    __syncthreads();
    pdl_wait();  // the logits and ids come from the previous kernels
    pdl_trigger();

    float acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
    int tokens = 0, bad = 0;
    const int step = gridDim.x * WARPS;
    for (int64_t t0 = blockIdx.x * WARPS + warp; t0 < T; t0 += 2 * (int64_t)step) {
        // two tokens at a time: two rows in flight per warp
        float v[2][kPer];
        bool on[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t t = t0 + (int64_t)u * step;
            on[u] = t < T && (mask == nullptr || mask[t] != 0);
            if (on[u]) load_row<VEC>(logits + t * E, E, lane, v[u]);
            if (on[u] && lane < k) {
                const int id = ids[t * k + lane];
                if (id >= 0 && id < E) atomicAdd(&sm.cnt[id], 1);
                else bad = 1;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (!on[u]) continue;  // the same for the whole warp
            softmax_row(v[u]);
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] += v[u][i];
            ++tokens;
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = col_of<VEC>(i, lane);
        if (c < 256) sm.psum[warp][c] = acc[i];
    }
    if (bad) sm.bad = 1;
    if (lane == 0 && tokens) atomicAdd(&sm.tokens, tokens);
    __syncthreads();

    if (!ONE) {
        for (int e = tid; e < E; e += WARPS * 32) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s += sm.psum[w][e];
            part.psum[(int64_t)blockIdx.x * E + e] = s;
            part.cnt[(int64_t)blockIdx.x * E + e] = sm.cnt[e];
        }
        if (tid == 0) {
            part.info[2 * blockIdx.x] = sm.tokens;
            part.info[2 * blockIdx.x + 1] = sm.bad;
            if (blockIdx.x == 0) *part.arrived = 0;
        }
        return;
    }
    double term = 0.0;
    if (tid < 256) {
        const int n = sm.tokens;
        if (tid < E) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s += sm.psum[w][tid];
            const double mean = n > 0 ? (double)s / n : 0.0;
            out.prob_mean[tid] = (float)mean;
            out.counts[tid] = sm.cnt[tid];
            term = balance_fraction(sm.cnt[tid], E, (double)k * n) * mean;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
        if (lane == 0) sm.term[warp] = term;
    }
    __syncthreads();
    if (tid == 0) {
        double s = 0.0;
        for (int w = 0; w < 8; ++w) s += sm.term[w];
        *out.loss = (float)(out.coef * s);
        *out.tokens = sm.tokens;
        *out.status = sm.bad ? MOE_ERR_DEVICE_BAD_INDEX : MOE_OK;
    }
}

// Loss, second pass: a block sums the partials of kColBlock experts over the
// first pass's blocks (in FP64, a fixed order) and leaves each expert's share
// of the loss; the last block to arrive adds the E shares in order.
__global__ void __launch_bounds__(256)
    k_balance_finish(int E, int k, int nblocks, BalancePartials part, BalanceOut out) {
    __shared__ double s_sum[32][kColBlock];
    __shared__ int s_cnt[32][kColBlock];
    __shared__ int s_tokens[8], s_bad[8], s_last;
    __shared__ double s_term[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.x * kColBlock + tid % kColBlock, slice = tid / kColBlock;
    double sum = 0.0;
    int cnt = 0;
    if (e < E)
#pragma unroll 4
        for (int b = slice; b < nblocks; b += 32) {
            sum += part.psum[(int64_t)b * E + e];
            cnt += part.cnt[(int64_t)b * E + e];
        }
    int tokens = 0, bad = 0;
    for (int b = tid; b < nblocks; b += 256) {
        tokens += part.info[2 * b];
        bad |= part.info[2 * b + 1];
    }
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    bad = __reduce_or_sync(0xffffffffu, bad);
    s_sum[slice][tid % kColBlock] = sum;
    s_cnt[slice][tid % kColBlock] = cnt;
    if (lane == 0) {
        s_tokens[warp] = tokens;
        s_bad[warp] = bad;
    }
    __syncthreads();
    int n = 0, any = 0;
    for (int w = 0; w < 8; ++w) {
        n += s_tokens[w];
        any |= s_bad[w];
    }
    if (tid < kColBlock && e < E) {
        double s = 0.0;
        int c = 0;
        for (int i = 0; i < 32; ++i) {
            s += s_sum[i][tid];
            c += s_cnt[i][tid];
        }
        const double mean = n > 0 ? s / n : 0.0;
        out.prob_mean[e] = (float)mean;
        out.counts[e] = c;
        part.term[e] = balance_fraction(c, E, (double)k * n) * mean;
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(part.arrived, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    double term = tid < E ? __ldcg(part.term + tid) : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
    if (lane == 0) s_term[warp] = term;
    __syncthreads();
    if (tid == 0) {
        double s = 0.0;
        for (int w = 0; w < 8; ++w) s += s_term[w];
        *out.loss = (float)(out.coef * s);
        *out.tokens = n;
        *out.status = any ? MOE_ERR_DEVICE_BAD_INDEX : MOE_OK;
    }
}

// ---------------------------------------------------------------------------
// Gradient of the logits: a warp per row, the softmax recomputed from the
// logits (cheaper than a saved row: nothing more is read).  Masked tokens get
// zeros and their logits are not read.
// ---------------------------------------------------------------------------
template <bool VEC>
__global__ void __launch_bounds__(kWarps * 32)
    k_route_backward(RouteBackwardArgs a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const int E = a.E, k = a.k;
    const bool balance = a.dloss != nullptr, need_p = balance || !a.renorm;
    float f1[kPer], cb = 0.0f;  // f_e - 1 of this lane's columns; dloss coef / n
#pragma unroll
    for (int i = 0; i < kPer; ++i) f1[i] = 0.0f;
    if (balance) {
        const int n = *a.tokens;
        const double kn = (double)k * n;
        cb = n > 0 ? (float)((double)*a.dloss * a.coef / n) : 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = col_of<VEC>(i, lane);
            if (c < E && n > 0) f1[i] = (float)(((double)a.counts[c] * E - kn) / kn);
        }
    }
    const int step = gridDim.x * kWarps;
    for (int64_t t = blockIdx.x * kWarps + warp; t < a.T; t += step) {
        float g[kPer];
        if (a.mask != nullptr && a.mask[t] == 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) g[i] = 0.0f;
            store_row<VEC>(a.dlogits + t * E, E, lane, g);
            continue;
        }
        float p[kPer];
        if (need_p) load_row<VEC>(a.logits + t * E, E, lane, p);
        int id = -1;
        float w = 0.0f, d = 0.0f;
        if (a.dw != nullptr && lane < k) {
            id = a.ids[t * k + lane];
            w = a.w[t * k + lane];
            d = a.dw[t * k + lane];
        }
        if (need_p) softmax_row(p);
#pragma unroll
        for (int i = 0; i < kPer; ++i) g[i] = 0.0f;
        if (a.dw != nullptr) {
            const float dot = warp_sum(w * d);
            const float mine = a.renorm ? w * (d - dot) : d;
            for (int j = 0; j < k; ++j) {
                const int idj = __shfl_sync(0xffffffffu, id, j);
                const float gj = __shfl_sync(0xffffffffu, mine, j);
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (idj == col_of<VEC>(i, lane)) g[i] += gj;
            }
            if (!a.renorm) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) g[i] = p[i] * (g[i] - dot);
            }
        }
        if (balance) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) s = fmaf(f1[i], p[i], s);
            s = warp_sum(s);
#pragma unroll
            for (int i = 0; i < kPer; ++i) g[i] = fmaf(cb * p[i], f1[i] - s, g[i]);
        }
        store_row<VEC>(a.dlogits + t * E, E, lane, g);
    }
}

inline bool vec_ok(int E) { return E % 4 == 0; }

}  // namespace

int balance_blocks(int T) {
    if (T <= kBalanceOneBlock) return 1;
    const int want = (T + 2 * kWarps - 1) / (2 * kWarps);
    return want < kBalanceMaxBlocks ? want : kBalanceMaxBlocks;
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T,
                                int E, int k, const BalancePartials& part, const BalanceOut& out,
                                cudaStream_t s) {
    const int nb = balance_blocks(T);
    cudaError_t e;
    if (nb == 1) {
        e = launch_pdl(vec_ok(E) ? k_balance_rows<true, true, kOneWarps>
                                 : k_balance_rows<false, true, kOneWarps>,
                       dim3(1), dim3(kOneWarps * 32), 0, s, logits, ids, mask, T, E, k, part, out);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    e = launch_pdl(vec_ok(E) ? k_balance_rows<true, false, kWarps>
                             : k_balance_rows<false, false, kWarps>,
                   dim3(nb), dim3(kWarps * 32), 0, s, logits, ids, mask, T, E, k, part, out);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_balance_finish, dim3((E + kColBlock - 1) / kColBlock), dim3(256), 0, s, E, k, nb,
                   part, out);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s) {
    const int64_t want = ((int64_t)a.T + kWarps - 1) / kWarps;
    const int64_t most = (int64_t)current_device_info().num_sms * 8;
    const cudaError_t e =
        launch_pdl(vec_ok(a.E) ? k_route_backward<true> : k_route_backward<false>,
                   dim3((unsigned)(want < most ? want : most)), dim3(kWarps * 32), 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
