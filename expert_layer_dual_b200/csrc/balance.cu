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
// Sixteen lanes hold a row, up to 16 values each in registers, so a warp works on
// two neighbouring rows: the row sums and maxima take four exchanges for two rows,
// and a lane's values leave room for four blocks an SM, whose loads cover the
// latency of memory.  Every logit is read once and every gradient written once, so
// the bytes are the floor: 20 and 41 us for 131072 rows of 256 experts.  Measured
// there: 27.6 us for the loss and 47.0 us for the gradient (4.9 and 5.7 TB/s;
// 49.5 us with the top-k part).
// Other splits of a row took longer: a warp per row, with the accurate expf and
// the top-k part by comparing every column with every id, 41 and 82 us, bound by
// its instructions (210 and 496 a row); eight lanes with 32 values each 54 and 52
// us, bound by the few warps its registers leave.  Few tokens are bound by the
// launches: 3.6 and 3.2 us for 64.
//
// Sums are FP32 within a row, over at most 64 rows of a lane and over a block's warps, FP64
// over the blocks; what more rows of a lane would round away is kept beside their sums, so
// the error does not grow with T.  No atomic on a float, so the results do not depend on
// scheduling.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr int kLanes = 16;               // lanes of a row
constexpr int kRows = 32 / kLanes;       // rows of a warp
constexpr int kGroup = 4 * kLanes;       // columns of a row read at once
constexpr int kWarps = 8;                // warps per block
constexpr int kOneWarps = 32;            // warps of the one-block kernel
constexpr int kRowWarps = 16;            // warps of the two-pass form's blocks
constexpr int kTurns = 64;               // rows that a lane adds up in FP32
constexpr int kFinishBlocks = 8;         // of k_balance_finish: 32 experts each

// The loss's first pass: one block that finishes the result, two passes, or two passes over
// so many tokens that a lane has more than kTurns rows (from 606209 tokens on).  The third
// form against the second: 620000 tokens of 256 experts 104.4 and 102.2 us, of 8 experts 74.6
// and 74.7, 2000000 of 64 226 and 227; with its additions in the second's place as well,
// 131072 tokens of 256 took 29.0 us, so 27.6.
enum Rows { kOneBlock, kTwoPasses, kManyRows };

// NV: groups of 64 columns (E <= 64 NV); value 4i + c of lane l is column 64i + 4l + c.
// VEC: E % 4 == 0, so the rows start on 16 bytes.
template <int NV, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int l, float* v) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * kGroup + l * 4;
        if (VEC) {
            float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (c < E) f = *reinterpret_cast<const float4*>(row + c);
            v[4 * i] = f.x;
            v[4 * i + 1] = f.y;
            v[4 * i + 2] = f.z;
            v[4 * i + 3] = f.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = c + j < E ? row[c + j] : -INFINITY;
        }
    }
}

template <int NV, bool VEC>
__device__ __forceinline__ void store_row(float* row, int E, int l, const float* v) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * kGroup + l * 4;
        if (VEC) {
            if (c < E)
                *reinterpret_cast<float4*>(row + c) =
                    make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < E) row[c + j] = v[4 * i + j];
        }
    }
}

// Over the lanes of a row.
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// v <- exp(v - max) of the row; returns 1 / sum.  The exponential is the hardware's
// exp2 of the difference times log2(e): the argument rounds by |l - max| 2^-23, the
// exponential by 2^-22, as much as the sums around it.  A row without any finite
// logit (every entry -inf) becomes zeros: it selects nothing.
template <int N>
__device__ __forceinline__ float exp_row(float* v) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
    m = row_max(m);
    if (m == -INFINITY) m = 0.0f;
    constexpr float log2e = 1.4426950408889634f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((v[i] - m) * log2e));
        v[i] = e;
        s += e;
    }
    s = row_sum(s);
    return s > 0.0f ? 1.0f / s : (s == 0.0f ? 0.0f : s);  // NaN stays NaN
}

// Adds a warp's sums, of its two rows together, to those in shared memory: hi, and lo of
// what rounds away (first: there are none yet, lo unused where nothing follows); a lane
// always has the same columns.
template <int N>
__device__ __forceinline__ void add_sums(float* hi, float* lo, float* acc, int l, int r, bool first) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        for (int o = kLanes; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    }
    if (r == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            float* const h = hi + i * kGroup + l * 4;
            if (first) {
                *reinterpret_cast<float4*>(h) = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
                continue;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = h[j], b = acc[4 * i + j], s = a + b, d = s - a;
                lo[i * kGroup + l * 4 + j] += (a - (s - d)) + (b - d);
                h[j] = s;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
}

// ---------------------------------------------------------------------------
// Loss, first pass: a warp takes two tokens at a time and keeps the sums of its
// tokens' probabilities in registers (a lane always holds the same columns);
// the assignments are counted in shared memory (integers).  The block's sums go
// to its row of the partials.  ONE: a single block, which finishes the result
// itself (few tokens: one launch).  MANY: after kTurns rows of a lane the warp's sums are
// added to those in shared memory, each with its rounding error (Knuth's two-sum).
// ---------------------------------------------------------------------------
template <int NV, bool VEC, Rows FORM, int WARPS>
__global__ void __launch_bounds__(WARPS * 32)
    k_balance_rows(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                   const uint8_t* __restrict__ mask, int T, int E, int k, BalancePartials part,
                   BalanceOut out) {
    constexpr int N = 4 * NV;
    constexpr bool ONE = FORM == kOneBlock, MANY = FORM == kManyRows;
    __shared__ __align__(16) float s_psum[WARPS][kGroup * NV];
    __shared__ __align__(16) float s_low[MANY ? WARPS : 1][MANY ? kGroup * NV : 1];  // rounded away of s_psum
    __shared__ int s_cnt[256], s_tokens, s_bad;
    __shared__ double s_term[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int l = lane % kLanes, r = lane / kLanes;
    for (int e = tid; e < 256; e += WARPS * 32) s_cnt[e] = 0;
    if constexpr (MANY)
        for (int i = lane; i < kGroup * NV; i += 32) s_low[warp][i] = 0.0f;
    if (tid == 0) s_tokens = s_bad = 0;
    __syncthreads();
    pdl_trigger();
    pdl_wait();  // the logits and ids come from the previous kernels

    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    int tokens = 0, bad = 0;
    bool first = true;
    const int64_t step = (int64_t)gridDim.x * WARPS * kRows;
    int64_t t0 = ((int64_t)blockIdx.x * WARPS + warp) * kRows;
    do {
        const int64_t stop = MANY ? min((int64_t)T, t0 + kTurns * step) : T;
        for (; t0 < stop; t0 += step) {
            const int64_t t = t0 + r;
            const bool on = t < T && (mask == nullptr || mask[t] != 0);
            float v[N];
            if (on) {
                load_row<NV, VEC>(logits + t * E, E, l, v);
                if (l < k) {
                    const int id = ids[t * k + l];
                    if (id >= 0 && id < E) atomicAdd(&s_cnt[id], 1);
                    else bad = 1;
                }
                tokens += l == 0;
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = -INFINITY;
            }
            const float inv = exp_row<N>(v);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
        }
        // the warp's two rows, then the block's warps
        add_sums<N>(s_psum[warp], s_low[MANY ? warp : 0], acc, l, r, first);
        first = false;
    } while (MANY && t0 < T);
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if (bad) s_bad = 1;
    if (lane == 0 && tokens) atomicAdd(&s_tokens, tokens);
    __syncthreads();

    if (!ONE) {
        for (int e = tid; e < E; e += WARPS * 32) {
            std::conditional_t<MANY, double, float> s = 0;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                s += s_psum[w][e];
                if constexpr (MANY) s += s_low[w][e];
            }
            part.psum[(int64_t)blockIdx.x * E + e] = (float)s;
            part.cnt[(int64_t)blockIdx.x * E + e] = s_cnt[e];
        }
        if (tid == 0) {
            part.info[2 * blockIdx.x] = s_tokens;
            part.info[2 * blockIdx.x + 1] = s_bad;
        }
        return;
    }
    const int n = s_tokens;
    double term = 0.0;
    const double inv = n > 0 ? 1.0 / ((double)k * n) : 0.0;
    if (tid < 256) {
        if (tid < E) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s += s_psum[w][tid];
            const double mean = s * inv * k;
            out.prob_mean[tid] = (float)mean;
            out.counts[tid] = s_cnt[tid];
            term = (double)s_cnt[tid] * E * inv * mean;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
        if (lane == 0) s_term[warp] = term;
    }
    __syncthreads();
    if (tid == 0) {
        double s = 0.0;
        for (int w = 0; w < 8; ++w) s += s_term[w];
        *out.loss = (float)(out.coef * s);
        *out.tokens = n;
        *out.status = s_bad ? MOE_ERR_DEVICE_BAD_INDEX : MOE_OK;
    }
}

// Loss, second pass: a cluster of eight blocks, 32 experts each.  Warp w takes the
// partials of the first pass's blocks w, w + 32, .. (a row of 32 experts per load,
// all of them in flight together); the sums over the warps are in FP64 and in a fixed
// order, as is the sum of the eight blocks' shares of the loss in the first block's
// shared memory.  (With 64 blocks of four experts, the last of which added the shares
// through global memory, the loss took 11.0 us for 16384 tokens, so 8.3.)
__global__ void __cluster_dims__(kFinishBlocks, 1, 1) __launch_bounds__(1024)
    k_balance_finish(int E, int k, int nblocks, BalancePartials part, BalanceOut out) {
    constexpr int PER = (kBalanceMaxBlocks + 31) / 32;
    __shared__ double s_sum[32][33];
    __shared__ int s_cnt[32][33];
    __shared__ int s_tokens[32], s_bad[32];
    __shared__ double s_term[32], s_share[kFinishBlocks];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // A block's shared memory may be reached once it is known to run: every block arrives
    // here and waits before the exchange, when all of them long have.
    cluster_arrive();
    pdl_trigger();
    pdl_wait();
    const int e = blockIdx.x * 32 + lane;
    float p[PER];
    int c[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = warp + i * 32;
        const bool in = e < E && b < nblocks;
        p[i] = in ? part.psum[(int64_t)b * E + e] : 0.0f;
        c[i] = in ? part.cnt[(int64_t)b * E + e] : 0;
    }
    static_assert(kBalanceMaxBlocks <= 1024, "a thread per block of the first pass");
    int tokens = 0, bad = 0;
    if (tid < nblocks) {
        tokens = part.info[2 * tid];
        bad = part.info[2 * tid + 1];
    }
    double sum = 0.0;
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        sum += p[i];
        cnt += c[i];
    }
    s_sum[warp][lane] = sum;
    s_cnt[warp][lane] = cnt;
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (lane == 0) {
        s_tokens[warp] = tokens;
        s_bad[warp] = bad;
    }
    __syncthreads();
    // warp w: expert 32 blockIdx.x + w
    const int n = __reduce_add_sync(0xffffffffu, s_tokens[lane]);
    const int any = __reduce_or_sync(0xffffffffu, s_bad[lane]);
    double s = s_sum[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int m = __reduce_add_sync(0xffffffffu, s_cnt[lane][warp]);
    if (lane == 0) {
        const int mine = blockIdx.x * 32 + warp;
        const double inv = n > 0 ? 1.0 / ((double)k * n) : 0.0, mean = s * inv * k;
        if (mine < E) {
            out.prob_mean[mine] = (float)mean;
            out.counts[mine] = m;
        }
        s_term[warp] = mine < E ? (double)m * E * inv * mean : 0.0;
    }
    __syncthreads();
    cluster_wait();
    if (warp == 0) {
        double term = s_term[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
        if (lane == 0)
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(smem_in_rank(&s_share[blockIdx.x], 0)), "d"(term)
                         : "memory");
    }
    __syncwarp();
    cluster_sync();
    if (blockIdx.x == 0 && tid == 0) {
        double total = 0.0;
#pragma unroll
        for (int b = 0; b < kFinishBlocks; ++b) total += s_share[b];
        *out.loss = (float)(out.coef * total);
        *out.tokens = n;
        *out.status = any ? MOE_ERR_DEVICE_BAD_INDEX : MOE_OK;
    }
}

// ---------------------------------------------------------------------------
// Gradient of the logits: two rows per warp as above, the softmax recomputed
// from the logits (nothing more is read).  The k values of the top-k part go to
// their columns through a row of shared memory that is zero in between; ids that
// repeat within a row are added up first, so their order does not matter.
// Masked tokens get zeros and their logits are not read.
// ---------------------------------------------------------------------------
constexpr int backward_blocks(int nv) { return nv >= 3 ? 4 : nv == 2 ? 5 : 6; }  // per SM, by registers

template <int NV, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, backward_blocks(NV))
    k_route_backward(const __grid_constant__ RouteBackwardArgs a) {
    constexpr int N = 4 * NV;
    __shared__ __align__(16) float s_row[kWarps][kRows][kGroup * NV], s_f1[kGroup * NV];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int l = lane % kLanes, r = lane / kLanes;
    float* const srow = s_row[warp][r];
    for (int c = l; c < kGroup * NV; c += kLanes) srow[c] = 0.0f;
    __syncwarp();
    pdl_trigger();
    pdl_wait();
    const int E = a.E, k = a.k;
    const bool balance = a.dloss != nullptr, need_p = balance || !a.renorm;
    float f1[N], cb = 0.0f;  // f_e - 1 of this lane's columns; dloss coef / n
#pragma unroll
    for (int i = 0; i < N; ++i) f1[i] = 0.0f;
    if (balance) {
        const int n = *a.tokens;
        cb = n > 0 ? *a.dloss * a.coef / (float)n : 0.0f;
        // a quotient per thread, then each lane's columns (in FP64 and sixteen a thread, 4096
        // tokens took 5.4 us, so 4.6); of two rounded integers, so within 1.5 * 2^-23
        if (tid < kGroup * NV) {
            const int64_t kn = (int64_t)k * n;
            s_f1[tid] = tid < E && n > 0 ? (float)((int64_t)a.counts[tid] * E - kn) / (float)kn : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(s_f1 + i * kGroup + l * 4);
            f1[4 * i] = f.x;
            f1[4 * i + 1] = f.y;
            f1[4 * i + 2] = f.z;
            f1[4 * i + 3] = f.w;
        }
    }
    const int64_t step = (int64_t)gridDim.x * kWarps * kRows;
    for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kRows; t0 < a.T; t0 += step) {
        const int64_t t = t0 + r;
        const bool in = t < a.T, on = in && (a.mask == nullptr || a.mask[t] != 0);
        float p[N];
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = -INFINITY;
        if (need_p && on) load_row<NV, VEC>(a.logits + t * E, E, l, p);
        int id = -1;
        float w = 0.0f, d = 0.0f;
        if (a.dw != nullptr && on && l < k) {
            id = a.ids[t * k + l];
            w = a.w[t * k + l];
            d = a.dw[t * k + l];
        }
        float inv = 0.0f, dot = 0.0f;
        if (need_p) inv = exp_row<N>(p);
        if (a.dw != nullptr) {
            dot = row_sum(w * d);
            const float mine = a.renorm ? w * (d - dot) : d;
            float sum = 0.0f;  // of the row's lanes with this id; the first of them writes
            bool first = true;
            for (int j = 0; j < k; ++j) {
                const int idj = __shfl_sync(0xffffffffu, id, j, kLanes);
                const float vj = __shfl_sync(0xffffffffu, mine, j, kLanes);
                if (idj == id) {
                    sum += vj;
                    first = first && j >= l;
                }
            }
            if (first && id >= 0 && id < E) srow[id] = sum;
            __syncwarp();
        }
        float s = 0.0f;
        if (balance) {
#pragma unroll
            for (int i = 0; i < N; ++i) s = fmaf(f1[i], p[i], s);
            s = row_sum(s) * inv;
        }
        const float ci = cb * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float g[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (a.dw != nullptr) {
                const float4 q = *reinterpret_cast<const float4*>(srow + i * kGroup + l * 4);
                g[0] = q.x;
                g[1] = q.y;
                g[2] = q.z;
                g[3] = q.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = p[4 * i + j];
                if (!a.renorm) g[j] = e * inv * (g[j] - dot);
                if (balance) g[j] = fmaf(ci * e, f1[4 * i + j] - s, g[j]);
                p[4 * i + j] = on ? g[j] : 0.0f;
            }
        }
        if (in) store_row<NV, VEC>(a.dlogits + t * E, E, l, p);
        if (a.dw != nullptr) {
            __syncwarp();
            if (id >= 0 && id < E) srow[id] = 0.0f;
            __syncwarp();
        }
    }
}

// The instance for E experts: 1 to 4 groups of 64 columns.
template <typename F>
cudaError_t by_width(int E, F f) {
    const bool vec = E % 4 == 0;
    if (E <= kGroup) return vec ? f.template operator()<1, true>() : f.template operator()<1, false>();
    if (E <= 2 * kGroup) return vec ? f.template operator()<2, true>() : f.template operator()<2, false>();
    if (E <= 3 * kGroup) return vec ? f.template operator()<3, true>() : f.template operator()<3, false>();
    return vec ? f.template operator()<4, true>() : f.template operator()<4, false>();
}

struct LaunchRows {
    const float* logits;
    const int32_t* ids;
    const uint8_t* mask;
    int T, E, k, blocks;
    BalancePartials part;
    BalanceOut out;
    cudaStream_t s;
    template <int NV, bool VEC>
    cudaError_t operator()() const {
        if (blocks == 1)
            return launch_pdl(k_balance_rows<NV, VEC, kOneBlock, kOneWarps>, dim3(1), dim3(kOneWarps * 32), 0, s,
                              logits, ids, mask, T, E, k, part, out);
        const bool many = T > (int64_t)kTurns * blocks * kRowWarps * kRows;
        return launch_pdl(many ? k_balance_rows<NV, VEC, kManyRows, kRowWarps> : k_balance_rows<NV, VEC, kTwoPasses, kRowWarps>,
                          dim3(blocks), dim3(kRowWarps * 32), 0, s, logits, ids, mask, T, E, k, part, out);
    }
};

struct LaunchBackward {
    RouteBackwardArgs a;
    cudaStream_t s;
    template <int NV, bool VEC>
    cudaError_t operator()() const {
        const int64_t want = ((int64_t)a.T + kWarps * kRows - 1) / (kWarps * kRows);
        // as many blocks as are resident together, with turns of one length: 16384 tokens
        // of 256 experts 9.0 us, 131072 49.5 us; with six per SM some 0.8 and 6 us more
        const int64_t most = (int64_t)current_device_info().num_sms * backward_blocks(NV);
        const int64_t turns = (want + most - 1) / most;
        return launch_pdl(k_route_backward<NV, VEC>, dim3((unsigned)((want + turns - 1) / turns)),
                          dim3(kWarps * 32), 0, s, a);
    }
};

}  // namespace

int balance_blocks(int T) {
    if (T <= kBalanceOneBlock) return 1;
    // 16 warps a block, two blocks an SM: with blocks of 8 (a block per 64 tokens, at most
    // four an SM) 16384 tokens took 13.0 us and 2048 7.4, of 32 10.1 and 6.8, so 11.0
    // and 6.3, the second pass at that time included
    const int64_t want = ((int64_t)T + kRowWarps * kRows - 1) / (kRowWarps * kRows);
    return want < kBalanceMaxBlocks ? (int)want : kBalanceMaxBlocks;
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T,
                                int E, int k, const BalancePartials& part, const BalanceOut& out,
                                cudaStream_t s) {
    const int nb = balance_blocks(T);
    cudaError_t e = by_width(E, LaunchRows{logits, ids, mask, T, E, k, nb, part, out, s});
    if (e != cudaSuccess || nb == 1) return e != cudaSuccess ? e : cudaGetLastError();
    e = launch_pdl(k_balance_finish, dim3(kFinishBlocks), dim3(1024), 0, s, E, k, nb, part, out);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s) {
    const cudaError_t e = by_width(a.E, LaunchBackward{a, s});
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
