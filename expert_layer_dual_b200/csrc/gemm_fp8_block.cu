// gemm_fp8_block.cu -- the FP8 e4m3 matrix product with one FP32 scale per block
// of 128, its two gradients, and the quantiser of the weight gradient's
// operands.
//
//   y  [m][n] = sum_b xs[m][b] ws[n/128][b] sum_{k in b} xq[m][k] wq[n][k]
//   dx [m][k] = sum_b ds[m][b] ws[b][k/128] sum_{n in b} dq[m][n] wq[n][k]
//   dw [n][k] = sum_b ds[b][n] xs[b][k]     sum_{m in b} dq[m][n] xq[m][k]
// (b: blocks of 128 of the summed index).  The rows m form G groups with one
// weight matrix each (offsets), or one group of all rows.
#include "common.cuh"
#include "fp8_block.cuh"
#include "launch.h"

namespace moe {
namespace {

enum Mode { kForward, kInput, kWeight };

constexpr int TM = 64, TN = 64, KC = 32;

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// Plain form: a 64 x 64 tile per block, 4 x 4 values per thread, operands
// widened to FP32 in shared memory 32 at a time; each 128-block's sum is
// scaled and added.
template <Mode MODE>
__global__ void __launch_bounds__(256) k_product(Fp8ProductArgs a) {
    __shared__ TileTable tt;
    __shared__ float sa[KC][TM + 1], sb[KC][TN + 1];
    const int tid = threadIdx.x;
    if (tid < 32) build_group_table(&tt, a.offsets, a.G, a.M, MODE == kWeight ? 128 : TM);
    __syncthreads();
    const int tx = tid & 15, ty = tid >> 4;
    int g, row0, rows, col0 = blockIdx.y * TN, blocks, block0 = 0;
    if (MODE == kWeight) {
        g = blockIdx.z;
        row0 = blockIdx.x * TM;
        rows = min(TM, a.N - row0);
        block0 = tt.mstart[g];
        blocks = tt.mstart[g + 1] - block0;
    } else {
        if ((int)blockIdx.x >= tt.mstart[a.G]) return;
        g = group_of(&tt, a.G, blockIdx.x);
        const int at = (blockIdx.x - tt.mstart[g]) * TM;
        row0 = tt.goff[g] + at;
        rows = min(TM, tt.goff[g + 1] - row0);
        blocks = (MODE == kForward ? a.K : a.N) / 128;
    }
    const int nb = a.N / 128, kb = a.K / 128;
    const float* ws = a.b_scale + (MODE == kWeight ? 0 : (int64_t)g * nb * kb);
    float acc[4][4] = {};
    for (int b = 0; b < blocks; ++b) {
        float part[4][4] = {};
        for (int c = 0; c < 128; c += KC) {
            for (int i = tid; i < KC * TM; i += 256) {
                const int kk = i % KC, r = i / KC;
                uint8_t va = 0, vb = 0;
                if (MODE == kForward) {
                    if (r < rows) va = a.a[(int64_t)(row0 + r) * a.K + b * 128 + c + kk];
                    vb = a.b[((int64_t)g * a.N + col0 + r) * a.K + b * 128 + c + kk];
                } else if (MODE == kInput) {
                    if (r < rows) va = a.a[(int64_t)(row0 + r) * a.N + b * 128 + c + kk];
                    vb = a.b[((int64_t)g * a.N + b * 128 + c + kk) * a.K + col0 + r];
                } else {
                    const int64_t t = (int64_t)(block0 + b) * 128 + c + kk;
                    va = a.a[(int64_t)(row0 + r) * a.rows_t + t];
                    vb = a.b[(int64_t)(col0 + r) * a.rows_t + t];
                }
                sa[kk][r] = e4m3_value(va);
                sb[kk][r] = e4m3_value(vb);
            }
            __syncthreads();
            for (int kk = 0; kk < KC; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        part[i][j] = fmaf(sa[kk][ty * 4 + i], sb[kk][tx * 4 + j], part[i][j]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty * 4 + i, c = col0 + tx * 4 + j;
                float s;
                if (MODE == kForward)
                    s = (r < rows ? a.a_scale[(int64_t)(row0 + r) * kb + b] : 0.0f) * ws[(c / 128) * kb + b];
                else if (MODE == kInput)
                    s = (r < rows ? a.a_scale[(int64_t)(row0 + r) * nb + b] : 0.0f) * ws[b * kb + c / 128];
                else
                    s = a.a_scale[(int64_t)(block0 + b) * a.N + row0 + r] *
                        a.b_scale[(int64_t)(block0 + b) * a.K + c];
                acc[i][j] = fmaf(s, part[i][j], acc[i][j]);
            }
    }
    const int cols = MODE == kForward ? a.N : a.K;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = ty * 4 + i, c = col0 + tx * 4 + j;
            if (r >= rows) continue;
            if (MODE == kWeight) {
                float* p = static_cast<float*>(a.out) + ((int64_t)g * a.N + row0 + r) * a.K + c;
                *p = a.accumulate ? *p + acc[i][j] : acc[i][j];
            } else {
                store_out(a.out, (int64_t)(row0 + r) * cols + c, acc[i][j], a.out_type);
            }
        }
}

// ---------------------------------------------------------------------------
// Token-block quantisation, transposed: x [M][cols] bf16 -> q_t [cols][rows_t],
// scale_t [rows_t/128][cols].  Each group's rows start a new block of 128
// (padded with zeros), so a column's 128 tokens of one block share one scale
// and the weight gradient reads both operands along the tokens.  A block of
// threads takes 128 tokens x 64 columns: 16-byte loads, the column maxima by
// shuffles and shared memory, and the codes turned in shared memory so that
// each column's 128 codes leave as one 128-byte run.  Bound by HBM: 2 bytes
// read and 1 written per value.
// ---------------------------------------------------------------------------
constexpr int QC = 64;

__global__ void __launch_bounds__(256)
    k_quant_tokens(const uint16_t* __restrict__ x, const int32_t* __restrict__ offsets, int G, int M,
                   int cols, int64_t rows_t, uint8_t* __restrict__ q, float* __restrict__ scale) {
    __shared__ TileTable tt;
    __shared__ float red[8][QC];
    __shared__ uint32_t codes[QC][33];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    if (warp == 0) build_group_table(&tt, offsets, G, M, 128);
    __syncthreads();
    const int blk = blockIdx.y;
    if (blk >= tt.mstart[G]) return;
    const int g = group_of(&tt, G, blk);
    const int64_t row0 = tt.goff[g] + (int64_t)(blk - tt.mstart[g]) * 128;
    const int rows = min((int64_t)128, tt.goff[g + 1] - row0);
    const int c0 = blockIdx.x * QC, c8 = (tid & 7) * 8, r4 = (tid >> 3) * 4;
    float f[4][8], m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (r4 + i < rows)
            u = __ldg(reinterpret_cast<const uint4*>(x + (row0 + r4 + i) * cols + c0 + c8));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[i][2 * j] = __uint_as_float(w[j] << 16);
            f[i][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], fabsf(f[i][j]));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 8));
        m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        if (lane < 8) red[warp][c8 + j] = m[j];
    }
    __syncthreads();
    if (tid < QC) {
        float a = red[0][tid];
#pragma unroll
        for (int w = 1; w < 8; ++w) a = fmaxf(a, red[w][tid]);
        const float s = a == 0.0f ? 1.0f : __fdiv_rn(a, 448.0f);
        scale[(int64_t)blk * cols + c0 + tid] = s;
        red[0][tid] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float s = red[0][c8 + j];
        const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(f[0][j], s), __fdiv_rn(f[1][j], s)), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(f[2][j], s), __fdiv_rn(f[3][j], s)), __NV_SATFINITE, __NV_E4M3);
        codes[c8 + j][tid >> 3] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    __syncthreads();
#pragma unroll
    for (int i = tid; i < QC * 8; i += 256) {
        const int c = i >> 3, p = (i & 7) * 4;
        st_global_v4(q + (int64_t)(c0 + c) * rows_t + (int64_t)blk * 128 + p * 4, codes[c][p],
                     codes[c][p + 1], codes[c][p + 2], codes[c][p + 3]);
    }
}

}  // namespace

cudaError_t launch_quant_tokens(const uint16_t* x, const int32_t* offsets, int G, int M, int cols,
                                uint8_t* q, float* scale, cudaStream_t s) {
    const int64_t rows_t = fp8_token_rows(M, offsets == nullptr ? 1 : G);
    const cudaError_t e =
        launch_pdl(k_quant_tokens, dim3(cols / QC, (unsigned)(rows_t / 128)), dim3(256), 0, s, x,
                   offsets, G, M, cols, rows_t, q, scale);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_gemm_fp8(const Fp8ProductArgs& a, cudaStream_t s) {
    k_product<kForward><<<dim3((a.M + TM - 1) / TM + a.G, a.N / TN), 256, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_gemm_fp8_dgrad(const Fp8ProductArgs& a, cudaStream_t s) {
    k_product<kInput><<<dim3((a.M + TM - 1) / TM + a.G, a.K / TN), 256, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_gemm_fp8_wgrad(const Fp8ProductArgs& a, cudaStream_t s) {
    k_product<kWeight><<<dim3(a.N / TM, a.K / TN, a.G), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
