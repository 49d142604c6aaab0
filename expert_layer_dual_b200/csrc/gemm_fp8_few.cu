// gemm_fp8_few.cu -- the FP8 block-128 product and its input gradient for few rows
// per group (single tokens, decode batches, small experts): the operands
// exchanged, the sum over blocks split over a cluster.
//
// The formulas are those of gemm_fp8_block.cu.  With few rows the weights' bytes
// bound the product, and a tile with the rows on the MMA's M side would pad them
// to 128 and promote 128 x 256 partials for nothing.  So the weights go on the M
// side (128 output columns per tile) and up to 64 rows on the N side (N = the rows
// rounded up to 16): a partial is 128 lanes x N columns, four of them in TMEM, and
// a thread holds one output column of every row.  A column of the partial is a
// row of x, so the scales come as a vector of x_scale * w_scale per block that
// the scale warp prepares in shared memory.
//
// With fewer tiles than SMs the blocks of the sum are split over a cluster of 2, 4
// or 8 CTAs; each leaves its FP32 tile in its shared memory, and every CTA adds a
// share of the rows over the cluster, in rank order (deterministic).
//
// Measured with the weights from DRAM: 1 x 6144 x 2048 6.9 us, 1 x 4096 x 6144 9.1, 64 x 4096 x
// 6144 11.3, the input gradient 64 x 6144 x 2048 9.3, and 1 x 8192 x 8192 14.7 us (67 MB, 4.6
// TB/s); with the weights in L2 the first four 5.9, 7.6 (the 128 x 256 tiles 23.5), 9.7 and
// 8.3.  At the small sizes the weights' bytes would take 2 to 4 us: the rest is the launch,
// the first load's latency and the cluster's exchange.  Grouped: 32 experts of 4096 x 6144 with
// two rows each 122 us, with 16 rows 126 (805 MB of weights, 6.6 and 6.4 TB/s).
#include <atomic>
#include <mutex>

#include "common.cuh"
#include "fp8_block.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr int FM = 128, FN = kFewRows, BK = 128;  // output columns and rows of a tile
constexpr int STAGES = 7, A_BYTES = FM * BK, B_BYTES = FN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int NPART = 4;                          // partials of FN TMEM columns
constexpr uint32_t TMEM_COLS = NPART * FN;
constexpr int EPI_WARPS = 8, MMA_WARP = 8, A_WARP = 9, B_WARP = 10, SCALE_WARP = 11;
constexpr int EPI_ROWS = FN * 4 / EPI_WARPS;      // rows (TMEM columns) of an epilogue warp
constexpr int THREADS = 32 * (SCALE_WARP + 1);
constexpr int SC_KB = 4, SC_BUFS = 4;             // scales: chunks of 4 blocks, four ahead
constexpr int RED_FLOATS = FN * FM;               // the tile left for the cluster

struct Bars {
    uint64_t full[STAGES];     // two arming arrivals (A and B) + their bytes
    uint64_t done[STAGES];     // MMA commit: the stage is free, the block's partial complete
    uint64_t pempty[NPART];    // partial read (one arrival per epilogue warp)
    uint64_t sfull[SC_BUFS];   // scale chunk written
    uint64_t sempty[SC_BUFS];  // scale chunk read (one arrival per epilogue warp)
    uint64_t rfull, rempty;    // tile left by / read by every epilogue warp of the cluster
    uint32_t tmem_slot;
    int abort_flag;
};

constexpr size_t smem_bytes(bool split) {
    return 1024 + STAGES * STAGE_BYTES + SC_BUFS * SC_KB * FN * 4 + (split ? RED_FLOATS * 4 : 0) +
           sizeof(Bars) + sizeof(TileTable) + 64;
}

struct Smem {
    uint32_t stages, scales, red, bars;
    TileTable* tt;
    __device__ __forceinline__ uint32_t full(int i) const { return bars + offsetof(Bars, full) + 8 * i; }
    __device__ __forceinline__ uint32_t done(int i) const { return bars + offsetof(Bars, done) + 8 * i; }
    __device__ __forceinline__ uint32_t pempty(int i) const { return bars + offsetof(Bars, pempty) + 8 * i; }
    __device__ __forceinline__ uint32_t sfull(int i) const { return bars + offsetof(Bars, sfull) + 8 * i; }
    __device__ __forceinline__ uint32_t sempty(int i) const { return bars + offsetof(Bars, sempty) + 8 * i; }
    __device__ __forceinline__ uint32_t rfull() const { return bars + offsetof(Bars, rfull); }
    __device__ __forceinline__ uint32_t rempty() const { return bars + offsetof(Bars, rempty); }
    __device__ __forceinline__ uint32_t abort_flag() const { return bars + offsetof(Bars, abort_flag); }
};

__device__ __forceinline__ void fail(const Smem& sm, int32_t* status) {
    report_status(status, MOE_ERR_DEVICE_TIMEOUT);
    asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(sm.abort_flag()) : "memory");
}

__device__ __forceinline__ uint32_t in_rank(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

// Every warp's writes and reads of the tiles so far, released to the CTAs of the
// cluster: one arrival per warp on each CTA's barrier.
__device__ __forceinline__ void arrive_cluster(uint32_t bar, uint32_t size) {
    __syncwarp();
    const uint32_t lane = threadIdx.x & 31;
    if (lane < size)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_rank(bar, lane))
                     : "memory");
}

// wait_phase with cluster-scope acquire (other CTAs' shared memory is read after it).
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                                  uint32_t abort_flag) {
    uint64_t t0 = 0;
    bool ok = false;
#pragma unroll 1
    for (uint32_t n = 1;; ++n) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred P;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n\t"
            "selp.b32 %0, 1, 0, P;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) {
            ok = true;
            break;
        }
        if ((n & 63u) == 0) {
            int stop;
            asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(stop) : "r"(abort_flag) : "memory");
            const uint64_t t = global_timer_ns();
            if (t0 == 0) t0 = t;
            if (stop || t - t0 > timeout_ns) break;
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// acc += columns (of this thread's TMEM lane) times their scales (floats at shared
// address cs).
template <int COLS>
__device__ __forceinline__ void promote(uint32_t taddr, uint32_t cs, uint64_t* acc) {
    float v[COLS];
    if (COLS == 32) tmem_load32(taddr, v); else tmem_load16(taddr, v);
#pragma unroll
    for (int i = 0; i < COLS / 4; ++i) {
        const float4 s = lds4(cs + 16 * i);
        acc[2 * i] = f32x2_fma(f32x2_pack(v[4 * i], v[4 * i + 1]), f32x2_pack(s.x, s.y), acc[2 * i]);
        acc[2 * i + 1] =
            f32x2_fma(f32x2_pack(v[4 * i + 2], v[4 * i + 3]), f32x2_pack(s.z, s.w), acc[2 * i + 1]);
    }
}

__device__ __forceinline__ void store_one(void* out, int64_t at, float v, int type) {
    if (type == MOE_OUT_F32)
        static_cast<float*>(out)[at] = v;
    else if (type == MOE_OUT_F16)
        static_cast<uint16_t*>(out)[at] = (uint16_t)pack_f16x2_sat(v, 0.0f);
    else
        static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
}

// The cluster's sums of one column (at shared address `here` of every CTA) for rows
// rank + (2j + odd) * SIZE, written to the output; four rows' loads in flight.
template <int SIZE>
__device__ __forceinline__ void add_rows(const Fp8ProductArgs& a, uint32_t here, int64_t at, int cols,
                                         int nrows, uint32_t rank, int odd) {
    uint32_t base[SIZE];
#pragma unroll
    for (int q = 0; q < SIZE; ++q) base[q] = in_rank(here, q);
    constexpr int U = SIZE == 8 ? 2 : 4, STEP = 2 * SIZE;
    for (int r = (int)rank + odd * SIZE; r < nrows; r += U * STEP) {
        float v[U][SIZE];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < SIZE; ++q)
                if (r + u * STEP < nrows)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(v[u][q])
                                 : "r"(base[q] + 4u * (r + u * STEP) * FM)
                                 : "memory");
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r + u * STEP >= nrows) break;
            float s = v[u][0];
#pragma unroll
            for (int q = 1; q < SIZE; ++q) s += v[u][q];
            store_one(a.out, at + (int64_t)(r + u * STEP) * cols, s, a.out_type);
        }
    }
}

template <bool INPUT>
__global__ void __launch_bounds__(THREADS, 1)
    k_product_few(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                  const __grid_constant__ Fp8ProductArgs a, uint32_t size, uint32_t b_rows) {
    extern __shared__ uint8_t smem_raw[];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x % size;  // clusters of `size` consecutive blocks
    Smem sm;
    sm.stages = (smem_u32(smem_raw) + 1023u) & ~1023u;
    sm.scales = sm.stages + STAGES * STAGE_BYTES;
    sm.red = sm.scales + SC_BUFS * SC_KB * FN * 4;
    sm.bars = sm.red + (size > 1 ? RED_FLOATS * 4 : 0);
    Bars* const b = reinterpret_cast<Bars*>(smem_raw + (sm.bars - smem_u32(smem_raw)));
    sm.tt = reinterpret_cast<TileTable*>(b + 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&b->full[s], 2);
            mbar_init(&b->done[s], 1);
        }
        for (int i = 0; i < NPART; ++i) mbar_init(&b->pempty[i], EPI_WARPS);
        for (int i = 0; i < SC_BUFS; ++i) {
            mbar_init(&b->sfull[i], 1);
            mbar_init(&b->sempty[i], EPI_WARPS);
        }
        mbar_init(&b->rfull, EPI_WARPS * size);
        mbar_init(&b->rempty, EPI_WARPS * size);
        b->abort_flag = 0;
        fence_barrier_init();
    }
    // What does not read the operands runs while the previous kernel drains.  The next
    // kernel may come once this one's TMEM is its own.
    if (warp == MMA_WARP) {
        tmem_alloc(&b->tmem_slot, TMEM_COLS);
        pdl_trigger();
    }
    if (warp == A_WARP && elect_one()) tma_prefetch_desc(&tm_w);
    if (warp == B_WARP && elect_one()) tma_prefetch_desc(&tm_x);
    if (warp == 0 && a.offsets == nullptr) build_group_table(sm.tt, nullptr, 1, a.M, FN);
    tc_fence_before_sync();
    if (size > 1)
        cluster_sync();  // every CTA's barriers exist before another arrives on them
    else
        __syncthreads();
    tc_fence_after_sync();
    pdl_wait();  // the operands come from the previous kernels
    // the status word: a wait that runs out does so seconds after this store
    if (blockIdx.x == 0 && threadIdx.x == 32) *a.status = MOE_OK;
    if (a.offsets != nullptr) {
        if (warp == 0) build_group_table(sm.tt, a.offsets, a.G, a.M, FN);
        __syncthreads();
    }
    const uint32_t tmem = b->tmem_slot;
    const int nb = a.N / 128, kbs = a.K / 128;
    const int n_tiles = INPUT ? kbs : nb;
    const int total = sm.tt->mstart[a.G] * n_tiles;
    const int first = blockIdx.x / size, step = gridDim.x / size;
    // this CTA's blocks of the sum
    const int all = INPUT ? nb : kbs, per = (all + (int)size - 1) / (int)size;
    const int kb0 = min(all, (int)rank * per), blocks = min(all, kb0 + per) - kb0;

    if (warp == A_WARP || warp == B_WARP) {
        // ---------------------------------------------------- TMA: weights, rows
        const bool is_w = warp == A_WARP;
        const CUtensorMap* map = is_w ? &tm_w : &tm_x;
        Ring<STAGES> st;
        st.round = 1u;  // a producer waits for the round before; in the self-test for one that never ends
        if (is_w && blockIdx.x + 1 == a.give_up) st.round = 0u;
        uint32_t issued = 0;
        bool ok = true;
        for (int i = first; ok && i < total; i += step) {
            const Tile t = decode_tile(sm.tt, a.G, n_tiles, i, FN);
            int x = kb0 * BK, y = t.row0;
            if (is_w) {
                y = t.g * a.N + (INPUT ? kb0 * BK : t.n * FM);
                if (INPUT) x = t.n * FM;
            }
            for (int kb = 0; kb < blocks; ++kb, st.next()) {
                if (!warp_wait_phase(sm.done(st.slot), st.round, a.timeout_ns, sm.abort_flag())) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    expect_bytes(sm.full(st.slot), is_w ? A_BYTES : b_rows * BK);
                    tma_load(sm.stages + st.slot * STAGE_BYTES + (is_w ? 0 : A_BYTES), map,
                             sm.full(st.slot), x, y);
                }
                __syncwarp();
                ++issued;
                if (INPUT && is_w) y += BK; else x += BK;
            }
        }
        if (!ok && lane == 0) fail(sm, a.status);
        // after a failure the copies in flight are waited for (bounded)
        if (lane == 0 && *reinterpret_cast<volatile int*>(&b->abort_flag))
            for (uint32_t j = issued > STAGES ? issued - STAGES : 0; j < issued; ++j)
                mbar_wait(&b->full[j % STAGES], (j / STAGES) & 1, a.timeout_ns, nullptr);
    } else if (warp == MMA_WARP) {
        // ---------------------------------------------------- MMA issuer
        Ring<STAGES> st;
        Ring<NPART> pt;
        bool ok = true;
        for (int i = first; ok && i < total; i += step) {
            const int n = (decode_tile(sm.tt, a.G, n_tiles, i, FN).nrows + 15) & ~15;
            const uint32_t idesc = idesc_e4m3(FM, n) | (INPUT ? kATransposed : 0u);
            for (int kb = 0; kb < blocks; ++kb, st.next(), pt.next()) {
                if (!warp_wait_phase(sm.pempty(pt.slot), pt.round ^ 1u, a.timeout_ns, sm.abort_flag()) ||
                    !warp_wait_phase(sm.full(st.slot), st.round, a.timeout_ns, sm.abort_flag())) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t sa = sm.stages + st.slot * STAGE_BYTES, sb = sa + A_BYTES;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)
                        umma_e4m3(tmem + pt.slot * FN,
                                  INPUT ? sdesc_mn_sw128(sa + kk * 32 * 128, A_BYTES)
                                        : sdesc_k_sw128(sa + kk * 32),
                                  sdesc_k_sw128(sb + kk * 32), idesc, kk != 0);
                    mma_commit(sm.done(st.slot));
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) fail(sm, a.status);
    } else if (warp == SCALE_WARP) {
        // ---------------------------------------------------- x_scale * w_scale per row
        const int per_row = all;
        Ring<SC_BUFS> ch;
        bool ok = true;
        for (int i = first; ok && i < total; i += step) {
            const Tile t = decode_tile(sm.tt, a.G, n_tiles, i, FN);
            const float* ws = a.b_scale + (int64_t)t.g * nb * kbs +
                              (INPUT ? (int64_t)kb0 * kbs + t.n : (int64_t)t.n * kbs + kb0);
            const float* xs = a.a_scale + (int64_t)t.row0 * per_row + kb0;
            for (int k0 = 0; k0 < blocks; k0 += SC_KB, ch.next()) {
                if (!warp_wait_phase(sm.sempty(ch.slot), ch.round ^ 1u, a.timeout_ns, sm.abort_flag())) {
                    ok = false;
                    break;
                }
                const int n = min(SC_KB, blocks - k0);
                float w[SC_KB], v[SC_KB][2];
#pragma unroll
                for (int kk = 0; kk < SC_KB; ++kk) {
                    w[kk] = kk < n ? __ldg(ws + (INPUT ? (int64_t)(k0 + kk) * kbs : k0 + kk)) : 0.0f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = lane + 32 * h;
                        v[kk][h] = kk < n && r < t.nrows ? __ldg(xs + (int64_t)r * per_row + k0 + kk) : 0.0f;
                    }
                }
                const uint32_t dst = sm.scales + 4u * (ch.slot * SC_KB * FN + lane);
#pragma unroll
                for (int kk = 0; kk < SC_KB; ++kk)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + 4u * (kk * FN + 32 * h)),
                                     "f"(v[kk][h] * w[kk])
                                     : "memory");
                __syncwarp();
                if (elect_one()) arrive(sm.sfull(ch.slot));
            }
        }
        if (!ok && lane == 0) fail(sm, a.status);
    } else {
        // ---------------------------------------------------- promotion and output
        const int quad = warp & 3, r0 = (warp >> 2) * EPI_ROWS;
        const int col = quad * 32 + lane;  // this thread's output column of the tile; its rows r0 ..
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + r0;
        const int cols = INPUT ? a.K : a.N;
        Ring<STAGES> st;
        Ring<NPART> pt;
        Ring<SC_BUFS> ch;
        uint32_t turn = 0;  // of the cluster's exchange
        bool ok = true;
        for (int i = first; ok && i < total; i += step) {
            const Tile t = decode_tile(sm.tt, a.G, n_tiles, i, FN);
            const int mine = min(EPI_ROWS, t.nrows - r0);  // rows of this warp (may be none)
            uint64_t acc[EPI_ROWS / 2];
#pragma unroll
            for (int j = 0; j < EPI_ROWS / 2; ++j) acc[j] = 0ull;
#pragma unroll 1
            for (int kb = 0; kb < blocks; ++kb, st.next(), pt.next()) {
                const int kk = kb % SC_KB;
                if ((kk == 0 &&
                     !warp_wait_phase(sm.sfull(ch.slot), ch.round, a.timeout_ns, sm.abort_flag())) ||
                    !warp_wait_phase(sm.done(st.slot), st.round, a.timeout_ns, sm.abort_flag())) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t cs = sm.scales + 4u * ((ch.slot * SC_KB + kk) * FN + r0);
                if (mine > 16)
                    promote<32>(taddr + pt.slot * FN, cs, acc);
                else if (mine > 0)
                    promote<16>(taddr + pt.slot * FN, cs, acc);
                tc_fence_before_sync();
                __syncwarp();
                if (elect_one()) arrive(sm.pempty(pt.slot));
                if (kk == SC_KB - 1 || kb == blocks - 1) {
                    if (elect_one()) arrive(sm.sempty(ch.slot));
                    ch.next();
                }
            }
            if (!ok) {
                if (lane == 0) fail(sm, a.status);
                break;
            }
            const int64_t at = (int64_t)t.row0 * cols + t.n * FM + col;
            if (size == 1) {
#pragma unroll
                for (int j = 0; j < EPI_ROWS / 2; ++j) {
                    float lo, hi;
                    f32x2_unpack(acc[j], lo, hi);
                    if (2 * j < mine) store_one(a.out, at + (int64_t)(r0 + 2 * j) * cols, lo, a.out_type);
                    if (2 * j + 1 < mine)
                        store_one(a.out, at + (int64_t)(r0 + 2 * j + 1) * cols, hi, a.out_type);
                }
            } else {
                // leave the tile for the cluster once its last readers are through
                if (!warp_wait_cluster(sm.rempty(), (turn & 1u) ^ 1u, a.timeout_ns, sm.abort_flag())) {
                    if (lane == 0) fail(sm, a.status);
                    break;
                }
                const uint32_t here = sm.red + 4u * col;
#pragma unroll
                for (int j = 0; j < EPI_ROWS / 2; ++j) {
                    float lo, hi;
                    f32x2_unpack(acc[j], lo, hi);
                    if (2 * j < mine) {
                        const uint32_t d = here + 4u * (r0 + 2 * j) * FM;
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(d), "f"(lo) : "memory");
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(d + 4u * FM), "f"(hi) : "memory");
                    }
                }
                arrive_cluster(sm.rfull(), size);
                if (!warp_wait_cluster(sm.rfull(), turn & 1u, a.timeout_ns, sm.abort_flag())) {
                    if (lane == 0) fail(sm, a.status);
                    break;
                }
                // rows rank, rank + size, ..: alternately by the two warps of a column
                switch (size) {
                    case 2: add_rows<2>(a, here, at, cols, t.nrows, rank, warp >> 2); break;
                    case 4: add_rows<4>(a, here, at, cols, t.nrows, rank, warp >> 2); break;
                    default: add_rows<8>(a, here, at, cols, t.nrows, rank, warp >> 2); break;
                }
                arrive_cluster(sm.rempty(), size);
                ++turn;
            }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, TMEM_COLS);
    }
    if (size > 1) cluster_sync();  // no CTA leaves while another may read its tile
}

// The kernel's attributes, and how many clusters of 1, 2, 4 and 8 CTAs the device holds
// at once (the GPCs' SM counts leave some idle), asked once per device.
struct DeviceSetup {
    std::mutex lock;
    std::atomic<bool> ready{false};
    int clusters[4] = {0, 0, 0, 0};
};

void launch_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, uint32_t size, unsigned clusters,
                   cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {size, 1, 1};
    *cfg = cudaLaunchConfig_t{};
    cfg->gridDim = dim3(clusters * size);
    cfg->blockDim = dim3(THREADS);
    cfg->dynamicSmemBytes = smem_bytes(size > 1);
    cfg->stream = s;
    cfg->attrs = attr;
    cfg->numAttrs = size > 1 ? 2 : 1;
}

template <bool INPUT>
cudaError_t set_up(DeviceSetup* d, int num_sms) {
    std::lock_guard<std::mutex> hold(d->lock);
    if (d->ready.load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(k_product_few<INPUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem_bytes(true));
    if (e != cudaSuccess) return e;
    d->clusters[0] = num_sms;
    for (int i = 1; i < 4; ++i) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg;
        launch_config(&cfg, attr, 1u << i, 1, nullptr);
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&d->clusters[i], k_product_few<INPUT>, &cfg)) != cudaSuccess)
            return e;
    }
    d->ready.store(true, std::memory_order_release);
    return cudaSuccess;
}

template <bool INPUT>
cudaError_t launch(const Fp8ProductArgs& a, cudaStream_t s) {
    static DeviceSetup setups[64];
    const DevInfo& dev = current_device_info();
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    DeviceSetup& d = setups[dev.device];
    if (!d.ready.load(std::memory_order_acquire)) {
        const cudaError_t e = set_up<INPUT>(&d, dev.num_sms);
        if (e != cudaSuccess) return e;
    }
    const uint32_t b_rows = a.M <= 16 ? 16 : a.M <= 32 ? 32 : FN;
    CUtensorMap tw, tx;
    const int red = INPUT ? a.N : a.K;  // the summed dimension
    if (!make_tmap_2d(&tw, a.b, 1, (uint64_t)a.G * a.N, a.K, INPUT ? BK : FM, INPUT ? FM : BK) ||
        !make_tmap_2d(&tx, a.a, 1, a.M, red, b_rows, BK))
        return cudaErrorInvalidValue;
    // the groups' rows are known on the device only: at most this many tiles
    const int64_t tiles = (a.offsets == nullptr ? (a.M + FN - 1) / FN
                                                : (int64_t)a.M / FN + (a.G < a.M ? a.G : a.M)) *
                          ((INPUT ? a.K : a.N) / FM);
    if (tiles >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    // Split the sum while every tile's cluster finds room and each CTA keeps two blocks.
    int lg = 0;
    while (lg < 3 && tiles <= d.clusters[lg + 1] && red / BK >= (4 << lg)) ++lg;
    const uint32_t size = 1u << lg;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg;
    launch_config(&cfg, attr, size, (unsigned)(tiles < d.clusters[lg] ? tiles : d.clusters[lg]), s);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_product_few<INPUT>, tw, tx, a, size, b_rows);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_fp8_few(const Fp8ProductArgs& a, cudaStream_t s) { return launch<false>(a, s); }
cudaError_t launch_gemm_fp8_dgrad_few(const Fp8ProductArgs& a, cudaStream_t s) {
    return launch<true>(a, s);
}

}  // namespace moe
