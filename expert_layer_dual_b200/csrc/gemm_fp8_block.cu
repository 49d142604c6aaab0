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

constexpr int BM = 128, PM = 256, BK = 128;    // rows of a CTA, of a pair; one scale block of the sum
constexpr int H = 2, BN = 128 * H;             // output columns of a pair's tile
constexpr int STAGES = 6, A_BYTES = BM * BK, B_BYTES = BN / 2 * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int NPART = 4;                       // partial buffers of 128 TMEM columns
constexpr uint32_t TMEM_COLS = 512;
constexpr int EPI_WARPS = 16, MMA_WARP = 16, A_WARP = 17, B_WARP = 18, SCALE_WARP = 19;
constexpr int THREADS = 32 * (SCALE_WARP + 1);  // 640
// Registers: 640 threads x 96 at launch; the four helper warps fall to 32 and the
// sixteen epilogue warps (64 accumulators each) rise to 112: 512 * 112 + 128 * 32
// = 640 * 96 (checked against the compiled kernel before its first launch).
constexpr int REGS = 96, REGS_EPI = 104, REGS_HELP = 64;
constexpr int SC_KB = 4, SC_BUFS = 4;           // scales: chunks of 4 blocks, four chunks ahead
constexpr uint16_t kPairMask = 0x3;

template <Mode MODE>
struct ScaleLayout {  // floats per block: the CTA's row scales, then the column side's
    static constexpr int PER_KB = BM + (MODE == kWeight ? BN : 4);
    static constexpr int FLOATS = SC_BUFS * SC_KB * PER_KB;
};

struct Bars {
    uint64_t full[STAGES];      // leader: two arming arrivals (A and B) + both CTAs' bytes
    uint64_t empty[STAGES];     // each CTA: the leader's multicast MMA commit
    uint64_t pfull[NPART];      // each CTA: the leader's multicast MMA commit
    uint64_t pempty[NPART];     // leader: the warps of both CTAs that read the partial
    uint64_t sfull[SC_BUFS];    // scale chunk landed (32 asynchronous arrivals)
    uint64_t sempty[SC_BUFS];   // scale chunk read (one arrival per epilogue warp)
    uint32_t tmem_slot;
    int abort_flag;
};

template <Mode MODE>
constexpr size_t smem_bytes() {
    return 1024 + STAGES * STAGE_BYTES + ScaleLayout<MODE>::FLOATS * 4 + sizeof(Bars) +
           sizeof(TileTable) + 64;
}

struct Smem {
    uint8_t* stages;
    float* scales;
    Bars* bars;
    TileTable* tt;
};

template <Mode MODE>
__device__ __forceinline__ Smem carve(uint8_t* raw) {
    Smem s;
    s.stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                          ~static_cast<uintptr_t>(1023));
    s.scales = reinterpret_cast<float*>(s.stages + STAGES * STAGE_BYTES);
    s.bars = reinterpret_cast<Bars*>(s.scales + ScaleLayout<MODE>::FLOATS);
    s.tt = reinterpret_cast<TileTable*>(s.bars + 1);
    return s;
}

// ---------------------------------------------------------------- bounded waits
// A phase that is about to complete is met by the first tries, without a read of
// the global timer; the time limit is kept by the slow loop.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                           const volatile int* abort) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
        if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    return CLUSTER ? mbar_wait_cluster(bar, parity, timeout_ns, abort)
                   : mbar_wait(bar, parity, timeout_ns, abort);
}

__device__ __forceinline__ bool warp_wait_phase(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                                const volatile int* abort) {
    return __all_sync(0xffffffffu, wait_phase<false>(bar, parity, timeout_ns, abort));
}

__device__ __forceinline__ void fail(Bars* b, int32_t* status) {
    report_status(status, MOE_ERR_DEVICE_TIMEOUT);
    *reinterpret_cast<volatile int*>(&b->abort_flag) = 1;
}

// One lane arrives on the leader's barrier.  Relaxed: what the barrier orders is
// the reuse of TMEM columns, whose loads this warp has waited for; no memory
// write travels with it, and a release at cluster scope would wait for the
// warp's stores to global memory.
__device__ __forceinline__ void warp_arrive_leader(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         smem_in_rank(bar, 0))
                     : "memory");
}

// ---------------------------------------------------------------- operands
// MMA of a CTA pair, e4m3.
__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor bit 16: B is stored with its N index innermost.
constexpr uint32_t kBTransposed = 1u << 16;

__device__ __forceinline__ uint64_t f32x2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f32x2_unpack(uint64_t r, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// ---------------------------------------------------------------- tiles
// One tile of a pair: rows row0 .. of the output (this CTA's 128 of 256), columns
// col0 .., group g, and the scale blocks [block0, block0 + blocks) that it sums
// over (kWeight: token blocks of the group; else all of them, from 0).
struct PTile {
    int g, row0, nrows, col0, block0, blocks;
};

template <Mode MODE>
struct Work {
    int total, n_tiles, k_tiles, blocks;
    __device__ __forceinline__ Work(const Fp8ProductArgs& a, const TileTable* tt) {
        if (MODE == kWeight) {
            n_tiles = (a.K + BN - 1) / BN;
            k_tiles = (a.N + PM - 1) / PM;
            total = a.G * n_tiles * k_tiles;
        } else {
            n_tiles = ((MODE == kForward ? a.N : a.K) + BN - 1) / BN;
            blocks = (MODE == kForward ? a.K : a.N) / BK;
            total = tt->mstart[a.G] * n_tiles;
        }
    }
    __device__ __forceinline__ PTile tile(const Fp8ProductArgs& a, const TileTable* tt, int i,
                                          uint32_t rank) const {
        PTile p;
        if (MODE == kWeight) {
            const int per = n_tiles * k_tiles;
            p.g = i / per;
            const int r = i - p.g * per;
            p.row0 = (r / n_tiles) * PM + (int)rank * BM;
            p.nrows = min(BM, max(0, a.N - p.row0));
            p.col0 = (r % n_tiles) * BN;
            p.block0 = tt->mstart[p.g];
            p.blocks = tt->mstart[p.g + 1] - p.block0;
        } else {
            const Tile t = decode_tile(tt, a.G, n_tiles, i, PM);
            p.g = t.g;
            p.row0 = t.row0 + (int)rank * BM;
            p.nrows = min(BM, max(0, t.nrows - (int)rank * BM));
            p.col0 = t.n * BN;
            p.block0 = 0;
            p.blocks = blocks;
        }
        return p;
    }
};

// ---------------------------------------------------------------- epilogue
// acc += f * (32 TMEM columns), in pairs; with column scales: acc += f * (cs * P).
template <bool COLSCALE>
__device__ __forceinline__ void promote32(uint32_t taddr, uint64_t ff, const float* cs, uint64_t* acc) {
    float v[32];
    tmem_load32(taddr, v);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        uint64_t p0 = f32x2_pack(v[2 * i], v[2 * i + 1]), p1 = f32x2_pack(v[2 * i + 2], v[2 * i + 3]);
        if (COLSCALE) {
            const float4 s = *reinterpret_cast<const float4*>(cs + 2 * i);
            p0 = f32x2_mul(p0, f32x2_pack(s.x, s.y));
            p1 = f32x2_mul(p1, f32x2_pack(s.z, s.w));
        }
        acc[i] = f32x2_fma(ff, p0, acc[i]);
        acc[i + 1] = f32x2_fma(ff, p1, acc[i + 1]);
    }
}

// Writes 32 consecutive values of one row (16-byte aligned).
template <Mode MODE>
__device__ __forceinline__ void store32(const Fp8ProductArgs& a, int64_t at, const uint64_t* acc) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) f32x2_unpack(acc[i], v[2 * i], v[2 * i + 1]);
    if (MODE == kWeight || a.out_type == MOE_OUT_F32) {
        float* dst = static_cast<float*>(a.out) + at;
        if (MODE == kWeight && a.accumulate) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 o = *reinterpret_cast<const float4*>(dst + 4 * q);
                v[4 * q] += o.x;
                v[4 * q + 1] += o.y;
                v[4 * q + 2] += o.z;
                v[4 * q + 3] += o.w;
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(dst + 4 * q) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    } else if (a.out_type == MOE_OUT_F16) {
        st_f16x32(static_cast<__half*>(a.out) + at, v);
    } else {
        uint16_t* dst = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            st_global_v4(dst + 8 * q, pack_bf16x2(v[8 * q], v[8 * q + 1]),
                         pack_bf16x2(v[8 * q + 2], v[8 * q + 3]), pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                         pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
    }
}

// ---------------------------------------------------------------------------
// The product on CTA pairs.  Per scale block of the summed index the pair
// leader issues, for each half of the tile's 256 columns, four M = 256, N = 128,
// K = 32 MMAs into a fresh 128-column partial (one of four in TMEM); the epilogue
// warps take each partial out of TMEM and add it, scaled, to FP32 accumulators in
// registers.  Half h holds columns 64h .. 64h+63 of the tile's two scale blocks
// (CTA 0 loads the operand of the first block's columns, CTA 1 of the second's),
// so a warp's 64 columns have one weight scale.
// ---------------------------------------------------------------------------
template <Mode MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    k_product_pair(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   Fp8ProductArgs a) {
    extern __shared__ uint8_t smem_raw[];
    Smem sm = carve<MODE>(smem_raw);
    Bars* b = sm.bars;
    const volatile int* ab = &b->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    using SL = ScaleLayout<MODE>;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&b->full[s], 2);
            mbar_init(&b->empty[s], 1);
        }
        for (int i = 0; i < NPART; ++i) {
            mbar_init(&b->pfull[i], 1);
            mbar_init(&b->pempty[i], 2 * EPI_WARPS / H);
        }
        for (int i = 0; i < SC_BUFS; ++i) {
            mbar_init(&b->sfull[i], 32);
            mbar_init(&b->sempty[i], EPI_WARPS);
        }
        b->abort_flag = 0;
        fence_barrier_init();
    }
    pdl_wait();  // the operands come from the previous kernels
    if (warp == 0) build_group_table(sm.tt, a.offsets, a.G, a.M, MODE == kWeight ? BK : PM);
    // the status word: a wait that runs out does so seconds after this store
    if (blockIdx.x == 0 && threadIdx.x == 32) *a.status = MOE_OK;
    __syncthreads();
    pdl_trigger();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    if (warp == MMA_WARP) tmem_alloc_pair(&b->tmem_slot, TMEM_COLS);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = b->tmem_slot;
    const Work<MODE> work(a, sm.tt);
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (warp >= EPI_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_HELP));
        if (warp == A_WARP || warp == B_WARP) {
            // ------------------------------------------------ TMA: one operand each
            if (lane == 0) {
                const bool is_a = warp == A_WARP;
                const CUtensorMap* map = is_a ? &tm_a : &tm_b;
                tma_prefetch_desc(map);
                const uint32_t full_leader = smem_in_rank(&b->full[0], 0);
                const uint32_t bytes = 2 * (is_a ? A_BYTES : B_BYTES);  // both CTAs'
                uint8_t* dst0 = sm.stages + (is_a ? 0 : A_BYTES);
                uint32_t it = 0;
                bool ok = true;
                for (int i = pair; ok && i < work.total; i += npairs) {
                    const PTile t = work.tile(a, sm.tt, i, rank);
                    const int col = t.col0 + (int)rank * (BN / 2);
                    for (int kb = 0; kb < t.blocks; ++kb, ++it) {
                        const int s = it % STAGES;
                        if (!wait_phase<false>(&b->empty[s], ((it / STAGES) & 1) ^ 1, a.timeout_ns, ab)) {
                            fail(b, a.status);
                            ok = false;
                            break;
                        }
                        if (rank == 0) mbar_arrive_expect_tx(&b->full[s], bytes);
                        int x, y;
                        if (is_a) {
                            x = (t.block0 + kb) * BK;
                            y = t.row0;
                        } else if (MODE == kForward) {
                            x = kb * BK;
                            y = t.g * a.N + col;
                        } else if (MODE == kInput) {
                            x = col;
                            y = t.g * a.N + kb * BK;
                        } else {
                            x = (t.block0 + kb) * BK;
                            y = col;
                        }
                        tma_load_2d_pair(dst0 + s * STAGE_BYTES, map,
                                         full_leader + s * (uint32_t)sizeof(uint64_t), x, y);
                    }
                }
                // after a failure the pair's copies in flight are waited for (bounded)
                if (*ab && rank == 0)
                    for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j)
                        mbar_wait(&b->full[j % STAGES], (j / STAGES) & 1, a.timeout_ns, nullptr);
            }
        } else if (warp == MMA_WARP) {
            // ------------------------------------------------ MMA issuer (leader)
            if (lane == 0 && rank == 0) {
                constexpr uint32_t idesc = idesc_e4m3(PM, 128) | (MODE == kInput ? kBTransposed : 0u);
                uint32_t it = 0, pt = 0;
                bool ok = true;
                for (int i = pair; ok && i < work.total; i += npairs) {
                    const int blocks = work.tile(a, sm.tt, i, 0).blocks;
                    for (int kb = 0; ok && kb < blocks; ++kb, ++it) {
                        const int s = it % STAGES;
                        if (!wait_phase<true>(&b->full[s], (it / STAGES) & 1, a.timeout_ns, ab)) {
                            fail(b, a.status);
                            ok = false;
                            break;
                        }
                        const uint32_t sa = smem_u32(sm.stages + s * STAGE_BYTES), sb = sa + A_BYTES;
#pragma unroll
                        for (int h = 0; h < H; ++h, ++pt) {
                            const uint32_t pb = pt % NPART;
                            if (!wait_phase<true>(&b->pempty[pb], ((pt / NPART) & 1) ^ 1, a.timeout_ns,
                                                  ab)) {
                                fail(b, a.status);
                                ok = false;
                                break;
                            }
                            tc_fence_after_sync();
#pragma unroll
                            for (int kk = 0; kk < BK / 32; ++kk) {
                                // K-major: half h starts 64 rows on, a K step 32 bytes on.
                                // kInput: half h starts 64 bytes on in the rows (N innermost),
                                // a K step 32 rows on.
                                const uint32_t bo = MODE == kInput ? h * 64 + kk * 32 * 128
                                                                   : h * 64 * 128 + kk * 32;
                                umma_e4m3_pair(tmem + pb * 128, sdesc_k_sw128(sa + kk * 32),
                                               sdesc_k_sw128(sb + bo), idesc, kk != 0);
                            }
                            umma_commit_pair(&b->pfull[pb], kPairMask);
                        }
                        umma_commit_pair(&b->empty[s], kPairMask);
                    }
                }
            }
        } else {
            // ------------------------------------------------ scales, SC_KB blocks at a time
            const float* row_scale = a.a_scale;
            uint32_t cc = 0;
            bool ok = true;
            for (int i = pair; ok && i < work.total; i += npairs) {
                const PTile t = work.tile(a, sm.tt, i, rank);
                const int nb = a.N / 128, kbs = a.K / 128;
                for (int k0 = 0; k0 < t.blocks; k0 += SC_KB, ++cc) {
                    const int buf = cc % SC_BUFS;
                    if (!warp_wait_phase(&b->sempty[buf], ((cc / SC_BUFS) & 1) ^ 1, a.timeout_ns, ab)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = smem_u32(sm.scales + buf * SC_KB * SL::PER_KB);
                    const int n = min(SC_KB, t.blocks - k0);
                    if (MODE == kWeight) {
                        for (int kk = 0; kk < n; ++kk) {
                            const int64_t blk = t.block0 + k0 + kk;
                            for (int r = lane; r < BM; r += 32)
                                cp_async_4(dst + 4u * (kk * SL::PER_KB + r),
                                           row_scale + blk * a.N + min(t.row0 + r, a.N - 1), 4u);
                            for (int c = lane; c < BN; c += 32)
                                cp_async_4(dst + 4u * (kk * SL::PER_KB + BM + c),
                                           a.b_scale + blk * a.K + min(t.col0 + c, a.K - 1), 4u);
                        }
                    } else {
                        const int per_row = MODE == kForward ? kbs : nb;
                        for (int j = lane; j < BM * SC_KB; j += 32) {
                            const int r = j / SC_KB, kk = j % SC_KB;
                            if (kk < n) {
                                const bool in = r < t.nrows;
                                cp_async_4(dst + 4u * (kk * SL::PER_KB + r),
                                           row_scale + (in ? (int64_t)(t.row0 + r) * per_row + k0 + kk : 0),
                                           in ? 4u : 0u);
                            }
                        }
                        const int c = lane & 1, kk = lane >> 1;  // two column blocks x SC_KB
                        if (kk < n) {
                            const int last = (MODE == kForward ? nb : kbs) - 1;
                            const int cb = min(t.col0 / 128 + c, last);
                            const int64_t at = (int64_t)t.g * nb * kbs +
                                               (MODE == kForward ? (int64_t)cb * kbs + k0 + kk
                                                                 : (int64_t)(k0 + kk) * kbs + cb);
                            cp_async_4(dst + 4u * (kk * SL::PER_KB + BM + c), a.b_scale + at, 4u);
                        }
                    }
                    cp_async_mbar_arrive_noinc(&b->sfull[buf]);
                }
            }
            if (!ok && lane == 0) fail(b, a.status);
            cp_async_commit();
            cp_async_wait<0>();
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        // ---------------------------------------------------- promotion and output
        const int quad = warp & 3, half = (warp >> 2) & 1, cb = warp >> 3;
        const int row = quad * 32 + lane;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + cb * 64;
        uint32_t pt = half, cc = 0;
        bool ok = true;
        for (int i = pair; ok && i < work.total; i += npairs) {
            const PTile t = work.tile(a, sm.tt, i, rank);
            uint64_t acc[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[j] = 0ull;
#pragma unroll 1
            for (int kb = 0; kb < t.blocks; ++kb, pt += H) {
                const int kk = kb % SC_KB, buf = cc % SC_BUFS;
                if (kk == 0 &&
                    !warp_wait_phase(&b->sfull[buf], (cc / SC_BUFS) & 1, a.timeout_ns, ab)) {
                    ok = false;
                    break;
                }
                const float* sc = sm.scales + (buf * SC_KB + kk) * SL::PER_KB;
                float f = sc[row];
                if (MODE != kWeight) f *= sc[BM + cb];
                const uint64_t ff = f32x2_pack(f, f);
                const uint32_t pb = pt % NPART;
                if (!warp_wait_phase(&b->pfull[pb], (pt / NPART) & 1, a.timeout_ns, ab)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const float* cs = sc + BM + cb * 128 + half * 64;
                promote32<MODE == kWeight>(taddr + pb * 128, ff, cs, acc);
                promote32<MODE == kWeight>(taddr + pb * 128 + 32, ff, cs + 32, acc + 16);
                tc_fence_before_sync();
                warp_arrive_leader(&b->pempty[pb]);
                if (kk == SC_KB - 1 || kb == t.blocks - 1) {
                    if (lane == 0) mbar_arrive(&b->sempty[buf]);
                    ++cc;
                }
            }
            if (!ok) {
                if (lane == 0) fail(b, a.status);
                break;
            }
            const int cols = MODE == kForward ? a.N : a.K;
            const int col = t.col0 + cb * 128 + half * 64;
            if (row < t.nrows && col < cols && !(MODE == kWeight && a.accumulate && t.blocks == 0)) {
                const int64_t r = MODE == kWeight ? (int64_t)t.g * a.N + t.row0 + row : t.row0 + row;
                store32<MODE>(a, r * cols + col, acc);
                store32<MODE>(a, r * cols + col + 32, acc + 16);
            }
            __syncwarp();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still touch it
    if (warp == MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

template <Mode MODE>
cudaError_t set_up_once() {
    static bool done[64] = {false};
    const int dev = current_device_info().device;
    if (dev < 64 && done[dev]) return cudaSuccess;
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, k_product_pair<MODE>);
    if (e != cudaSuccess) return e;
    if (at.numRegs != REGS) return cudaErrorInvalidConfiguration;  // the split would not add up
    e = cudaFuncSetAttribute(k_product_pair<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes<MODE>());
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

template <Mode MODE>
cudaError_t launch_pair(const Fp8ProductArgs& a, cudaStream_t s) {
    CUtensorMap ta, tb;
    bool ok;
    int64_t tiles;
    if (MODE == kForward) {
        ok = make_tmap_2d(&ta, a.a, 1, a.M, a.K, BM, BK) &&
             make_tmap_2d(&tb, a.b, 1, (uint64_t)a.G * a.N, a.K, BN / 2, BK);
    } else if (MODE == kInput) {
        ok = make_tmap_2d(&ta, a.a, 1, a.M, a.N, BM, BK) &&
             make_tmap_2d(&tb, a.b, 1, (uint64_t)a.G * a.N, a.K, BK, BN / 2);
    } else {
        ok = make_tmap_2d(&ta, a.a, 1, a.N, a.rows_t, BM, BK) &&
             make_tmap_2d(&tb, a.b, 1, a.K, a.rows_t, BN / 2, BK);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (MODE == kWeight)
        tiles = (int64_t)a.G * ((a.N + PM - 1) / PM) * ((a.K + BN - 1) / BN);
    else  // the groups' rows are known on the device only: at most this many
        tiles = ((int64_t)a.M / PM + (a.G < a.M ? a.G : a.M)) *
                (((MODE == kForward ? a.N : a.K) + BN - 1) / BN);
    if (tiles >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    cudaError_t e = set_up_once<MODE>();
    if (e != cudaSuccess) return e;
    const int64_t pairs = current_device_info().num_sms / 2;
    e = launch_pdl(k_product_pair<MODE>, dim3(2 * (unsigned)(tiles < pairs ? tiles : pairs)),
                   dim3(THREADS), smem_bytes<MODE>(), s, ta, tb, a);
    return e != cudaSuccess ? e : cudaGetLastError();
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
    return launch_pair<kForward>(a, s);
}

cudaError_t launch_gemm_fp8_dgrad(const Fp8ProductArgs& a, cudaStream_t s) {
    return launch_pair<kInput>(a, s);
}

cudaError_t launch_gemm_fp8_wgrad(const Fp8ProductArgs& a, cudaStream_t s) {
    return launch_pair<kWeight>(a, s);
}

}  // namespace moe
