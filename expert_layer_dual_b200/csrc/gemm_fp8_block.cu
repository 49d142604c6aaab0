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
constexpr int BN = 256;                        // output columns of a pair's tile
constexpr int STAGES = 6, A_BYTES = BM * BK, B_BYTES = BN / 2 * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int NPART = 2;                       // partial buffers of BN TMEM columns
constexpr uint32_t TMEM_COLS = 512;
constexpr int EPI_WARPS = 16;                  // epilogue warps, EPI_COLS columns each
constexpr int EPI_COLS = BN * 4 / EPI_WARPS;
constexpr int MMA_WARP = EPI_WARPS, A_WARP = EPI_WARPS + 1, B_WARP = EPI_WARPS + 2,
              SCALE_WARP = EPI_WARPS + 3;
constexpr int THREADS = 32 * (SCALE_WARP + 1);
// Registers: 640 threads x 96 at launch; the four helper warps fall to 32 and the
// sixteen epilogue warps (64 accumulators each) rise to 112: 512 * 112 + 128 * 32
// = 640 * 96 (checked against the compiled kernel before its first launch).
constexpr int REGS = 96, REGS_EPI = 112, REGS_HELP = 32;
constexpr int SC_KB = 4, SC_BUFS = 4;           // scales: chunks of 4 blocks, four chunks ahead
constexpr uint16_t kPairMask = 0x3;

// One chunk of scales, in floats: the CTA's 128 row scales of SC_KB blocks
// ([row][block] for kForward and kInput, as they lie in memory; [block][row] for
// kWeight), then the column side's: [block][2] weight scales, or [block][BN].
template <Mode MODE>
struct ScaleLayout {
    static constexpr int COLS = BM * SC_KB;  // where the column side's start
    static constexpr int CHUNK = COLS + SC_KB * (MODE == kWeight ? BN : 4);
    static constexpr int FLOATS = SC_BUFS * CHUNK;
};

struct Bars {
    uint64_t full[STAGES];      // leader: two arming arrivals (A and B) + both CTAs' bytes
    uint64_t done[STAGES];      // each CTA: the leader's multicast MMA commit: the stage is
                                // free and the block's partial is complete
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

// The block's shared memory by 32-bit shared addresses (generic pointers cost
// the loops registers they do not have).
struct Smem {
    uint32_t stages, scales, bars;
    TileTable* tt;
    __device__ __forceinline__ uint32_t full(int i) const { return bars + offsetof(Bars, full) + 8 * i; }
    __device__ __forceinline__ uint32_t done(int i) const { return bars + offsetof(Bars, done) + 8 * i; }
    __device__ __forceinline__ uint32_t pempty(int i) const { return bars + offsetof(Bars, pempty) + 8 * i; }
    __device__ __forceinline__ uint32_t sfull(int i) const { return bars + offsetof(Bars, sfull) + 8 * i; }
    __device__ __forceinline__ uint32_t sempty(int i) const { return bars + offsetof(Bars, sempty) + 8 * i; }
    __device__ __forceinline__ uint32_t abort_flag() const { return bars + offsetof(Bars, abort_flag); }
};

// ---------------------------------------------------------------- shared memory
__device__ __forceinline__ float lds(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a));
    return v;
}
__device__ __forceinline__ bool try_phase(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, P;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded wait for a phase (see mbar_wait); the timer and the abort flag are read
// once in 64 tries only.  It acquires at CTA scope in the leader too, whose
// barriers take arrivals from both CTAs: what they order are asynchronous copies
// (counted in bytes on the barrier) and TMEM reads, no generic memory write of
// the other CTA.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                           uint32_t abort_flag) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1;; ++n) {
        if (try_phase(bar, parity)) return true;
        if ((n & 63u) == 0) {
            int stop;
            asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(stop) : "r"(abort_flag) : "memory");
            const uint64_t t = global_timer_ns();
            if (t0 == 0) t0 = t;
            if (stop || t - t0 > timeout_ns) return false;
        }
    }
}

// Warp-collective: one outcome for the warp.
__device__ __forceinline__ bool warp_wait_phase(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                                uint32_t abort_flag) {
    return __all_sync(0xffffffffu, wait_phase(bar, parity, timeout_ns, abort_flag));
}

// True in one lane of a converged warp.  The single-thread roles run their loops
// with the whole warp and issue under this predicate: the operands then stay in
// uniform registers (an MMA of N = 128 issued by `lane == 0` took 80 cycles, so
// 64, the tensor core's own time).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void fail(const Smem& sm, int32_t* status) {
    report_status(status, MOE_ERR_DEVICE_TIMEOUT);
    asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(sm.abort_flag()) : "memory");
}

// Shared::cluster address of shared address a in the pair's leader.
__device__ __forceinline__ uint32_t in_leader(uint32_t a) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
    return r;
}

// One lane arrives on the leader's barrier (a cluster address).  Relaxed: what the
// barrier orders is the reuse of TMEM columns, whose loads this warp has waited
// for; no memory write travels with it, and a release at cluster scope would
// wait for the warp's stores to global memory.
__device__ __forceinline__ void warp_arrive_leader(uint32_t bar) {
    __syncwarp();
    if (elect_one())
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                     : "memory");
}

// A position in a ring of N slots: the slot and the parity of its round.
template <int N>
struct Ring {
    uint32_t slot = 0, round = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            round ^= 1u;
        }
    }
};

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
// umma_commit_pair and tma_load_2d_pair by shared addresses.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"(kPairMask)
        : "memory");
}
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster,
                                          int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y)
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

// ---------------------------------------------------------------- scales
__device__ __forceinline__ bool aligned16(const void* p) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// The scale warp: keeps SC_BUFS chunks of SC_KB blocks' scales in flight ahead of
// the epilogue (asynchronous copies that arrive on the chunk's barrier by
// themselves).  16-byte copies where the layout allows (four blocks of a row, or
// four columns, side by side and aligned), else 4-byte ones.  Rows and columns
// past the tile read a neighbour's scale or, past the matrix, the last one: what
// they scale is not stored.
template <Mode MODE>
__device__ __forceinline__ void scale_role(const Fp8ProductArgs& a, const Smem& sm, const Work<MODE>& work,
                                        uint32_t rank, int pair, int npairs) {
    using SL = ScaleLayout<MODE>;
    const int lane = threadIdx.x & 31;
    const int nb = a.N / 128, kbs = a.K / 128;
    const int per_row = MODE == kForward ? kbs : nb;
    const bool wide = MODE == kWeight ? aligned16(a.a_scale) && aligned16(a.b_scale)
                                      : aligned16(a.a_scale) && per_row % 4 == 0;
    Ring<SC_BUFS> ring;
    bool ok = true;
    for (int i = pair; ok && i < work.total; i += npairs) {
        const PTile t = work.tile(a, sm.tt, i, rank);
        for (int k0 = 0; k0 < t.blocks; k0 += SC_KB, ring.next()) {
            if (!warp_wait_phase(sm.sempty(ring.slot), ring.round ^ 1u, a.timeout_ns, sm.abort_flag())) {
                ok = false;
                break;
            }
            const uint32_t dst = sm.scales + 4u * ring.slot * SL::CHUNK;
            const int n = min(SC_KB, t.blocks - k0);
            if (MODE == kWeight) {
                for (int kk = 0; kk < n; ++kk) {
                    const int64_t blk = t.block0 + k0 + kk;
                    const float* ra = a.a_scale + blk * a.N;
                    const float* cb = a.b_scale + blk * a.K;
                    const uint32_t dr = dst + 4u * (kk * BM), dc = dst + 4u * (SL::COLS + kk * BN);
                    if (wide) {
                        const int r = lane * 4;
                        cp_async_16(dr + 4u * r, ra + min(t.row0 + r, a.N - 4), 16u);
#pragma unroll
                        for (int c = lane * 4; c < BN; c += 128)
                            cp_async_16(dc + 4u * c, cb + min(t.col0 + c, a.K - 4), 16u);
                    } else {
#pragma unroll 1
                        for (int r = lane; r < BM; r += 32)
                            cp_async_4(dr + 4u * r, ra + min(t.row0 + r, a.N - 1), 4u);
#pragma unroll 1
                        for (int c = lane; c < BN; c += 32)
                            cp_async_4(dc + 4u * c, cb + min(t.col0 + c, a.K - 1), 4u);
                    }
                }
            } else {
#pragma unroll 1
                for (int r = lane; r < BM; r += 32) {
                    const float* src = a.a_scale + (int64_t)min(t.row0 + r, a.M - 1) * per_row + k0;
                    const uint32_t d = dst + 16u * r;
                    if (wide) {
                        cp_async_16(d, src, 16u);
                    } else {
#pragma unroll 1
                        for (int kk = 0; kk < n; ++kk) cp_async_4(d + 4u * kk, src + kk, 4u);
                    }
                }
                const int c = lane & 1, kk = lane >> 1;  // two column blocks x SC_KB
                if (kk < n) {
                    const int last = (MODE == kForward ? nb : kbs) - 1;
                    const int col = min(t.col0 / 128 + c, last);
                    const int64_t at = (int64_t)t.g * nb * kbs +
                                       (MODE == kForward ? (int64_t)col * kbs + k0 + kk
                                                         : (int64_t)(k0 + kk) * kbs + col);
                    cp_async_4(dst + 4u * (SL::COLS + kk * 4 + c), a.b_scale + at, 4u);
                }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm.sfull(ring.slot))
                         : "memory");
        }
    }
    if (!ok && lane == 0) fail(sm, a.status);
    cp_async_commit();
    cp_async_wait<0>();
}

// ---------------------------------------------------------------- epilogue
#define R4(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3])
#define W4(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3])
// 32 FP32 columns of this thread's TMEM lane; complete after tmem_arrived.
__device__ __forceinline__ void tmem_fetch32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : W4(r, 0), W4(r, 4), W4(r, 8), W4(r, 12), W4(r, 16), W4(r, 20), W4(r, 24), W4(r, 28)
        : "r"(taddr)
        : "memory");
}
// Waits for this thread's TMEM loads; names the registers, so that no use of them
// can be scheduled before it.
__device__ __forceinline__ void tmem_arrived(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : R4(r, 0), R4(r, 4), R4(r, 8), R4(r, 12), R4(r, 16), R4(r, 20), R4(r, 24), R4(r, 28)
                 :
                 : "memory");
}
#undef R4
#undef W4

// acc += f * (32 columns of the partial), in pairs; with column scales (at shared
// address cs): f * (cs * P).
template <bool COLSCALE>
__device__ __forceinline__ void promote32(const uint32_t* r, uint64_t ff, uint32_t cs, uint64_t* acc) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        uint64_t p0 = f32x2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        uint64_t p1 = f32x2_pack(__uint_as_float(r[2 * i + 2]), __uint_as_float(r[2 * i + 3]));
        if (COLSCALE) {
            const float4 s = lds4(cs + 8 * i);
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
// leader issues four M = 256, N = 256, K = 32 MMAs into a fresh partial (one of two
// in TMEM) and one commit; the epilogue warps take each partial out of TMEM and
// add it, scaled, to FP32 accumulators in registers while the next block's MMAs
// run.  CTA 0 loads the operand of the tile's first 128 columns, CTA 1 of the
// second, so a warp's columns have one weight scale.
//
// Measured, one pair per two SMs: four such MMAs take 512 cycles (the nominal
// rate), and a commit to both CTAs 70 to 90 of its issuer's time, so a block has
// one commit, which frees the stage and publishes the partial through the same
// barrier.
// ---------------------------------------------------------------------------
template <Mode MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    k_product_pair(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ Fp8ProductArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    using SL = ScaleLayout<MODE>;
    Smem sm;
    sm.stages = (smem_u32(smem_raw) + 1023u) & ~1023u;
    sm.scales = sm.stages + STAGES * STAGE_BYTES;
    sm.bars = sm.scales + 4 * SL::FLOATS;
    Bars* const b = reinterpret_cast<Bars*>(smem_raw + (sm.bars - smem_u32(smem_raw)));
    sm.tt = reinterpret_cast<TileTable*>(b + 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&b->full[s], 2);
            mbar_init(&b->done[s], 1);
        }
        for (int i = 0; i < NPART; ++i) mbar_init(&b->pempty[i], 2 * EPI_WARPS);
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
            const bool is_a = warp == A_WARP;
            const CUtensorMap* map = is_a ? &tm_a : &tm_b;
            if (elect_one()) tma_prefetch_desc(map);
            const uint32_t full_leader = in_leader(sm.full(0));
            const uint32_t bytes = 2 * (is_a ? A_BYTES : B_BYTES);  // both CTAs'
            const uint32_t dst0 = sm.stages + (is_a ? 0 : A_BYTES);
            Ring<STAGES> st;
            uint32_t issued = 0;
            bool ok = true;
            for (int i = pair; ok && i < work.total; i += npairs) {
                const PTile t = work.tile(a, sm.tt, i, rank);
                const int col = t.col0 + (int)rank * (BN / 2);
                int x, y;  // of the tile's first block
                if (is_a) {
                    x = t.block0 * BK;
                    y = t.row0;
                } else if (MODE == kForward) {
                    x = 0;
                    y = t.g * a.N + col;
                } else if (MODE == kInput) {
                    x = col;
                    y = t.g * a.N;
                } else {
                    x = t.block0 * BK;
                    y = col;
                }
                for (int kb = 0; kb < t.blocks; ++kb, st.next()) {
                    if (!warp_wait_phase(sm.done(st.slot), st.round ^ 1u, a.timeout_ns, sm.abort_flag())) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        if (rank == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
                                             sm.full(st.slot)),
                                         "r"(bytes)
                                         : "memory");
                        load_pair(dst0 + st.slot * STAGE_BYTES, map, full_leader + 8 * st.slot, x, y);
                    }
                    __syncwarp();
                    ++issued;
                    if (MODE == kInput && !is_a) y += BK; else x += BK;
                }
            }
            if (!ok && lane == 0) fail(sm, a.status);
            // after a failure the pair's copies in flight are waited for (bounded)
            if (rank == 0 && lane == 0 && *reinterpret_cast<volatile int*>(&b->abort_flag))
                for (uint32_t j = issued > STAGES ? issued - STAGES : 0; j < issued; ++j)
                    mbar_wait(&b->full[j % STAGES], (j / STAGES) & 1, a.timeout_ns, nullptr);
        } else if (warp == MMA_WARP) {
            // ------------------------------------------------ MMA issuer (leader)
            if (rank == 0) {
                constexpr uint32_t idesc = idesc_e4m3(PM, BN) | (MODE == kInput ? kBTransposed : 0u);
                Ring<STAGES> st;
                Ring<NPART> pt;
                bool ok = true;
                for (int i = pair; ok && i < work.total; i += npairs) {
                    const int blocks = work.tile(a, sm.tt, i, 0).blocks;
                    for (int kb = 0; kb < blocks; ++kb, st.next(), pt.next()) {
                        if (!warp_wait_phase(sm.full(st.slot), st.round, a.timeout_ns, sm.abort_flag()) ||
                            !warp_wait_phase(sm.pempty(pt.slot), pt.round ^ 1u, a.timeout_ns,
                                             sm.abort_flag())) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t sa = sm.stages + st.slot * STAGE_BYTES, sb = sa + A_BYTES;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < BK / 32; ++kk)
                                // a K step: 32 bytes on (K innermost), or 32 rows on (kInput)
                                umma_e4m3_pair(tmem + pt.slot * BN, sdesc_k_sw128(sa + kk * 32),
                                               sdesc_k_sw128(sb + (MODE == kInput ? kk * 32 * 128 : kk * 32)),
                                               idesc, kk != 0);
                            commit_pair(sm.done(st.slot));
                        }
                        __syncwarp();
                    }
                }
                if (!ok && lane == 0) fail(sm, a.status);
            }
        } else {
            // ------------------------------------------------ scales, SC_KB blocks at a time
            scale_role<MODE>(a, sm, work, rank, pair, npairs);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        // ---------------------------------------------------- promotion and output
        const int quad = warp & 3, part = warp >> 2;  // TMEM lanes, columns
        const int row = quad * 32 + lane;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + part * EPI_COLS;
        const uint32_t pempty_leader = in_leader(sm.pempty(0));
        constexpr bool CS = MODE == kWeight;
        constexpr int NQ = EPI_COLS / 32;
        Ring<STAGES> st;
        Ring<SC_BUFS> ch;
        uint32_t pb = 0;
        bool ok = true;
        for (int i = pair; ok && i < work.total; i += npairs) {
            const int blocks = work.tile(a, sm.tt, i, rank).blocks;
            uint64_t acc[16 * NQ];
#pragma unroll
            for (int j = 0; j < 16 * NQ; ++j) acc[j] = 0ull;
#pragma unroll 1
            for (int kb = 0; kb < blocks; ++kb) {
                const int kk = kb % SC_KB;
                if (kk == 0 && !warp_wait_phase(sm.sfull(ch.slot), ch.round, a.timeout_ns, sm.abort_flag())) {
                    ok = false;
                    break;
                }
                const uint32_t sc = sm.scales + 4u * ch.slot * SL::CHUNK;
                float f = lds(sc + 4u * (CS ? kk * BM + row : row * SC_KB + kk));
                if (!CS) f *= lds(sc + 4u * (SL::COLS + kk * 4 + part * EPI_COLS / 128));
                const uint64_t ff = f32x2_pack(f, f);
                const uint32_t cs = sc + 4u * (SL::COLS + kk * BN + part * EPI_COLS);
                if (!warp_wait_phase(sm.done(st.slot), st.round, a.timeout_ns, sm.abort_flag())) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                uint32_t r[32];
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    tmem_fetch32(taddr + pb * BN + 32 * q, r);
                    tmem_arrived(r);
                    if (q == NQ - 1) {  // the partial is in registers
                        tc_fence_before_sync();
                        warp_arrive_leader(pempty_leader + 8 * pb);
                    }
                    promote32<CS>(r, ff, cs + 128 * q, acc + 16 * q);
                }
                st.next();
                pb ^= 1u;
                if (kk == SC_KB - 1 || kb == blocks - 1) {
                    __syncwarp();
                    if (elect_one()) arrive(sm.sempty(ch.slot));
                    ch.next();
                }
            }
            if (!ok) {
                if (lane == 0) fail(sm, a.status);
                break;
            }
            // decoded again rather than kept: the loop has no registers to spare
            const PTile t = work.tile(a, sm.tt, i, rank);
            const int cols = MODE == kForward ? a.N : a.K;
            const int col = t.col0 + part * EPI_COLS;
            if (row < t.nrows && col < cols && !(MODE == kWeight && a.accumulate && t.blocks == 0)) {
                const int64_t r = MODE == kWeight ? (int64_t)t.g * a.N + t.row0 + row : t.row0 + row;
#pragma unroll
                for (int q = 0; q < NQ; ++q) store32<MODE>(a, r * cols + col + 32 * q, acc + 16 * q);
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
