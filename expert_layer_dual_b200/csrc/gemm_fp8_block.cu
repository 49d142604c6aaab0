// gemm_fp8_block.cu -- the FP8 e4m3 matrix product with one FP32 scale per block
// of 128, its two gradients, and the quantiser of the weight gradient's
// operands.
//
//   y  [m][n] = sum_b xs[m][b] ws[n/128][b] sum_{k in b} xq[m][k] wq[n][k]
//   dx [m][k] = sum_b ds[m][b] ws[b][k/128] sum_{n in b} dq[m][n] wq[n][k]
//   dw [n][k] = sum_b ds[b][n] xs[b][k]     sum_{m in b} dq[m][n] xq[m][k]
// (b: blocks of 128 of the summed index).  The rows m form G groups with one
// weight matrix each (offsets), or one group of all rows.
#include <atomic>
#include <mutex>

#include "common.cuh"
#include "fp8_block.cuh"
#include "launch.h"

namespace moe {
namespace {

enum Mode { kForward, kInput, kWeight };

constexpr int BM = 128, BN = 256, BK = 128;    // a tile's rows and columns; one scale block of the sum
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int MAX_STAGES = 4;                  // operands of as many blocks;
template <Mode MODE>                           // kWeight: three, and the output on its way out
constexpr int kStages = MODE == kWeight ? 3 : MAX_STAGES;
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
constexpr int SC_KB = 4, MAX_SC_BUFS = 4;       // scales: chunks of 4 blocks,
template <Mode MODE>
constexpr int kScBufs = MODE == kWeight ? 2 : MAX_SC_BUFS;  // as many ahead
constexpr int OUT_ATOM = 8 * 128;               // kWeight: 8 rows x 32 columns of the output,
constexpr int OUT_WARP = 4 * OUT_ATOM;          // two pairs of them per epilogue warp

// One chunk of scales, in floats: the CTA's 128 row scales of SC_KB blocks
// ([row][block] for kForward and kInput, as they lie in memory; [block][row] for
// kWeight), then the column side's: [block][2] weight scales, or [block][BN].
template <Mode MODE>
struct ScaleLayout {
    static constexpr int COLS = BM * SC_KB;  // where the column side's start
    static constexpr int CHUNK = COLS + SC_KB * (MODE == kWeight ? BN : 4);
    static constexpr int FLOATS = kScBufs<MODE> * CHUNK;
};

struct Bars {
    uint64_t full[MAX_STAGES];  // two arming arrivals (A and B) + their bytes
    uint64_t done[MAX_STAGES];  // MMA commit: the stage is free, the block's partial complete
    uint64_t pempty[NPART];     // partial read (one arrival per epilogue warp)
    uint64_t sfull[MAX_SC_BUFS];   // scale chunk landed (32 asynchronous arrivals)
    uint64_t sempty[MAX_SC_BUFS];  // scale chunk read (one arrival per epilogue warp)
    uint32_t tmem_slot;
    int abort_flag;
};

template <Mode MODE>
constexpr size_t smem_bytes() {
    return 1024 + kStages<MODE> * STAGE_BYTES + (MODE == kWeight ? EPI_WARPS * OUT_WARP : 0) +
           ScaleLayout<MODE>::FLOATS * 4 + sizeof(Bars) +
           sizeof(TileTable) + 64;
}

// The block's shared memory, by shared addresses.
struct Smem {
    uint32_t stages, out, scales, bars;
    TileTable* tt;
    __device__ __forceinline__ uint32_t full(int i) const { return bars + offsetof(Bars, full) + 8 * i; }
    __device__ __forceinline__ uint32_t done(int i) const { return bars + offsetof(Bars, done) + 8 * i; }
    __device__ __forceinline__ uint32_t pempty(int i) const { return bars + offsetof(Bars, pempty) + 8 * i; }
    __device__ __forceinline__ uint32_t sfull(int i) const { return bars + offsetof(Bars, sfull) + 8 * i; }
    __device__ __forceinline__ uint32_t sempty(int i) const { return bars + offsetof(Bars, sempty) + 8 * i; }
    __device__ __forceinline__ uint32_t abort_flag() const { return bars + offsetof(Bars, abort_flag); }
};

__device__ __forceinline__ void fail(const Smem& sm, int32_t* status) {
    report_status(status, MOE_ERR_DEVICE_TIMEOUT);
    asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(sm.abort_flag()) : "memory");
}

// ---------------------------------------------------------------- tiles
// One tile: rows row0 .. (nrows <= 128) and columns col0 .. (256) of the output, group
// g, and the scale blocks [block0, block0 + blocks) that this CTA sums over (kWeight:
// token blocks of the group; else all of them, from 0), or its share of them.
struct PTile {
    int g, row0, nrows, col0, block0, blocks;
};

// SPLIT: a cluster of a.split CTAs works on each tile, CTA `rank` on its share of the
// blocks (four at a time, as the scales are read).
template <Mode MODE, bool SPLIT>
struct Work {
    int total, n_tiles, k_tiles, blocks, first, step;
    __device__ __forceinline__ Work(const Fp8ProductArgs& a, const TileTable* tt) {
        if (MODE == kWeight) {
            n_tiles = (a.K + BN - 1) / BN;
            k_tiles = a.N / BM;
            total = a.G * n_tiles * k_tiles;
        } else {
            n_tiles = ((MODE == kForward ? a.N : a.K) + BN - 1) / BN;
            blocks = (MODE == kForward ? a.K : a.N) / BK;
            total = tt->mstart[a.G] * n_tiles;
        }
        first = SPLIT ? blockIdx.x / a.split : blockIdx.x;
        step = SPLIT ? gridDim.x / a.split : gridDim.x;
    }
    __device__ __forceinline__ PTile tile(const Fp8ProductArgs& a, const TileTable* tt, int i) const {
        PTile p;
        if (MODE == kWeight) {
            const int per = n_tiles * k_tiles;
            p.g = i / per;
            const int r = i - p.g * per;
            // rows first (columns first, 8192 x 4096 x 6144 took 252 us, so 249, and 32 experts of
            // 2048 x 1408 over 5003 rows 78.6, so 76.1)
            p.row0 = (r % k_tiles) * BM;
            p.nrows = BM;
            p.col0 = (r / k_tiles) * BN;
            p.block0 = tt->mstart[p.g];
            p.blocks = tt->mstart[p.g + 1] - p.block0;
        } else {
            const Tile t = decode_tile(tt, a.G, n_tiles, i, BM);
            p.g = t.g;
            p.row0 = t.row0;
            p.nrows = t.nrows;
            p.col0 = t.n * BN;
            p.block0 = 0;
            p.blocks = blocks;
        }
        if (SPLIT) {
            const int size = a.split, per = ((p.blocks + size - 1) / size + SC_KB - 1) / SC_KB * SC_KB;
            const int lo = min(p.blocks, (int)(blockIdx.x % size) * per);
            p.block0 += lo;
            p.blocks = min(p.blocks - lo, per);
        }
        return p;
    }
};

// ---------------------------------------------------------------- scales
// The scale warp: keeps kScBufs chunks of SC_KB blocks' scales in flight ahead of
// the epilogue (asynchronous copies that arrive on the chunk's barrier by
// themselves).  16-byte copies where the layout allows (four blocks of a row, or
// four columns, side by side and aligned), else 4-byte ones.  Rows and columns
// past the tile read a neighbour's scale or, past the matrix, the last one: what
// they scale is not stored.
template <Mode MODE, bool SPLIT>
__device__ __forceinline__ void scale_role(const Fp8ProductArgs& a, const Smem& sm, const Work<MODE, SPLIT>& work) {
    using SL = ScaleLayout<MODE>;
    const int lane = threadIdx.x & 31;
    const int nb = a.N / 128, kbs = a.K / 128;
    const int per_row = MODE == kForward ? kbs : nb;
    const bool wide = MODE == kWeight ? aligned16(a.a_scale) && aligned16(a.b_scale)
                                      : aligned16(a.a_scale) && per_row % 4 == 0;
    Ring<kScBufs<MODE>> ring;
    bool ok = true;
    for (int i = work.first; ok && i < work.total; i += work.step) {
        const PTile t = work.tile(a, sm.tt, i);
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
                    const float* src =
                        a.a_scale + (int64_t)min(t.row0 + r, a.M - 1) * per_row + t.block0 + k0;
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
                                       (MODE == kForward ? (int64_t)col * kbs + t.block0 + k0 + kk
                                                         : (int64_t)(t.block0 + k0 + kk) * kbs + col);
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
// acc += f * (COLS columns of the partial), in pairs.
template <int COLS>
__device__ __forceinline__ void promote(const uint32_t* r, uint64_t ff, uint64_t* acc) {
#pragma unroll
    for (int i = 0; i < COLS / 2; ++i)
        acc[i] = f32x2_fma(ff, f32x2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), acc[i]);
}
// The same with column scales, for what tmem_fetch16 brings: f of rows l / 4 and l / 4
// + 8, c the scales of this thread's columns.
__device__ __forceinline__ void promote_scaled(const uint32_t* r, float f0, float f1, const uint64_t* c,
                                               uint64_t* acc0, uint64_t* acc1) {
    const uint64_t ff0 = f32x2_pack(f0, f0), ff1 = f32x2_pack(f1, f1);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const uint64_t p0 = f32x2_pack(__uint_as_float(r[4 * g]), __uint_as_float(r[4 * g + 1]));
        const uint64_t p1 = f32x2_pack(__uint_as_float(r[4 * g + 2]), __uint_as_float(r[4 * g + 3]));
        acc0[g] = f32x2_fma(ff0, f32x2_mul(p0, c[g]), acc0[g]);
        acc1[g] = f32x2_fma(ff1, f32x2_mul(p1, c[g]), acc1[g]);
    }
}

// Four chunks of eight words in each of four neighbouring lanes, turned: lane j of the
// four ends with chunk j of all four lanes, in lane order.  The accumulators hold
// a row per lane; turned, the four lanes store 128 consecutive bytes of one row
// at a time.  (A store of 32 bytes from each of 32 rows keeps the store unit four
// times as long: a weight gradient bound by its output took 103 us so, 85 turned.)
__device__ __forceinline__ void turn_chunks(uint32_t* v) {
    const int j = threadIdx.x & 3;
#pragma unroll
    for (int step = 1; step < 4; step <<= 1) {
        const bool up = (j & step) != 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & step) continue;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                uint32_t &lo = v[8 * k + w], &hi = v[8 * (k + step) + w];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, step);
                if (up) lo = got; else hi = got;
            }
        }
    }
}

// Eight words at p: one 32-byte store where p is aligned for it.
__device__ __forceinline__ void store8(uint32_t* p, const uint32_t* v) {
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                     "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        st_global_v4(p, v[0], v[1], v[2], v[3]);
        st_global_v4(p + 4, v[4], v[5], v[6], v[7]);
    }
}

// kForward, kInput: writes a warp's 32 rows x EPI_COLS columns: row0 is the output row of lane 0, `valid`
// of the rows are stored, acc the lane's row.
__device__ __forceinline__ void store_tile(const Fp8ProductArgs& a, int64_t row0, int valid, int cols, int col,
                                           const uint64_t* acc) {
    static_assert(EPI_COLS == 64, "two halves of 32 words, or one of 32 pairs");
    const int lane = threadIdx.x & 31, first = lane & ~3, j = lane & 3;
    if (a.out_type == MOE_OUT_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float lo, hi;
                f32x2_unpack(acc[16 * h + i], lo, hi);
                w[2 * i] = __float_as_uint(lo);
                w[2 * i + 1] = __float_as_uint(hi);
            }
            turn_chunks(w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (first + i >= valid) break;
                float* dst = static_cast<float*>(a.out) + (row0 + first + i) * cols + col + 32 * h + 8 * j;
                store8(reinterpret_cast<uint32_t*>(dst), w + 8 * i);
            }
        }
    } else {
        const bool f16 = a.out_type == MOE_OUT_F16;
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float lo, hi;
            f32x2_unpack(acc[i], lo, hi);
            w[i] = f16 ? pack_f16x2_sat(lo, hi) : pack_bf16x2(lo, hi);
        }
        turn_chunks(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (first + i >= valid) break;
            uint16_t* dst = static_cast<uint16_t*>(a.out) + (row0 + first + i) * cols + col + 16 * j;
            store8(reinterpret_cast<uint32_t*>(dst), w + 8 * i);
        }
    }
}

template <int PENDING>  // bulk stores of this thread that may still read shared memory
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(PENDING) : "memory");
}
template <int PENDING>
__device__ __forceinline__ void bulk_wait() {
    asm volatile("cp.async.bulk.wait_group %0;" ::"n"(PENDING) : "memory");
}

// kWeight: sends a warp's 32 rows x EPI_COLS columns on their way through shared memory
// (`buf`, two slots of eight rows), while the warp goes on to the next tile.  In
// shared memory the rows of 32 columns lie as the tensor map's 128-byte swizzle has
// them: 16-byte piece p of row r in place p ^ r.  (Stored from registers, after turning
// chunks among four lanes, 32 experts of 2048 x 1408 over 5003 rows, 369 MB of output,
// took 84.0 us, so 78.6, and 76.1 with rows first; without the L2 policy 1.5 us more.  The bytes
// alone take 50 us as a fill, 56 at the copy's rate.  Added to the output, which reads them
// too, 166 us: the loads stand in front of the staging.)  A lane has row l / 4 and of each
// eight columns a pair; odd rows take the groups of eight in another order, so that
// the stores of half a warp fall on distinct banks.
__device__ __forceinline__ void send_tile(const Fp8ProductArgs& a, const CUtensorMap* map, uint32_t buf,
                                          int64_t row0, int col, uint64_t* acc) {
    const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    const bool odd = (r & 1) != 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (a.accumulate) {
            const float* old = static_cast<const float*>(a.out) + (row0 + 8 * q + r) * a.K + col + 2 * j;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const float2 o = *reinterpret_cast<const float2*>(old + 8 * g);
                float lo, hi;
                f32x2_unpack(acc[8 * q + g], lo, hi);
                acc[8 * q + g] = f32x2_pack(lo + o.x, hi + o.y);
            }
        }
        const uint32_t slot = buf + (q & 1) * 2 * OUT_ATOM;
        if (lane == 0) bulk_wait_read<1>();  // what was sent from this slot last
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint64_t v = odd ? acc[8 * q + 4 * h + (g ^ 2)] : acc[8 * q + 4 * h + g];
                const int piece = (2 * (odd ? g ^ 2 : g) + (j >> 1)) ^ r;
                asm volatile("st.shared.b64 [%0], %1;" ::"r"(slot + h * OUT_ATOM + 128 * r + 16 * piece + 8 * (j & 1)),
                             "l"(v)
                             : "memory");
            }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            uint64_t first_out;  // the operands stay in L2 rather than the output
            asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first_out));
#pragma unroll
            for (int h = 0; h < 2; ++h)
                asm volatile(
                    "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group.L2::cache_hint "
                    "[%0, {%1, %2}], [%3], %4;" ::"l"(map),
                    "r"(col + 32 * h), "r"((int)(row0 + 8 * q)), "r"(slot + h * OUT_ATOM), "l"(first_out)
                    : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
}

// A tile split over a cluster: every CTA leaves its sums in its shared memory (where
// the operands were: every MMA that read them is complete), and adds its share of
// the rows over the CTAs, in rank order.
constexpr int LEFT_COLS = BN + 8;  // of a row: eight rows' pairs, or quarters, on distinct banks
static_assert(BM * LEFT_COLS * 4 <= 3 * STAGE_BYTES, "the tile fits where the operands were");

template <Mode MODE>
__device__ __forceinline__ void leave_tile(const Smem& sm, int quad, int part, int lane, const uint64_t* acc) {
    if (MODE == kWeight) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const int at = (quad * 32 + 8 * q + (lane >> 2)) * LEFT_COLS + part * EPI_COLS + 8 * g + 2 * (lane & 3);
                asm volatile("st.shared.b64 [%0], %1;" ::"r"(sm.stages + 4u * at), "l"(acc[8 * q + g]) : "memory");
            }
    } else {
#pragma unroll
        for (int i = 0; i < EPI_COLS / 4; ++i) {
            const int at = (quad * 32 + lane) * LEFT_COLS + part * EPI_COLS + 4 * i;
            asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(sm.stages + 4u * at), "l"(acc[2 * i]),
                         "l"(acc[2 * i + 1])
                         : "memory");
        }
    }
}

// Whether CTA `rank` of the cluster gave up before the cluster's barrier: its shared
// memory then holds no sums.
__device__ __forceinline__ bool share_failed(const Smem& sm, int rank) {
    uint32_t at;
    int flag;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sm.abort_flag()), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(flag) : "r"(at) : "memory");
    return flag != 0;
}

template <Mode MODE, int SIZE>
__device__ __forceinline__ void add_tiles(const Fp8ProductArgs& a, const Smem& sm, const PTile& t, int warp,
                                          int lane) {
    const int rank = blockIdx.x % SIZE, cols = MODE == kForward ? a.N : a.K, col = t.col0 + 8 * lane;
    if (col >= cols) return;
    // nothing to add to a group without rows
    if (MODE == kWeight && a.accumulate && sm.tt->mstart[t.g] == sm.tt->mstart[t.g + 1]) return;
    const int64_t row0 = MODE == kWeight ? (int64_t)t.g * a.N + t.row0 : t.row0;
    uint32_t from[SIZE];
#pragma unroll
    for (int c = 0; c < SIZE; ++c)
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from[c]) : "r"(sm.stages + 32u * lane), "r"(c));
#pragma unroll 1
    for (int r = rank * (BM / SIZE) + warp; r < (rank + 1) * (BM / SIZE); r += EPI_WARPS) {
        if (r >= t.nrows) break;
        float s[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 v[SIZE];
#pragma unroll
            for (int c = 0; c < SIZE; ++c)
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(v[c].x), "=f"(v[c].y), "=f"(v[c].z), "=f"(v[c].w)
                             : "r"(from[c] + 4u * r * LEFT_COLS + 16u * h)
                             : "memory");
            float4 u = v[0];
#pragma unroll
            for (int c = 1; c < SIZE; ++c) {
                u.x += v[c].x;
                u.y += v[c].y;
                u.z += v[c].z;
                u.w += v[c].w;
            }
            s[4 * h] = u.x;
            s[4 * h + 1] = u.y;
            s[4 * h + 2] = u.z;
            s[4 * h + 3] = u.w;
        }
        const int64_t at = (row0 + r) * cols + col;
        if (MODE == kWeight || a.out_type == MOE_OUT_F32) {
            float* dst = static_cast<float*>(a.out) + at;
            if (MODE == kWeight && a.accumulate) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] += dst[i];
            }
            st_global_v4(dst, __float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]),
                         __float_as_uint(s[3]));
            st_global_v4(dst + 4, __float_as_uint(s[4]), __float_as_uint(s[5]), __float_as_uint(s[6]),
                         __float_as_uint(s[7]));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = a.out_type == MOE_OUT_F16 ? pack_f16x2_sat(s[2 * i], s[2 * i + 1])
                                                 : pack_bf16x2(s[2 * i], s[2 * i + 1]);
            st_global_v4(static_cast<uint16_t*>(a.out) + at, w[0], w[1], w[2], w[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// The product.  Per scale block of the summed index one warp issues four M = 128,
// N = 256, K = 32 MMAs into a fresh partial (one of two in TMEM) and one commit,
// which frees the stage and publishes the partial through the same barrier; the
// epilogue warps take each partial out of TMEM and add it, scaled, to FP32
// accumulators in registers while the next block's MMAs run.
//
// Bound: the tensor cores' 512 cycles a block (4 MMAs of 128), and the way round:
// commit, wait, TMEM loads, products, arrival, next issue.  Cycles per block of a
// 128 x 256 tile: 815 in all, 720 without the MMAs, 613 without the promotion,
// 520 with neither.  At large sizes the power limit levels what is left of the
// difference: 8192 x 4096 x 6144 takes 177 to 181 us (2.3 PFLOP/s) at ~1.5 GHz, 143 us
// without its promotion, and variants with 5% fewer cycles took the same time
// at a lower clock.  The weight gradient (two products a value) takes 249 us (268 added
// to the output), 4096 x 6144 x 2048 rows of the input gradient 49 us, 32 groups of 8192 rows
// 267 us (their 805 MB of weights alone 122 us; the groups' last tiles pad 336 tiles of
// rows to 432).
//
// Sixteen epilogue warps of 64 accumulators each fit without spills (480 cycles of
// promotion with spilled registers, so 256).  On CTA pairs (M = 256, the operands'
// shared-memory traffic a third less) the longer way round through the other
// CTA's barriers took what the rate gave: 187 against 185 us for 8192 x 4096 x 6144,
// and ragged groups lost to the 256-row tiles (290 against 275 us); so one CTA per
// tile.  128 x 128 tiles with four partials took 14% more cycles (weight gradient);
// two halves of the epilogue warps a partial apart, 4 to 12% more.
// ---------------------------------------------------------------------------
template <Mode MODE, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
    k_product(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ Fp8ProductArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    using SL = ScaleLayout<MODE>;
    constexpr int STAGES = kStages<MODE>;
    Smem sm;
    sm.stages = (smem_u32(smem_raw) + 1023u) & ~1023u;
    sm.out = sm.stages + STAGES * STAGE_BYTES;
    sm.scales = sm.out + (MODE == kWeight ? EPI_WARPS * OUT_WARP : 0);
    sm.bars = sm.scales + 4 * SL::FLOATS;
    Bars* const b = reinterpret_cast<Bars*>(smem_raw + (sm.bars - smem_u32(smem_raw)));
    sm.tt = reinterpret_cast<TileTable*>(b + 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&b->full[s], 2);
            mbar_init(&b->done[s], 1);
        }
        for (int i = 0; i < NPART; ++i) mbar_init(&b->pempty[i], EPI_WARPS);
        for (int i = 0; i < kScBufs<MODE>; ++i) {
            mbar_init(&b->sfull[i], 32);
            mbar_init(&b->sempty[i], EPI_WARPS);
        }
        b->abort_flag = 0;
        fence_barrier_init();
    }
    // What does not read the operands runs while the previous kernel drains.  The next
    // kernel may come once this one's TMEM is its own.
    if (warp == MMA_WARP) {
        tmem_alloc(&b->tmem_slot, TMEM_COLS);
        pdl_trigger();
    }
    if (warp == A_WARP && elect_one()) tma_prefetch_desc(&tm_a);
    if (warp == B_WARP && elect_one()) tma_prefetch_desc(&tm_b);
    pdl_wait();  // the operands come from the previous kernels
    if (warp == 0) build_group_table(sm.tt, a.offsets, a.G, a.M, MODE == kWeight ? BK : BM);
    // the status word: a wait that runs out does so seconds after this store
    if (blockIdx.x == 0 && threadIdx.x == 32) *a.status = MOE_OK;
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = b->tmem_slot;
    const Work<MODE, SPLIT> work(a, sm.tt);

    if (warp >= EPI_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_HELP));
        if (warp == A_WARP || warp == B_WARP) {
            // ------------------------------------------------ TMA: one operand each
            const bool is_a = warp == A_WARP;
            const CUtensorMap* map = is_a ? &tm_a : &tm_b;
            const uint32_t dst0 = sm.stages + (is_a ? 0 : A_BYTES);
            Ring<STAGES> st;
            st.round = 1u;  // a producer waits for the round before; in the self-test for one that never ends
            if (is_a && blockIdx.x + 1 == a.give_up) st.round = 0u;
            uint32_t issued = 0;
            bool ok = true;
            for (int i = work.first; ok && i < work.total; i += work.step) {
                const PTile t = work.tile(a, sm.tt, i);
                int x, y;  // of the tile's first block
                if (is_a) {
                    x = t.block0 * BK;
                    y = t.row0;
                } else if (MODE == kForward) {
                    x = t.block0 * BK;
                    y = t.g * a.N + t.col0;
                } else if (MODE == kInput) {
                    x = t.col0;
                    y = t.g * a.N + t.block0 * BK;
                } else {
                    x = t.block0 * BK;
                    y = t.col0;
                }
                for (int kb = 0; kb < t.blocks; ++kb, st.next()) {
                    if (!warp_wait_phase(sm.done(st.slot), st.round, a.timeout_ns, sm.abort_flag())) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t dst = dst0 + st.slot * STAGE_BYTES;
                        expect_bytes(sm.full(st.slot), is_a ? A_BYTES : B_BYTES);
                        tma_load(dst, map, sm.full(st.slot), x, y);
                        if (MODE == kInput && !is_a)  // rows of 128 columns: two boxes
                            tma_load(dst + B_BYTES / 2, map, sm.full(st.slot), x + 128, y);
                    }
                    __syncwarp();
                    ++issued;
                    if (MODE == kInput && !is_a) y += BK; else x += BK;
                }
            }
            if (!ok && lane == 0) fail(sm, a.status);
            // after a failure the copies in flight are waited for (bounded)
            if (lane == 0 && *reinterpret_cast<volatile int*>(&b->abort_flag))
                for (uint32_t j = issued > STAGES ? issued - STAGES : 0; j < issued; ++j)
                    mbar_wait(&b->full[j % STAGES], (j / STAGES) & 1, a.timeout_ns, nullptr);
        } else if (warp == MMA_WARP) {
            // ------------------------------------------------ MMA issuer
            constexpr uint32_t idesc = idesc_e4m3(BM, BN) | (MODE == kInput ? kBTransposed : 0u);
            Ring<STAGES> st;
            Ring<NPART> pt;
            bool ok = true;
            for (int i = work.first; ok && i < work.total; i += work.step) {
                const int blocks = work.tile(a, sm.tt, i).blocks;
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
                            // a K step: 32 bytes on (K innermost), or 32 rows on (kInput's B)
                            umma_e4m3(tmem + pt.slot * BN, sdesc_k_sw128(sa + kk * 32),
                                      MODE == kInput ? sdesc_mn_sw128(sb + kk * 32 * 128, B_BYTES / 2)
                                                     : sdesc_k_sw128(sb + kk * 32),
                                      idesc, kk != 0);
                        mma_commit(sm.done(st.slot));
                    }
                    __syncwarp();
                }
            }
            if (!ok && lane == 0) fail(sm, a.status);
        } else {
            // ------------------------------------------------ scales, SC_KB blocks at a time
            scale_role<MODE, SPLIT>(a, sm, work);
        }
        __syncwarp();
        if (SPLIT) cluster_sync();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        // ---------------------------------------------------- promotion and output
        const int quad = warp & 3, part = warp >> 2;  // TMEM lanes, columns
        const int row = quad * 32 + lane;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + part * EPI_COLS;
        constexpr bool CS = MODE == kWeight;
        uint32_t done = 0;  // blocks so far: their stages and partials follow from it
        Ring<kScBufs<MODE>> ch;
        bool ok = true;
        for (int i = work.first; ok && i < work.total; i += work.step) {
            const int blocks = work.tile(a, sm.tt, i).blocks;
            uint64_t acc[EPI_COLS / 2];
#pragma unroll
            for (int j = 0; j < EPI_COLS / 2; ++j) acc[j] = 0ull;
#pragma unroll 1
            for (int k0 = 0; ok && k0 < blocks; k0 += SC_KB, ch.next()) {
                if (!warp_wait_phase(sm.sfull(ch.slot), ch.round, a.timeout_ns, sm.abort_flag())) {
                    ok = false;
                    break;
                }
                const uint32_t sc = sm.scales + 4u * ch.slot * SL::CHUNK;
                const int n = min(SC_KB, blocks - k0);
#pragma unroll 1
                for (int kk = 0; kk < n; ++kk) {
                    float f[CS ? 4 : 1];  // CS: of rows lane / 4 + 8 q
                    if (CS) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) f[q] = lds(sc + 4u * (kk * BM + quad * 32 + 8 * q + (lane >> 2)));
                    } else {
                        f[0] = lds(sc + 4u * (row * SC_KB + kk)) *
                               lds(sc + 4u * (SL::COLS + kk * 4 + part * EPI_COLS / 128));
                    }
                    const uint32_t cs = sc + 4u * (SL::COLS + kk * BN + part * EPI_COLS + 2 * (lane & 3));
                    uint64_t c[4];  // CS: the scales of half this thread's columns
                    if (CS) {
#pragma unroll
                        for (int g = 0; g < 4; ++g) c[g] = lds2(cs + 32 * g);
                    }
                    if (!warp_wait_phase(sm.done(done % STAGES), done / STAGES & 1u, a.timeout_ns, sm.abort_flag())) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t pb = done % NPART, p = taddr + pb * BN;
                    auto release = [&] {  // the partial is in registers
                        tc_fence_before_sync();
                        __syncwarp();
                        if (elect_one()) arrive(sm.pempty(pb));
                    };
                    if constexpr (CS) {
                        // Four rows of sixteen columns a thread: with a row a thread, every
                        // thread would read all of its 64 columns' scales, 131 KB a block, more
                        // than shared memory gives in the block's time (298 against 274 us,
                        // 8192 rows x 4096 x 6144).  A quarter in flight over the products of
                        // another, the next scales ahead of the wait (274 against 260).
                        uint32_t r[2][16];
                        tmem_fetch16(p, r[0]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {  // rows of the lower and the upper half by turns
                            tmem_arrived16(r[q & 1]);
                            if (q + 1 < 4)
                                tmem_fetch16(p + ((q + 1) & 1) * (16u << 16) + ((q + 1) >> 1) * 32, r[(q + 1) & 1]);
                            else
                                release();
                            const int h = q & 1, k = q >> 1;
                            promote_scaled(r[h], f[2 * h], f[2 * h + 1], c, acc + 16 * h + 4 * k,
                                           acc + 16 * h + 8 + 4 * k);
                            if (q == 1) {
#pragma unroll
                                for (int g = 0; g < 4; ++g) c[g] = lds2(cs + 128 + 32 * g);
                            }
                        }
                    } else {
                        // 32 at a time, the other warps' products over the loads (16 in flight
                        // over 16 as above 235 against 182 us, 8192 x 4096 x 6144)
                        const uint64_t ff = f32x2_pack(f[0], f[0]);
                        uint32_t r[32];
#pragma unroll
                        for (int q = 0; q < EPI_COLS / 32; ++q) {
                            tmem_fetch32(p + 32 * q, r);
                            tmem_arrived(r);
                            if (q == EPI_COLS / 32 - 1) release();
                            promote<32>(r, ff, acc + 16 * q);
                        }
                    }
                    ++done;
                }
                __syncwarp();
                if (ok && elect_one()) arrive(sm.sempty(ch.slot));
            }
            if (!ok) {
                if (lane == 0) fail(sm, a.status);
                break;
            }
            if constexpr (SPLIT) {  // the only tile
                leave_tile<MODE>(sm, quad, part, lane, acc);
                break;
            }
            // decoded again rather than kept: the loop has no registers to spare
            const PTile t = work.tile(a, sm.tt, i);
            const int cols = MODE == kForward ? a.N : a.K;
            const int col = t.col0 + part * EPI_COLS;
            if (col < cols && !(MODE == kWeight && a.accumulate && t.blocks == 0)) {
                const int64_t row0 = MODE == kWeight ? (int64_t)t.g * a.N + t.row0 : t.row0;
                if constexpr (MODE == kWeight)
                    send_tile(a, &tm_out, sm.out + warp * OUT_WARP, row0 + quad * 32, col, acc);
                else
                    store_tile(a, row0 + quad * 32, t.nrows - quad * 32, cols, col, acc);
            }
            __syncwarp();
        }
        if (MODE == kWeight && !SPLIT && lane == 0) bulk_wait<0>();  // the output has left
        if constexpr (SPLIT) {
            __syncwarp();
            cluster_sync();  // every CTA's tile is in its shared memory
            // one share missing: the tile stays as it was, in every CTA's rows
            if (!__any_sync(0xffffffffu, lane < a.split && share_failed(sm, lane))) {
                const PTile t = work.tile(a, sm.tt, work.first);
                switch (a.split) {
                    case 2: add_tiles<MODE, 2>(a, sm, t, warp, lane); break;
                    case 4: add_tiles<MODE, 4>(a, sm, t, warp, lane); break;
                    default: add_tiles<MODE, 8>(a, sm, t, warp, lane); break;
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    if (SPLIT) {
        cluster_sync();  // no CTA leaves while another may read its tile
    } else {
        __syncthreads();
    }
    if (warp == MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Once per device: the register split has to add up in the kernels as compiled, their
// shared memory is opted into, and how many clusters of 2, 4 and 8 CTAs the device holds
// at once is asked (the GPCs' SM counts leave some idle).
struct DeviceSetup {
    std::mutex lock;
    std::atomic<bool> ready{false};
    int clusters[4] = {0, 0, 0, 0};
};

template <Mode MODE, bool SPLIT>
cudaError_t opt_in() {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, k_product<MODE, SPLIT>);
    if (e != cudaSuccess) return e;
    if (at.numRegs != REGS) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(k_product<MODE, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<MODE>());
}

void split_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int size, int clusters, size_t smem,
                  cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)size, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    *cfg = cudaLaunchConfig_t{};
    cfg->gridDim = dim3((unsigned)(clusters * size));
    cfg->blockDim = dim3(THREADS);
    cfg->dynamicSmemBytes = smem;
    cfg->stream = s;
    cfg->attrs = attr;
    cfg->numAttrs = 2;
}

template <Mode MODE>
cudaError_t set_up(DeviceSetup* d) {
    std::lock_guard<std::mutex> hold(d->lock);
    if (d->ready.load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = opt_in<MODE, false>();
    if (e == cudaSuccess) e = opt_in<MODE, true>();
    for (int i = 1; e == cudaSuccess && i < 4; ++i) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg;
        split_config(&cfg, attr, 1 << i, 1, smem_bytes<MODE>(), nullptr);
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&d->clusters[i], k_product<MODE, true>, &cfg);
    }
    if (e == cudaSuccess) d->ready.store(true, std::memory_order_release);
    return e;
}

template <Mode MODE>
cudaError_t launch_tiles(Fp8ProductArgs a, cudaStream_t s) {
    CUtensorMap ta, tb, tout;
    bool ok;
    if (MODE == kForward) {
        ok = make_tmap_2d(&ta, a.a, 1, a.M, a.K, BM, BK) &&
             make_tmap_2d(&tb, a.b, 1, (uint64_t)a.G * a.N, a.K, BN, BK);
    } else if (MODE == kInput) {
        ok = make_tmap_2d(&ta, a.a, 1, a.M, a.N, BM, BK) &&
             make_tmap_2d(&tb, a.b, 1, (uint64_t)a.G * a.N, a.K, BK, 128);
    } else {
        ok = make_tmap_2d(&ta, a.a, 1, a.N, a.rows_t, BM, BK) &&
             make_tmap_2d(&tb, a.b, 1, a.K, a.rows_t, BN, BK);
    }
    if (MODE == kWeight)
        ok = ok && make_tmap_2d(&tout, a.out, 4, (uint64_t)a.G * a.N, a.K, 8, 32);
    else
        tout = ta;  // not used
    if (!ok) return cudaErrorInvalidValue;
    // the groups' rows are known on the device only: there at most this many tiles
    const bool known = MODE == kWeight || a.offsets == nullptr;
    const int groups = a.G < a.M ? a.G : a.M;
    const int64_t tiles =
        MODE == kWeight ? (int64_t)a.G * (a.N / BM) * ((a.K + BN - 1) / BN)
                        : (known ? ((int64_t)a.M + BM - 1) / BM : (int64_t)a.M / BM + groups) *
                              (((MODE == kForward ? a.N : a.K) + BN - 1) / BN);
    if (tiles >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    static DeviceSetup setups[64];
    const DevInfo& dev = current_device_info();
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    DeviceSetup& d = setups[dev.device];
    cudaError_t e;
    if (!d.ready.load(std::memory_order_acquire) && (e = set_up<MODE>(&d)) != cudaSuccess) return e;

    // Few tiles and a long sum: as many CTAs a tile as find room.  Measured, one CTA
    // against the split: weight gradients of 1024 x 1024 (32 tiles, four CTAs each) over
    // 2048 rows 14.7 against 16.6 us, 4096 rows 24.7 against 18.3, 16384 rows 80.8
    // against 33.0; products of 1024 rows by 2048 columns (64 tiles, two each) with K =
    // 4096 19.2 against 19.6 us, 6144 26.1 against 24.1, 8192 33.2 against 28.4.  (A
    // launch of its own for the last wave's tiles, split so, gained 2% at 64 blocks
    // and lost 4% at 32.)
    const int64_t blocks = MODE == kWeight ? a.rows_t / BK / groups : (MODE == kForward ? a.K : a.N) / BK;
    int lg = 0;
    while (known && blocks >= (MODE == kWeight ? 32 : 48) && lg < 3 && tiles <= d.clusters[lg + 1]) ++lg;
    if (lg > 0) {
        a.split = 1 << lg;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg;
        split_config(&cfg, attr, a.split, (int)tiles, smem_bytes<MODE>(), s);
        e = cudaLaunchKernelEx(&cfg, k_product<MODE, true>, ta, tb, tout, a);
    } else {
        e = launch_pdl(k_product<MODE, false>, dim3((unsigned)(tiles < dev.num_sms ? tiles : dev.num_sms)),
                       dim3(THREADS), smem_bytes<MODE>(), s, ta, tb, tout, a);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Token-block quantisation, transposed: x [M][cols] bf16 -> q_t [cols][rows_t],
// scale_t [rows_t/128][cols].  Each group's rows start a new block of 128
// (padded with zeros), so a column's 128 tokens of one block share one scale
// and the weight gradient reads both operands along the tokens.  A block of
// threads takes 128 tokens x 64 columns: 16-byte loads, the column maxima by
// shuffles and shared memory, and the codes turned in shared memory so that
// each column's 128 codes leave as one 128-byte run.  2 bytes are read and 1
// written per value: 8192 x 6144 values take 31.5 us (4.8 TB/s; 47 us with an
// IEEE division per value, which bound it), in 32 ragged groups 45.4.  Eight blocks an
// SM, in 32 registers with spills, took 30.5 and 41.9 us there, but 5.6 for 5.0 us with
// 3001 x 1408: not taken.
// ---------------------------------------------------------------------------
constexpr int QC = 64;

__global__ void __launch_bounds__(256)
    k_quant_tokens(const uint16_t* __restrict__ x, const int32_t* __restrict__ offsets, int G, int M,
                   int cols, int64_t rows_t, uint8_t* __restrict__ q, float* __restrict__ scale) {
    __shared__ int2 s_rows;
    __shared__ __align__(16) uint32_t red[8][QC / 2];  // read and written 16 bytes at a time
    __shared__ __align__(16) float2 quot[QC];
    __shared__ uint32_t codes[QC][33];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    const int blk = blockIdx.y;
    int64_t row0 = (int64_t)blk * 128, end = M;  // one group: its rows in order
    if (offsets != nullptr) {
        if (warp == 0) {
            int first = 0, last = -1;
            if (!locate_block(offsets, G, M, blk, &first, &last)) last = -1;
            if (lane == 0) s_rows = make_int2(first, last);
        }
        __syncthreads();
        row0 = s_rows.x;
        end = s_rows.y;
        if (end < 0) return;
    }
    const int rows = (int)min((int64_t)128, end - row0);
    // a thread: four tokens of eight columns, a word holding two columns
    const int c0 = blockIdx.x * QC, c8 = (tid & 7) * 8, r4 = (tid >> 3) * 4;
    uint32_t w[4][4], m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (r4 + i < rows)
            u = __ldg(reinterpret_cast<const uint4*>(x + (row0 + r4 + i) * cols + c0 + c8));
        w[i][0] = u.x;
        w[i][1] = u.y;
        w[i][2] = u.z;
        w[i][3] = u.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        m[j] = bf16x2_absmax4(w[0][j], w[1][j], w[2][j], w[3][j]);
        m[j] = bf16x2_max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 8));
        m[j] = bf16x2_max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
    }
    if (lane < 8) *reinterpret_cast<uint4*>(&red[warp][c8 / 2]) = make_uint4(m[0], m[1], m[2], m[3]);
    __syncthreads();
    if (tid < QC) {
        uint32_t a = red[0][tid / 2];
#pragma unroll
        for (int v = 1; v < 8; ++v) a = bf16x2_max(a, red[v][tid / 2]);
        const GroupQuotient q8(block_scale(__uint_as_float((tid & 1) ? a & 0xFFFF0000u : a << 16)));
        scale[(int64_t)blk * cols + c0 + tid] = q8.s;
        quot[tid] = make_float2(q8.s, q8.r);
    }
    __syncthreads();
    if (warp * 16 < rows) {  // (without this rule the ragged groups above took 47.5 us)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // the two columns of word j, four tokens each: the words' low and high halves
            const uint32_t a = w[0][j], b = w[1][j], c = w[2][j], d = w[3][j];
            const float4 t = *reinterpret_cast<const float4*>(&quot[c8 + 2 * j]);
            codes[c8 + 2 * j][tid >> 3] = GroupQuotient(t.x, t.y).codes4(
                f32x2_pack(__uint_as_float(a << 16), __uint_as_float(b << 16)),
                f32x2_pack(__uint_as_float(c << 16), __uint_as_float(d << 16)));
            codes[c8 + 2 * j + 1][tid >> 3] = GroupQuotient(t.z, t.w).codes4(
                f32x2_pack(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u)),
                f32x2_pack(__uint_as_float(c & 0xFFFF0000u), __uint_as_float(d & 0xFFFF0000u)));
        }
    } else {  // none of the warp's tokens
#pragma unroll
        for (int j = 0; j < 8; ++j) codes[c8 + j][tid >> 3] = 0;
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
    return use_few_rows(a, a.N, current_device_info().num_sms) ? launch_gemm_fp8_few(a, s)
                                                               : launch_tiles<kForward>(a, s);
}

cudaError_t launch_gemm_fp8_dgrad(const Fp8ProductArgs& a, cudaStream_t s) {
    return use_few_rows(a, a.K, current_device_info().num_sms) ? launch_gemm_fp8_dgrad_few(a, s)
                                                               : launch_tiles<kInput>(a, s);
}

cudaError_t launch_gemm_fp8_wgrad(const Fp8ProductArgs& a, cudaStream_t s) {
    return launch_tiles<kWeight>(a, s);
}

}  // namespace moe
