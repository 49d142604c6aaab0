// fp8_block.cuh -- shared by the FP8 block-128 products and the token-block
// quantiser: the group table of a row matrix, and device helpers.
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

// One warp: the first row, and the end of its group, of block `blk` of the groups' rows
// in blocks of 128 (rows of the table above, without a table: a scan over the
// lanes' groups in registers); false past the last block.
__device__ __forceinline__ bool locate_block(const int32_t* __restrict__ offsets, int G, int M, int blk,
                                             int* row0, int* end) {
    const int lane = threadIdx.x & 31;
    const int per = (G + 31) / 32;
    const int g0 = min(G, lane * per), g1 = min(G, g0 + per);
    auto offset = [&](int g) { return min(M, max(0, __ldg(offsets + g))); };
    int top = 0;
    for (int g = g0; g < g1; ++g) top = max(top, offset(g));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = max(top, v);
    }
    int before = __shfl_up_sync(0xffffffffu, top, 1);
    if (lane == 0) before = 0;
    int sum = 0;
    for (int g = g0, at = before; g < g1; ++g) {
        at = max(at, offset(g));
        sum += (max(at, offset(g + 1)) - at + 127) / 128;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, incl > blk);
    if (past == 0) return false;
    int r = 0, e = 0, left = blk - (incl - sum);  // of the first lane past it
    for (int g = g0, at = before; g < g1; ++g) {
        at = max(at, offset(g));
        const int next = max(at, offset(g + 1)), n = (next - at + 127) / 128;
        if (left >= 0 && left < n) {
            r = at + left * 128;
            e = next;
        }
        left -= n;
    }
    const int owner = __ffs(past) - 1;
    *row0 = __shfl_sync(0xffffffffu, r, owner);
    *end = __shfl_sync(0xffffffffu, e, owner);
    return true;
}

// ---------------------------------------------------------------- device helpers
// Shared memory is addressed by 32-bit shared addresses: generic pointers cost
// the promotion loops registers that they do not have.
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
__device__ __forceinline__ uint64_t lds2(uint32_t a) {  // a pair for the packed products
    uint64_t v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(a));
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
// once in 64 tries only.
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

// Warp-collective: one outcome for the warp.  The first try stands apart from the
// bounded loop: most waits end with it.
__device__ __forceinline__ bool warp_wait_phase(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                                uint32_t abort_flag) {
    if (__all_sync(0xffffffffu, try_phase(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_phase(bar, parity, timeout_ns, abort_flag));
}

// True in one lane of a converged warp.  The single-thread roles run their loops
// with the whole warp and issue under this predicate: the operands then stay in
// uniform registers.  Measured: an MMA of N = 128 issued by `lane == 0` took 80
// cycles, issued so 64, the tensor core's own time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                         int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

// Shared-memory descriptor of an operand stored with its M (or N) index innermost
// and the 128-byte swizzle: each row of 128 bytes holds 128 of the index at one k,
// groups of eight k are 1024 bytes apart (stride field), the next 128 of the
// index `next` bytes on (leading field).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t next) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((next >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
// Instruction descriptor bits 15 and 16: A, B stored with M, N innermost.
constexpr uint32_t kATransposed = 1u << 15, kBTransposed = 1u << 16;

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
// 32 FP32 columns of 16 TMEM lanes, shared out over rows and columns: of the columns
// 8g .. 8g + 7, r[4g] and r[4g + 1] are columns 2 (l % 4) and the next of TMEM lane
// l / 4 (l: this thread's lane), r[4g + 2] and r[4g + 3] of TMEM lane l / 4 + 8.
__device__ __forceinline__ void tmem_fetch16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : W4(r, 0), W4(r, 4), W4(r, 8), W4(r, 12)
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_arrived16(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : R4(r, 0), R4(r, 4), R4(r, 8), R4(r, 12)
                 :
                 : "memory");
}
#undef R4
#undef W4

__device__ __forceinline__ bool aligned16(const void* p) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// ---------------------------------------------------------------- e4m3 codes of a group
// s = fp32(amax) / 448 (1 for a group of zeros, or of NaN only), rounded as the IEEE division: the
// product with 1/448 corrected by one FMA residual (Markstein's final correction of a
// quotient, 1990), which is the rounded quotient where nothing underflows or overflows on
// the way (every bf16 amax is tested), else the division.
__device__ __forceinline__ float block_scale(float amax) {
    constexpr float r = 1.0f / 448.0f;
    if (amax >= 0x1p-90f && amax <= 0x1p100f) {
        const float q = amax * r;
        return fmaf(fmaf(-448.0f, q, amax), r, q);
    }
    return amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
}

// Codes e4m3(fp32(v / s)) of bf16 values, rounded to nearest even and saturating,
// with the quotient of the IEEE division, without dividing: the product with the
// reciprocal, corrected by one FMA residual (Markstein's, as above), is the rounded quotient for
// every bf16 significand against the scale of every bf16 maximum, whichever way
// the reciprocal is rounded (1 ulp; all 3 * 128 * 128 cases are tested), as long
// as nothing underflows; below 2^-100 the code is a zero either way.  Scales near
// the ends of the FP32 range divide.  The quotient is taken negated, so that zeros
// keep their signs (-0 + 0 is +0, but -0 - 0 is -0): its codes have the sign bit
// turned; NaN has the code 0x7F whatever its sign.
// (Bracketing the quotient between two roundings and dividing where they differ
// was slower: bf16 values over a bf16 maximum meet exact ties in a group out of
// seven.  8192 x 6144 values: 38 us so, 41 with divisions, 30.6 with the
// correction, 25.2 with the rows' other instructions fewer too.)
struct GroupQuotient {
    float s, r;  // r = 0: divide
    __device__ __forceinline__ GroupQuotient(float scale, float reciprocal) : s(scale), r(reciprocal) {}
    __device__ __forceinline__ explicit GroupQuotient(float scale) : s(scale) {
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
        if (!(scale >= 0x1p-100f && scale <= 0x1p100f)) r = 0.0f;
    }
    // e4m3 codes of a pair, the first in the low byte
    static __device__ __forceinline__ uint32_t cvt(uint64_t p) {
        float a, b;
        f32x2_unpack(p, a, b);
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
        return c;
    }
    __device__ __forceinline__ uint64_t minus_quotient(uint64_t p) const {
        if (r == 0.0f) {
            float a, b;
            f32x2_unpack(p, a, b);
            return f32x2_pack(__fdiv_rn(-a, s), __fdiv_rn(-b, s));
        }
        const uint64_t mr = f32x2_pack(-r, -r), ss = f32x2_pack(s, s);
        const uint64_t q = f32x2_mul(p, mr);
        return f32x2_fma(f32x2_fma(q, ss, p), mr, q);
    }
    // codes of four values
    __device__ __forceinline__ uint32_t codes4(uint64_t p0, uint64_t p1) const {
        const uint32_t c = cvt(minus_quotient(p0)) | cvt(minus_quotient(p1)) << 16;
        const uint32_t nan = (c & 0x7F7F7F7Fu) + 0x01010101u;  // bit 7 of each byte
        return (c ^ 0x80808080u) & ~(nan & 0x80808080u);
    }
};

// The two bf16 values of a word, widened.
__device__ __forceinline__ uint64_t bf16x2_widen(uint32_t w) {
    return f32x2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// Packed bf16: magnitudes, and the larger of each (NaN gives way to a number, as
// with fmaxf).
__device__ __forceinline__ uint32_t bf16x2_abs(uint32_t a) { return a & 0x7FFF7FFFu; }
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}
__device__ __forceinline__ uint32_t bf16x2_absmax4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return bf16x2_max(bf16x2_max(bf16x2_abs(a), bf16x2_abs(b)), bf16x2_max(bf16x2_abs(c), bf16x2_abs(d)));
}

}  // namespace moe
