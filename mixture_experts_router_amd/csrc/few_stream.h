// Building blocks of the few-token kernels (the whole layer for up to 16
// tokens and the 4-bit matrix-vector product): up to 16 token rows are the
// columns of one 16x16x32 MFMA, sixteen weight rows its rows, so a weight
// value is loaded once and multiplied with every token.
//
// Each wave streams its own weights: steps of 16 rows x 128 bytes (whole cache
// lines; 64 K values of bf16, 256 of 4-bit codes) go straight from global
// memory into the slots of a ring in LDS that only this wave uses, so no
// barrier paces the stream and a few instructions, the same for every step,
// keep it running (an earlier form with the ring in registers, its turns
// unrolled, spent most of a one-token call fetching instructions).
//
// A step's MFMAs: lane (r, g) = (l % 16, l / 16) takes 16-byte pieces of row
// r.  bf16: pieces g and 4 + g, an MFMA each (K = 32 i + 8 g).  4-bit: pieces
// g and 4 + g hold the codes at K = 32 g and 128 + 32 g of the step.  MXFP4
// and NVFP4: MFMA i of a piece takes each lane's codes 8 i .. 8 i + 7 (K =
// 128 h + 32 g + 8 i), so a lane needs only its own scales; INT4: the four
// lanes of a row first exchange words so that MFMA i covers the 32 consecutive
// values at K = 128 h + 32 i, whose common scale is applied to the fp32 sums.
#pragma once

#include "moe_common.h"

namespace moe {

enum FewFmt { kFewBf16 = 0, kFewMx = 1, kFewNv = 2, kFewI4 = 3 };

constexpr int kFewTokens = 16;   // MFMA columns

// A value that is the same in all lanes, and known to be.  Every branch around
// an MFMA depends on such a value: MFMAs ignore the lane mask, so a branch
// that the compiler turned into a mask would not keep them from running.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int wave_index() { return uniform(threadIdx.x >> 6); }

template <int F>
struct FewStep {
    static constexpr int K = F == kFewBf16 ? 64 : 256;           // K values
    static constexpr int FRAGS = K / 32;                          // MFMAs
    // ring slot: 16 rows of 128 bytes, then (MXFP4, NVFP4) the lanes' scale words of the two pieces
    static constexpr bool SCALES = F == kFewMx || F == kFewNv;
    static constexpr int SLOT = 2048 + (SCALES ? 512 : 0);
    static constexpr int OPS = 2 + (SCALES ? 2 : 0);              // loads
    static constexpr int SB = F == kFewNv ? 2 : 1;                // scale bytes of a piece
    // Whole lines read once carry the non-temporal hint; 4-bit rows of a multiple of 32 bytes straddle lines,
    // whose other part the next step wants.
    static constexpr bool STREAM = F == kFewBf16;
};

__host__ __device__ constexpr int few_steps(int f, int K) { return f == kFewBf16 ? K / 64 : (K + 255) / 256; }

// K index of element 0 of B fragment (f, g): the token operand of MFMA f
// (counted from the start of the row), lane group g.
template <int F>
__device__ __forceinline__ int few_frag_k(int f, int g) {
    if constexpr (F == kFewBf16 || F == kFewI4) return 32 * f + 8 * g;
    else return 128 * (f >> 2) + 32 * g + 8 * (f & 3);
}

// INT4 codes become the bf16 pairs (k, k + 4): the token operand in that order.
__device__ __forceinline__ u32x4 few_i4_order(const u32x4 &v) {
    return u32x4{(v[0] & 0xFFFFu) | (v[2] << 16), (v[0] >> 16) | (v[2] & 0xFFFF0000u),
                 (v[1] & 0xFFFFu) | (v[3] << 16), (v[1] >> 16) | (v[3] & 0xFFFF0000u)};
}

// Addresses of a matrix's steps for one lane.  Sixteen rows are two blocks of
// eight consecutive rows (`top` and `low`); lane l loads 16 bytes of row l / 8
// of each, the piece swizzled so that the fragment reads have no bank
// conflicts.  A 4-bit row may end inside a step: pieces past its end read the
// row's first piece, whose codes then meet zero token values.
template <int F>
struct FewRows {
    const uint8_t *top, *low;      // weight rows
    const uint8_t *stop, *slow;    // scale rows
    int ntop = 7, nlow = 7;        // last row of each block that exists (the others repeat it)
};

template <int F>
struct FewLane {
    int pieces;                    // of a row
    uint32_t pitch, spitch;        // bytes of a row of weights, of scales
    uint32_t row, piece;           // loads: this lane's row of a block, its piece within a step
    uint32_t r, g;

    __device__ __forceinline__ explicit FewLane(int k) {
        const uint32_t l = threadIdx.x & 63;
        pitch = F == kFewBf16 ? 2 * k : k / 2;
        spitch = F == kFewMx ? k / 32 : k / 16;
        pieces = k / (F == kFewBf16 ? 8 : 32);
        row = l >> 3;
        piece = (l & 7) ^ row;
        r = l & 15;
        g = l >> 4;
    }
    // offset in its scale row of the scales of piece 4 h + g of step s; the row's first past its end
    __device__ __forceinline__ uint32_t scale_at(int s, int h) const {
        const int p = 8 * s + 4 * h + (int)g;
        return FewStep<F>::SB * (p < pieces ? p : 0);
    }
    // scale row of MFMA row r
    __device__ __forceinline__ const uint8_t *scale_row(const FewRows<F> &m) const {
        return r < 8 ? m.stop + min((int)r, m.ntop) * (size_t)spitch : m.slow + min((int)r - 8, m.nlow) * (size_t)spitch;
    }
    // Requests step s into `slot` (wave-uniform).  wb, wn / sb, sn: the extent of the matrices (debug build).
    __device__ __forceinline__ void issue(const FewRows<F> &m, int s, uint8_t *slot, [[maybe_unused]] const void *wb,
                                          [[maybe_unused]] size_t wn, [[maybe_unused]] const void *sb,
                                          [[maybe_unused]] size_t sn) const {
        const uint32_t off = F != kFewBf16 && 8 * s + (int)piece >= pieces ? 0u : 128 * s + 16 * piece;
        dma16<FewStep<F>::STREAM>(MOE_CHECKED(m.top + (min((int)row, m.ntop) * (size_t)pitch + off), 16, wb, wn), slot);
        dma16<FewStep<F>::STREAM>(MOE_CHECKED(m.low + (min((int)row, m.nlow) * (size_t)pitch + off), 16, wb, wn),
                                  slot + 1024);
        if constexpr (FewStep<F>::SCALES) {
            // the aligned word that holds this lane's one or two scale bytes
            const uint8_t *base = scale_row(m);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uintptr_t at = reinterpret_cast<uintptr_t>(base + scale_at(s, h));
                dma4(MOE_CHECKED(reinterpret_cast<const uint8_t *>(at & ~(uintptr_t)3), 4, sb, (sn + 3) & ~(size_t)3),
                     slot + 2048 + 256 * h);
            }
        }
    }
    // 16-byte piece 4 h + g of this lane's row in a slot whose loads are complete
    __device__ __forceinline__ u32x4 load(const uint8_t *slot, int h) const {
        return *reinterpret_cast<const u32x4 *>(slot + 128 * r + (((4 * h + g) ^ (r & 7)) << 4));
    }
    // its scales; lo: the address of its scale row modulo 4
    __device__ __forceinline__ uint32_t scale(const uint8_t *slot, int s, int h, uint32_t lo) const {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(slot + 2048 + 256 * h + 4 * (threadIdx.x & 63));
        return (w >> (8 * ((lo + scale_at(s, h)) & 3))) & (F == kFewMx ? 0xFFu : 0xFFFFu);
    }
};

// Waves along K of a unit of 16 rows, where `count` units of `steps` steps are
// shared by eight waves: as few as leave no wave longer at work (fewer waves
// to a unit, fewer sums to join).
__host__ __device__ __forceinline__ int few_kwaves(int count, int steps) {
    int best = 1, cost = ((count + 7) / 8) * steps;
    for (int kw = 2; kw <= 8; kw *= 2) {
        const int ug = 8 / kw, c = ((count + ug - 1) / ug) * ((steps + kw - 1) / kw);
        if (c < cost) {
            cost = c;
            best = kw;
        }
    }
    return best;
}

// Waits until at most N of this wave's loads are outstanding (and its LDS
// reads are done: a slot just read may be loaded again).
template <int N>
__device__ __forceinline__ void few_wait() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void few_lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// MFMA step s of a loaded piece (bf16, MXFP4, NVFP4): the weight operand.
template <int F>
__device__ __forceinline__ u32x4 few_operand(const u32x4 &c, uint32_t scale, int s) {
    if constexpr (F == kFewBf16) {
        return c;
    } else if constexpr (F == kFewMx) {
        const float f = __uint_as_float((scale & 0xFFu) << 23);   // 2^(byte - 127), a normal number for bytes 2..250
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[s], f, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[s], f, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[s], f, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[s], f, 3))};
    } else {
        return e2m1x8_times_scale(c[s], e4m3_to_f32(s < 2 ? scale & 0xFFu : scale >> 8));
    }
}

// Words of the four lanes of a row transposed: lane group g's word s becomes
// group s's word g, so word s of every lane then belongs to K block 32s.
// (Two exchange stages: permlane32_swap swaps the upper half of its first
// operand with the lower half of its second, permlane16_swap the odd rows of
// the first with the even rows of the second.)
__device__ __forceinline__ void few_transpose(u32x4 &c) {
    const auto a = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
    const auto p = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto q = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    c = u32x4{p[0], p[1], q[0], q[1]};
}

// Eight INT4 codes as bf16 values 16 + code: a code in bits 3..6 of the
// mantissa of 16.0 adds exactly its value.  (The offset, and the zero point,
// leave the fp32 sums with the scale; 16 rather than a larger power of two
// keeps that cancellation to about two bits.)
__device__ __forceinline__ u32x4 few_i4_operand(uint32_t w) {
    constexpr uint32_t mask = 0x00780078u, base = 0x41804180u;
    return u32x4{((w << 3) & mask) | base, ((w >> 1) & mask) | base, ((w >> 5) & mask) | base, ((w >> 9) & mask) | base};
}

}  // namespace moe
