// Building blocks of the few-token kernels (the whole layer for up to 16
// tokens and the 4-bit matrix-vector product): up to 16 token rows are the
// columns of one 16x16x32 MFMA, sixteen weight rows its rows, so a weight
// value is loaded once, straight into the registers that feed the MFMA, and
// multiplied with every token.  What differs between the weight formats is
// how one 16-byte load per lane becomes MFMA operands:
//
//   bf16    16 rows x 32 K: lane (r, g) loads K values 8g .. 8g+7 of row r,
//           one MFMA.
//   4-bit   16 rows x 128 K: lane (r, g) loads the 32 codes at K = 32g of
//           row r, four MFMAs.  MXFP4 and NVFP4: MFMA s takes each lane's
//           codes 8s .. 8s+7 (K = 32g + 8s), so a lane needs only its own
//           scales; INT4: the four lanes of a row first exchange words so
//           that MFMA s covers the 32 consecutive values at K = 32s, whose
//           common scale is applied to the fp32 sums.
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
struct FewBlock {
    static constexpr int K = F == kFewBf16 ? 32 : 128;   // K values of one load
    static constexpr int STEPS = K / 32;                 // MFMAs of one load
};

__host__ __device__ constexpr int few_blocks(int f, int K) { return f == kFewBf16 ? K / 32 : (K + 127) / 128; }

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

// Byte offset in its weight row of lane group g's 16 bytes of block b;
// pieces past K (the last block of a 4-bit row) read the row's first bytes,
// which then meet zero token values.
template <int F>
__device__ __forceinline__ int few_piece(int b, int g, int K) {
    if constexpr (F == kFewBf16) return 64 * b + 16 * g;
    else return 128 * b + 32 * g < K ? 64 * b + 16 * g : 0;
}

// The scale bytes of that piece: one E8M0 byte (MXFP4) or two E4M3 bytes
// (NVFP4) of a row of scales.
template <int F>
__device__ __forceinline__ uint32_t few_scale(const uint8_t *row, int b, int g, int K, [[maybe_unused]] const void *base,
                                              [[maybe_unused]] size_t bytes) {
    const int i = 128 * b + 32 * g < K ? 4 * b + g : 0;
    if constexpr (F == kFewMx) return *MOE_CHECKED(row + i, 1, base, bytes);
    else if constexpr (F == kFewNv) return *reinterpret_cast<const uint16_t *>(MOE_CHECKED(row + 2 * i, 2, base, bytes));
    else return 0u;
}

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
