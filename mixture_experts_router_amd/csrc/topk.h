// Top-k selection and softmax weights of one token by one wave, shared by the
// routing kernels and the few-token layer.
#pragma once

#include "moe_common.h"

namespace moe {

// Order-preserving integer key of a float: larger float -> larger key.
// -0.0 is mapped to +0.0 so equal values tie.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Wave-wide maximum in every lane: DPP steps inside each row of 16 lanes
// (quad swaps, then the half-row and row mirrors), then the gfx950 lane swaps
// between the two halves and between neighbouring rows.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));    // quad [1,0,3,2]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));    // quad [2,3,0,1]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));   // row_half_mirror
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));   // row_mirror
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);   // lanes l and l ^ 32
    v = max(h[0], h[1]);
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);   // rows 0<->1, 2<->3
    return max(r[0], r[1]);
}

// The k largest of the keys held by a wave (lane l's key[i] is expert
// l + 64 i, 0 = none): lane j returns slot j's softmax weight over the k
// selected logits and sets my_idx to its expert.
template <int VPL>
__device__ __forceinline__ float topk_slots(uint32_t (&key)[VPL], int k, int &my_idx) {
    const int lane = threadIdx.x & 63;
    // k rounds of wave argmax; lane j keeps slot j.
    my_idx = 0;
    uint32_t my_key = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t lm = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) lm = max(lm, key[i]);
        const uint32_t km = wave_max_u32(lm);
        // the lowest expert index holding km: the lowest lane of the lowest
        // i with a hit (scalar selects, no branch per i)
        int sel = 0;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i) {
            const uint64_t hit = __ballot(key[i] == km);
            // (bit 63 keeps the count defined for an empty mask, whose
            // result is not selected, and changes no nonzero one)
            sel = hit ? 64 * i + (int)__builtin_ctzll(hit | (1ull << 63)) : sel;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (64 * i + lane == sel) key[i] = 0u;
        if (lane == j) {
            my_idx = sel;
            my_key = km;
        }
    }
    // weights: exp(l_j - l_0) in every slot lane at once, their sum in slot order
    const float top = key_value((uint32_t)__builtin_amdgcn_readfirstlane((int)my_key));
    const float ex = lane < k ? expf(key_value(my_key) - top) : 0.f;
    float sum = 0.f;
    for (int m = 0; m < k; ++m) sum += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ex), m));
    return ex / sum;
}

}  // namespace moe
