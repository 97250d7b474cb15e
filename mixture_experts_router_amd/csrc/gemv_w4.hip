// Matrix-vector products with 4-bit weights and group scales for up to 16
// tokens (moe_gemv_w4): y[t][n] = sum_k x[t][k] W[n][k], W in MXFP4, NVFP4 or
// INT4 codes, with a bias and a GEGLU in the epilogue.
//
// A weight is read once and multiplied with every token (few_stream.h), so
// the weight bytes bound the product.  A workgroup keeps the token rows of its
// K range in LDS in MFMA order and runs through a range of 16-row units, its
// waves splitting K; sums are fp32 and rounded once.  Where the token rows of
// the whole K exceed the LDS, or the units are too few to fill the GPU, several
// workgroups share a range along K: each stores its fp32 sums, and the last to
// finish adds them in K order, whichever it is.
//
// INT4: W = scale (code - zero) with one scale and zero per group of 32, 64 or
// 128 K values.  The matrix cores multiply the exact values 16 + code, one
// group at a time, and each group's fp32 sum is corrected by the group's token
// sum: y += scale (sum_k (16 + code) x - (16 + zero) sum_k x).
#include <algorithm>

#include "few_stream.h"
#include "moe_launch.h"

namespace moe {

namespace {

constexpr int kGemvWaves = 8, kGemvThreads = 64 * kGemvWaves;
constexpr int kGemvXBytes = 128 * 1024;
constexpr int kGemvBlocks = 256;    // a workgroup per CU

struct GemvArgs {
    const uint16_t *x;
    const uint8_t *w, *scales, *zeros;
    const float *global;      // NVFP4 matrix scale
    const float *bias;
    void *y;
    float *part;              // [unit][slice][T][16] sums where slices > 1
    uint32_t *ctr;            // one counter per range of units, zero between calls
    long long ldx, ldy;
    int T, N, K;
    int outs, units;          // y columns; units of 16 weight rows
    int ranges, slices;       // workgroups: ranges x slices
    int geglu, y_fp32;
};

struct GemvSmem {
    uint8_t x[kGemvXBytes];
    float xsum[kGemvXBytes / 2 / 32];          // INT4: token sums [group][token]
    f32x4 red[2][kGemvWaves][64];
    int last;
};
static_assert(sizeof(GemvSmem) <= 160 * 1024, "LDS of one workgroup");

// Weight row of the MFMA's row m in unit u, clamped to a row that exists (the
// results of the others are not stored).
__device__ __forceinline__ int gemv_row(const GemvArgs &p, int u, int m) {
    if (p.geglu) {
        const int c = min(8 * u + (m & 7), p.outs - 1);
        return m < 8 ? c : p.outs + c;
    }
    return min(16 * u + m, p.N - 1);
}

// The epilogue of one value per thread: sums of weight row m of unit u and
// token t (all 64 lanes of a wave call it; m = lane % 16).
template <int F>
__device__ __forceinline__ void gemv_store(const GemvArgs &p, int u, int m, int t, float sum) {
    const int n = gemv_row(p, u, m);
    if constexpr (F == kFewNv) sum *= *p.global;
    if (p.bias) sum += *MOE_CHECKED(p.bias + n, 4, p.bias, (size_t)p.N * 4);
    int col = 16 * u + m;
    bool on = t < p.T && col < p.outs;
    if (p.geglu) {
        const float up = __shfl_down(sum, 8);
        col = 8 * u + m;
        on = t < p.T && m < 8 && col < p.outs;
        sum = gelu_tanh(sum) * up;
    }
    if (!on) return;
    const long long at = t * p.ldy + col;
    [[maybe_unused]] const size_t vals = (size_t)((p.T - 1) * p.ldy + p.outs);
    if (p.y_fp32) *MOE_CHECKED(static_cast<float *>(p.y) + at, 4, p.y, vals * 4) = sum;
    else *MOE_CHECKED(static_cast<uint16_t *>(p.y) + at, 2, p.y, vals * 2) = (uint16_t)f32_to_bf16_rne(sum);
}

template <int F, int GROUP>
__global__ __launch_bounds__(kGemvThreads) void gemv_w4_kernel(GemvArgs p) {
    __shared__ GemvSmem sm;
    constexpr int STEPS = FewBlock<F>::STEPS;
    const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
    const int range = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    const int nb = few_blocks(F, p.K);
    const int s0 = (int)((long long)slice * nb / p.slices), s1 = (int)((long long)(slice + 1) * nb / p.slices);
    const int u0 = (int)((long long)range * p.units / p.ranges), u1 = (int)((long long)(range + 1) * p.units / p.ranges);
    const int T = p.T, K = p.K, tr = min(r, T - 1);
    [[maybe_unused]] const size_t xbytes = (size_t)((T - 1) * p.ldx + K) * 2;

    // token rows of this K range, zero past K
    for (int i = threadIdx.x; i < (s1 - s0) * STEPS * 4 * T; i += kGemvThreads) {
        const int t = i % T, fg = i / T, k = few_frag_k<F>(s0 * STEPS + (fg >> 2), fg & 3);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (k < K) v = *reinterpret_cast<const u32x4 *>(MOE_CHECKED(p.x + t * p.ldx + k, 16, p.x, xbytes));
        *reinterpret_cast<u32x4 *>(sm.x + (size_t)i * 16) = F == kFewI4 ? few_i4_order(v) : v;
    }
    __syncthreads();
    if constexpr (F == kFewI4) {
        const int per = GROUP / 8;   // 16-byte pieces of one group and token, at stride 16 T
        for (int i = threadIdx.x; i < (s1 - s0) * (128 / GROUP) * T; i += kGemvThreads) {
            const int t = i % T, grp = i / T;
            float s = 0.f;
            for (int j = 0; j < per; ++j) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(sm.x + ((size_t)(grp * per + j) * T + t) * 16);
#pragma unroll
                for (int q = 0; q < 4; ++q) s += bf16_to_f32(v[q] & 0xFFFFu) + bf16_to_f32(v[q] >> 16);
            }
            sm.xsum[i] = s;
        }
        __syncthreads();
    }

    const int b0 = s0 + wave * (s1 - s0) / kGemvWaves, b1 = s0 + (wave + 1) * (s1 - s0) / kGemvWaves;
    const size_t pitch = (size_t)K / 2, spitch = F == kFewI4 ? K / (GROUP ? GROUP : 1) : (F == kFewMx ? K / 32 : K / 16);
    [[maybe_unused]] const size_t wbytes = (size_t)p.N * pitch, sbytes = (size_t)p.N * spitch;
    for (int u = u0; u < u1; ++u) {
        const uint8_t *wrow = p.w + gemv_row(p, u, r) * pitch;
        const uint8_t *srow = F == kFewI4 ? nullptr : p.scales + gemv_row(p, u, r) * spitch;
        size_t grow[4];   // INT4: first group of the four weight rows whose sums this lane holds
#pragma unroll
        for (int q = 0; q < 4; ++q) grow[q] = gemv_row(p, u, 4 * g + q) * spitch;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int b = b0; b < b1; ++b) {
            u32x4 c = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4 *>(MOE_CHECKED(wrow + few_piece<F>(b, g, K), 16, p.w, wbytes)));
            if constexpr (F == kFewI4) {
                few_transpose(c);
                f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int f = b * STEPS + i, fl = f - s0 * STEPS;
                    part = mfma16x16x32(few_i4_operand(c[i]),
                                        *reinterpret_cast<const u32x4 *>(sm.x + ((size_t)(fl * 4 + g) * T + tr) * 16), part);
                    if ((i + 1) * 32 % GROUP) continue;
                    if (32 * f < K) {
                        const float xs = sm.xsum[fl * 32 / GROUP * T + tr];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const size_t at = grow[q] + 32 * f / GROUP;
                            const float s = bf16_to_f32(*reinterpret_cast<const uint16_t *>(
                                MOE_CHECKED(p.scales + 2 * at, 2, p.scales, sbytes * 2)));
                            const float z = p.zeros ? (float)*MOE_CHECKED(p.zeros + at, 1, p.zeros, sbytes) : 8.f;
                            acc[q] = fmaf(s, fmaf(-(16.f + z), xs, part[q]), acc[q]);
                        }
                    }
                    part = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            } else {
                const uint32_t sc = few_scale<F>(srow, b, g, K, p.scales, sbytes);
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int fl = (b - s0) * STEPS + i;
                    acc = mfma16x16x32(few_operand<F>(c, sc, i),
                                       *reinterpret_cast<const u32x4 *>(sm.x + ((size_t)(fl * 4 + g) * T + tr) * 16), acc);
                }
            }
        }
        f32x4(*red)[64] = sm.red[u & 1];
        red[wave][lane] = acc;
        __syncthreads();
        // lane 16 (m / 4) + t, element m % 4 of each wave's sums: weight row m, token t
        if (threadIdx.x < 256) {
            const int m = threadIdx.x & 15, t = threadIdx.x >> 4;
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < kGemvWaves; ++v) sum += red[v][16 * (m >> 2) + t][m & 3];
            if (p.slices == 1)
                gemv_store<F>(p, u, m, t, sum);
            else if (t < T)
                *MOE_CHECKED(p.part + (((size_t)u * p.slices + slice) * T + t) * 16 + m, 4, p.part,
                             (size_t)p.units * p.slices * T * 64) = sum;
        }
    }
    if (p.slices == 1) return;
    // the last workgroup of the range adds the slices (their stores complete
    // and device-visible before each counts itself done)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const bool last = atomicInc(p.ctr + range, p.slices - 1) == (uint32_t)p.slices - 1;
        if (last) __threadfence();
        sm.last = last;
    }
    __syncthreads();
    if (!sm.last || threadIdx.x >= 256) return;
    const int m = threadIdx.x & 15, t = threadIdx.x >> 4;
    for (int u = u0; u < u1; ++u) {
        float sum = 0.f;
        for (int s = 0; t < T && s < p.slices; ++s)
            sum += *MOE_CHECKED(p.part + (((size_t)u * p.slices + s) * T + t) * 16 + m, 4, p.part,
                                (size_t)p.units * p.slices * T * 64);
        gemv_store<F>(p, u, m, t, sum);
    }
}

}  // namespace

// Workgroups of a product: `ranges` of units times `slices` of K.  The slices
// are as many as the token rows need to fit the LDS.
GemvPlan gemv_plan(int T, int N, int K, bool geglu) {
    GemvPlan g;
    g.outs = geglu ? N / 2 : N;
    g.units = geglu ? (g.outs + 7) / 8 : (N - 1) / 16 + 1;
    const int blocks = (K - 1) / 128 + 1, fit = kGemvXBytes / (256 * T);
    g.slices = (blocks + fit - 1) / fit;
    g.ranges = std::min(g.units, std::max(1, kGemvBlocks / g.slices));
    return g;
}

size_t gemv_part_bytes(const GemvPlan &g, int T) {
    return g.slices > 1 ? (size_t)g.units * g.slices * T * 64 : 0;
}

hipError_t launch_gemv_w4(const GemvW4 &l, hipStream_t st) {
    const GemvPlan g = gemv_plan(l.T, l.N, l.K, l.geglu);
    GemvArgs p{};
    p.x = l.x;
    p.w = l.w;
    p.scales = l.scales;
    p.zeros = l.zeros;
    p.global = l.global;
    p.bias = l.bias;
    p.y = l.y;
    p.part = l.part;
    p.ctr = l.counters;
    p.ldx = l.ldx;
    p.ldy = l.ldy;
    p.T = l.T;
    p.N = l.N;
    p.K = l.K;
    p.outs = g.outs;
    p.units = g.units;
    p.ranges = g.ranges;
    p.slices = g.slices;
    p.geglu = l.geglu;
    p.y_fp32 = l.y_fp32;
    const dim3 grid(g.ranges * g.slices), block(kGemvThreads);
    if (l.fmt == GemvFormat::kMXFP4) gemv_w4_kernel<kFewMx, 0><<<grid, block, 0, st>>>(p);
    else if (l.fmt == GemvFormat::kNVFP4) gemv_w4_kernel<kFewNv, 0><<<grid, block, 0, st>>>(p);
    else if (l.group == 32) gemv_w4_kernel<kFewI4, 32><<<grid, block, 0, st>>>(p);
    else if (l.group == 64) gemv_w4_kernel<kFewI4, 64><<<grid, block, 0, st>>>(p);
    else gemv_w4_kernel<kFewI4, 128><<<grid, block, 0, st>>>(p);
    return hipGetLastError();
}

#ifdef MOE_DEBUG
MOE_DEBUG_READER(debug_read_gemv)
#endif

}  // namespace moe
