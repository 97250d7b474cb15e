// Matrix-vector products with 4-bit weights and group scales for up to 16
// tokens (moe_gemv_w4): y[t][n] = sum_k x[t][k] W[n][k], W in MXFP4, NVFP4 or
// INT4 codes, with a bias and a GEGLU in the epilogue.
//
// A weight is read once and multiplied with every token (few_stream.h), so
// the weight bytes bound the product.  A workgroup keeps the token rows of its
// K range in LDS in MFMA order and runs through a range of 16-row units; a
// unit's K is split over as many of its waves as the range leaves free.  Sums
// are fp32 and rounded once.  Where the token rows of the whole K exceed the
// LDS, several workgroups share a range along K: each stores its fp32 sums,
// and the last to finish adds them in K order, whichever it is.
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
constexpr int kGemvArea = 150 * 1024;   // LDS for the rings, the token rows and (INT4) their sums
constexpr int kGemvBlocks = 256;        // a workgroup per CU

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
    alignas(1024) uint8_t area[kGemvArea];
    f32x4 red[kGemvWaves][64];
    int last;
};
static_assert(sizeof(GemvSmem) <= 160 * 1024, "LDS of one workgroup");

// A ring slot of the formats here: the step's codes, then its scales (and
// zeros): aligned words that hold the wanted bytes, 64 to a load.  INT4 loads
// the words of (row l % 16, group l / 16 + 4 i).
template <int F, int GROUP, bool ZEROS>
struct GemvSlot {
    static constexpr int NS = F == kFewI4 ? (GROUP == 32 ? 2 : 1) : 0;
    static constexpr int SLOT = FewStep<F, true>::SLOT + 256 * NS * (ZEROS ? 2 : 1);
    static constexpr int OPS = FewStep<F, true>::OPS + NS * (ZEROS ? 2 : 1);
};

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

// S: steps in each wave's ring.
template <int F, int GROUP, bool ZEROS, int S>
__global__ __launch_bounds__(kGemvThreads) void gemv_w4_kernel(GemvArgs p) {
    __shared__ GemvSmem sm;
    using G = GemvSlot<F, GROUP, ZEROS>;
    constexpr int SLOT = G::SLOT, OPS = G::OPS, FRAGS = FewStep<F>::FRAGS;
    const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
    const int range = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    const int nst = few_steps(F, p.K);
    const int c0 = (int)((long long)slice * nst / p.slices), c1 = (int)((long long)(slice + 1) * nst / p.slices);
    const int u0 = (int)((long long)range * p.units / p.ranges), u1 = (int)((long long)(range + 1) * p.units / p.ranges);
    const int T = p.T, K = p.K, tr = min(r, T - 1);
    const int KW = few_kwaves(u1 - u0, c1 - c0), UG = kGemvWaves / KW, kw = wave % KW;
    const int s0 = c0 + kw * (c1 - c0) / KW, s1 = c0 + (kw + 1) * (c1 - c0) / KW;
    const FewLane<F, true> ln(K);   // NVFP4 rows of 32 K values more or less
    uint8_t *ring = sm.area + wave * S * SLOT, *xs = sm.area + kGemvWaves * S * SLOT;
    const int nx = (c1 - c0) * FRAGS * 4 * T;   // 16-byte pieces of the token rows
    [[maybe_unused]] float *xsum = reinterpret_cast<float *>(xs + (size_t)nx * 16);
    [[maybe_unused]] const size_t xbytes = (size_t)((T - 1) * p.ldx + K) * 2;
    const size_t wn = (size_t)p.N * ln.pitch;
    [[maybe_unused]] const int pg = GROUP ? K / (GROUP ? GROUP : 1) : 0;   // groups of a row
    const size_t sn = (size_t)p.N * (F == kFewI4 ? 2 * pg : (int)ln.spitch);

    // the step to request next: of unit lu
    int lu = u0 + wave / KW, ls = s0, lslot = 0;
    FewRows rows;
    [[maybe_unused]] size_t lgroup = 0;         // INT4: first group of this lane's row (MFMA row lane % 16)
    auto point = [&]() {
        const int top = p.geglu ? 8 * lu : 16 * lu, low = p.geglu ? p.outs + top : min(top + 8, p.N - 1);
        const int ntop = min(7, (p.geglu ? p.outs : p.N) - 1 - top), nlow = p.geglu ? ntop : min(7, p.N - 1 - low);
        rows = ln.rows(p.w + (size_t)top * ln.pitch, p.w + (size_t)low * ln.pitch, p.scales + (size_t)top * ln.spitch,
                       p.scales + (size_t)low * ln.spitch, ntop, nlow);
        if constexpr (F == kFewI4) lgroup = (size_t)gemv_row(p, lu, r) * pg;
    };
    auto request = [&]() {
        uint8_t *q = ring + lslot * SLOT;
        ln.issue(rows, ls, q, p.w, wn, p.scales, sn);
        if constexpr (F == kFewI4) {
#pragma unroll
            for (int i = 0; i < G::NS; ++i) {
                const int j = ls * (256 / GROUP) + g + 4 * i;
                const size_t at = lgroup + (j < pg ? j : 0);
                dma4(MOE_CHECKED(p.scales + 2 * (at & ~(size_t)1), 4, p.scales, (sn + 3) & ~(size_t)3), q + 2048 + 256 * i);
                if constexpr (ZEROS)
                    dma4(MOE_CHECKED(p.zeros + (at & ~(size_t)3), 4, p.zeros, ((size_t)p.N * pg + 3) & ~(size_t)3),
                         q + 2048 + 256 * (G::NS + i));
            }
        }
        lslot = lslot + 1 == S ? 0 : lslot + 1;
        if (++ls == s1) {
            ls = s0;
            lu += UG;
            if (lu < u1) point();
        }
    };
    if (s0 == s1) lu = u1;   // more waves than steps
    if (lu < u1) {
        point();
        for (int i = 0; i < S && lu < u1; ++i) request();
    }

    // token rows of this K range, zero past K
    for (int i = threadIdx.x; i < nx; i += kGemvThreads) {
        const int t = i % T, fg = i / T, k = few_frag_k<F>(c0 * FRAGS + (fg >> 2), fg & 3);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (k < K) v = *reinterpret_cast<const u32x4 *>(MOE_CHECKED(p.x + t * p.ldx + k, 16, p.x, xbytes));
        *reinterpret_cast<u32x4 *>(xs + (size_t)i * 16) = F == kFewI4 ? few_i4_order(v) : v;
    }
    __syncthreads();
    if constexpr (F == kFewI4) {
        constexpr int per = GROUP / 8;   // 16-byte pieces of one group and token, at stride 16 T
        for (int i = threadIdx.x; i < nx / per; i += kGemvThreads) {
            const int t = i % T, grp = i / T;
            float s = 0.f;
            for (int j = 0; j < per; ++j) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(xs + ((size_t)(grp * per + j) * T + t) * 16);
#pragma unroll
                for (int q = 0; q < 4; ++q) s += bf16_to_f32(v[q] & 0xFFFFu) + bf16_to_f32(v[q] >> 16);
            }
            xsum[i] = s;
        }
        __syncthreads();
    }

    const uint8_t *xl = xs + (g * T + tr) * 16;   // this lane's piece of a token fragment
    int slot = 0;
    for (int v0 = u0; v0 < u1; v0 += UG) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        [[maybe_unused]] f32x4 half[2] = {acc, acc};   // of the two halves of every step
        const int u = v0 + wave / KW;
        if (uniform(u < u1)) {
            // where in its word a scale (zero) of this lane's rows lies: the low bits of its index
            [[maybe_unused]] uint32_t lo = 0, low4[4];
            if constexpr (F == kFewI4) {
#pragma unroll
                for (int q = 0; q < 4; ++q) low4[q] = (uint32_t)gemv_row(p, u, 4 * g + q) * (uint32_t)pg;
            } else {
                lo = (uint32_t)reinterpret_cast<uintptr_t>(p.scales) + (uint32_t)gemv_row(p, u, r) * ln.spitch;
            }
            for (int st = s0; st < s1; ++st) {
                const uint8_t *q = ring + slot * SLOT;
                if (lu < u1) few_wait<(S - 1) * OPS>();
                else few_wait<0>();
                const uint8_t *xq = xl + (size_t)(st - c0) * FRAGS * 64 * T;
                if constexpr (F == kFewI4) {
                    f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        u32x4 c = ln.load(q, h);
                        few_transpose(c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int f = 4 * h + i, j = f * 32 / GROUP;
                            part = mfma16x16x32(few_i4_operand(c[i]), *reinterpret_cast<const u32x4 *>(xq + f * 64 * T), part);
                            if ((i + 1) * 32 % GROUP) continue;
                            const int grp = st * (256 / GROUP) + j;
                            if (uniform(grp < pg)) {
                                const float xv = xsum[(grp - c0 * (256 / GROUP)) * T + tr];
                                const u32x4 sw = *reinterpret_cast<const u32x4 *>(q + 2048 + 4 * (16 * j + 4 * g));
                                u32x4 zw = {8u, 8u, 8u, 8u};
                                if constexpr (ZEROS)
                                    zw = *reinterpret_cast<const u32x4 *>(q + 2048 + 256 * G::NS + 4 * (16 * j + 4 * g));
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t at = low4[e] + grp;
                                    const float s = __uint_as_float(at & 1 ? sw[e] & 0xFFFF0000u : sw[e] << 16);
                                    const float z = ZEROS ? (float)((zw[e] >> (8 * (at & 3))) & 0xFFu) : 8.f;
                                    acc[e] = fmaf(s, fmaf(-(16.f + z), xv, part[e]), acc[e]);
                                }
                            }
                            part = f32x4{0.f, 0.f, 0.f, 0.f};
                        }
                    }
                    few_lds_done();
                    if (lu < u1) request();
                } else {
                    // everything of the step into registers at once, then its slot is free for another
                    const u32x4 c[2] = {ln.load(q, 0), ln.load(q, 1)};
                    const uint32_t sc[2] = {ln.scale(q, st, 0, lo), ln.scale(q, st, 1, lo)};
                    u32x4 xf[FRAGS];
#pragma unroll
                    for (int f = 0; f < FRAGS; ++f) xf[f] = *reinterpret_cast<const u32x4 *>(xq + f * 64 * T);
                    few_lds_done();
                    if (lu < u1) request();
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            half[h] = mfma16x16x32(few_operand<F>(c[h], sc[h], i), xf[4 * h + i], half[h]);
                }
                slot = slot + 1 == S ? 0 : slot + 1;
            }
        }
        if constexpr (F != kFewI4) acc = half[0] + half[1];
        sm.red[wave][lane] = acc;
        __syncthreads();
        // four waves finish a unit (lane 16 (m / 4) + t, element m % 4 of each wave's sums: weight row m, token t)
        for (int i = wave; i < 4 * UG; i += kGemvWaves) {
            const int unit = v0 + (i >> 2), m = lane & 15, t = 4 * (i & 3) + (lane >> 4);
            if (uniform(unit < u1 && 4 * (i & 3) < T)) {
                float sum = 0.f;
                for (int v = 0; v < KW; ++v) sum += sm.red[(i >> 2) * KW + v][16 * (m >> 2) + t][m & 3];
                if (p.slices == 1)
                    gemv_store<F>(p, unit, m, t, sum);
                else if (t < T)
                    *MOE_CHECKED(p.part + (((size_t)unit * p.slices + slice) * T + t) * 16 + m, 4, p.part,
                                 (size_t)p.units * p.slices * T * 64) = sum;
            }
        }
        __syncthreads();
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
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the invalidation is complete before the others load
        sm.last = last;
    }
    __syncthreads();
    if (!uniform(sm.last)) return;
    for (int i = wave; i < 4 * (u1 - u0); i += kGemvWaves) {
        const int unit = u0 + (i >> 2), m = lane & 15, t = 4 * (i & 3) + (lane >> 4);
        if (4 * (i & 3) >= T) continue;
        float sum = 0.f;
        for (int s = 0; t < T && s < p.slices; ++s)
            sum += *MOE_CHECKED(p.part + (((size_t)unit * p.slices + s) * T + t) * 16 + m, 4, p.part,
                                (size_t)p.units * p.slices * T * 64);
        gemv_store<F>(p, unit, m, t, sum);
    }
}

// Steps in a ring: the deep one where it leaves the token rows room, else the
// shallow one.
constexpr int kGemvDeep = 6, kGemvShallow = 3;

// LDS bytes that `steps` steps of token rows (and INT4's token sums) take.
size_t gemv_x_bytes(int T, int steps) { return (size_t)steps * 512 * T + (size_t)steps * 32 * T; }
size_t gemv_ring_bytes(int slot, int s) { return (size_t)kGemvWaves * s * slot; }

template <int F, int GROUP, bool ZEROS>
void launch_format(const GemvArgs &p, hipStream_t st) {
    constexpr int slot = GemvSlot<F, GROUP, ZEROS>::SLOT;
    const dim3 grid(p.ranges * p.slices), block(kGemvThreads);
    const int steps = (few_steps(F, p.K) + p.slices - 1) / p.slices;
    if (gemv_x_bytes(p.T, steps) + gemv_ring_bytes(slot, kGemvDeep) <= (size_t)kGemvArea)
        gemv_w4_kernel<F, GROUP, ZEROS, kGemvDeep><<<grid, block, 0, st>>>(p);
    else
        gemv_w4_kernel<F, GROUP, ZEROS, kGemvShallow><<<grid, block, 0, st>>>(p);
}

}  // namespace

// Workgroups of a product: `ranges` of units times `slices` of K, as many
// slices as the token rows need to fit the LDS next to the shallow ring.
GemvPlan gemv_plan(GemvFormat fmt, int group, bool zeros, int T, int N, int K, bool geglu) {
    GemvPlan g;
    g.outs = geglu ? N / 2 : N;
    g.units = geglu ? (g.outs + 7) / 8 : (N - 1) / 16 + 1;
    const int steps = (K - 1) / 256 + 1;
    const int words = fmt == GemvFormat::kINT4 ? (group == 32 ? 2 : 1) * (zeros ? 2 : 1) : fmt == GemvFormat::kNVFP4 ? 2 : 1;
    const int fit = (int)((kGemvArea - gemv_ring_bytes(2048 + 256 * words, kGemvShallow)) / gemv_x_bytes(T, 1));
    g.slices = (steps + fit - 1) / fit;
    g.ranges = std::min(g.units, std::max(1, kGemvBlocks / g.slices));
    return g;
}

size_t gemv_part_bytes(const GemvPlan &g, int T) {
    return g.slices > 1 ? (size_t)g.units * g.slices * T * 64 : 0;
}

hipError_t launch_gemv_w4(const GemvW4 &l, hipStream_t st) {
    const GemvPlan g = gemv_plan(l.fmt, l.group, l.zeros != nullptr, l.T, l.N, l.K, l.geglu);
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
    if (l.fmt == GemvFormat::kMXFP4) launch_format<kFewMx, 0, false>(p, st);
    else if (l.fmt == GemvFormat::kNVFP4) launch_format<kFewNv, 0, false>(p, st);
    else if (l.group == 32) l.zeros ? launch_format<kFewI4, 32, true>(p, st) : launch_format<kFewI4, 32, false>(p, st);
    else if (l.group == 64) l.zeros ? launch_format<kFewI4, 64, true>(p, st) : launch_format<kFewI4, 64, false>(p, st);
    else l.zeros ? launch_format<kFewI4, 128, true>(p, st) : launch_format<kFewI4, 128, false>(p, st);
    return hipGetLastError();
}

#ifdef MOE_DEBUG
MOE_DEBUG_READER(debug_read_gemv)
#endif

}  // namespace moe
