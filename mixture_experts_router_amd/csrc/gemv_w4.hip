// Matrix-vector products with 4-bit weights and group scales for up to 16
// tokens (moe_gemv_w4): y[t][n] = sum_k x[t][k] W[n][k], W in MXFP4, NVFP4 or
// INT4 codes, with a bias and a GEGLU in the epilogue.
//
// A weight is read once and multiplied with every token (few_stream.h), so
// the weight bytes bound the product.  A workgroup keeps the token rows of its
// K range in LDS in MFMA order (or windows of them, where they do not fit) and
// runs through a range of 16-row units.  Sums are fp32 and rounded once.  Where
// there are few units and a long K, several workgroups share a range along K:
// each stores its fp32 sums, and the last to finish adds them in K order,
// whichever it is.
//
// Measured: 1 token x 2112 -> 2816 in INT4 and x 2816 -> 2112 GEGLU in MXFP4 6.3
// us, which is the host's time for a call (7.5 and 5.8 on the GPU under the
// profiler); 8 tokens x 2816 -> 5001 INT4 9.2; 4 tokens x 8192 -> 8192 NVFP4
// 13.1 (37.9 MB: 2.9 TB/s), 10.8 without its arithmetic; 16 tokens x 2816 ->
// 131072 INT4 58 (205 MB: 3.5 TB/s).  The last is bound by its instructions,
// 160 vector and 17 matrix ones to a step of 16 x 256 weights, and by the three
// steps of a ring that 90 KB of token rows leave room for.
//
// INT4: W = scale (code - zero) with one scale and zero per group of 32, 64 or
// 128 K values.  The matrix cores multiply the exact values 16 + code, one
// group at a time: y = sum over groups of scale sum_k (16 + code) x
// - sum over groups of scale (16 + zero) sum_k x, the second of which is an
// fp32 matrix product over the groups.
#include <algorithm>
#include <type_traits>

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
    int y_wide;               // rows of y allow stores of four values
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

// The epilogue of unit u: lane 16 g + t has the sums of weight rows 4 g + q of
// the unit and token t.
template <int F>
__device__ __forceinline__ void gemv_store(const GemvArgs &p, int u, f32x4 sum) {
    const int t = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    if constexpr (F == kFewNv) sum *= *p.global;
    if (p.bias) {
        // uniform addresses in read-only memory, so scalar loads: a vector load would be waited for behind the
        // ring's, all of which would have to arrive
        const auto *bias = reinterpret_cast<const __attribute__((address_space(4))) float *>(
            reinterpret_cast<uintptr_t>(p.bias));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = bias[uniform(gemv_row(p, u, 4 * i + q))];
            sum[q] += g == 0 ? b[0] : g == 1 ? b[1] : g == 2 ? b[2] : b[3];
        }
    }
    int col = 16 * u + 4 * g;
    bool on = t < p.T;
    if (p.geglu) {
        // gate rows 0..7, up rows 8..15: a gate's up value is 32 lanes above
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t b = __float_as_uint(sum[q]);
            sum[q] = gelu_tanh(sum[q]) * __uint_as_float(__builtin_amdgcn_permlane32_swap(b, b, false, false)[1]);
        }
        col = 8 * u + 4 * g;
        on = on && g < 2;
    }
    if (!on) return;
    const long long at = t * p.ldy + col;
    [[maybe_unused]] const size_t vals = (size_t)((p.T - 1) * p.ldy + p.outs);
    if (p.y_fp32) {
        float *y = static_cast<float *>(p.y) + at;
        if (p.y_wide && col + 4 <= p.outs) {
            *reinterpret_cast<f32x4 *>(MOE_CHECKED(y, 16, p.y, vals * 4)) = sum;
        } else {
            for (int q = 0; q < 4 && col + q < p.outs; ++q) *MOE_CHECKED(y + q, 4, p.y, vals * 4) = sum[q];
        }
    } else {
        uint16_t *y = static_cast<uint16_t *>(p.y) + at;
        if (p.y_wide && col + 4 <= p.outs) {
            *reinterpret_cast<uint64_t *>(MOE_CHECKED(y, 8, p.y, vals * 2)) =
                pack_bf16x2(sum[0], sum[1]) | (uint64_t)pack_bf16x2(sum[2], sum[3]) << 32;
        } else {
            for (int q = 0; q < 4 && col + q < p.outs; ++q)
                *MOE_CHECKED(y + q, 2, p.y, vals * 2) = (uint16_t)f32_to_bf16_rne(sum[q]);
        }
    }
}

// The units of a product's range: sixteen weight rows (GEGLU: eight gate rows
// and the matching eight up rows), steps c0 .. c1 - 1 of them.
template <int F, int GROUP, bool ZEROS, int S_, int WINDOW_>
struct GemvUnits {
    static constexpr int WINDOW = WINDOW_;
    static constexpr int S = S_, SLOT = GemvSlot<F, GROUP, ZEROS>::SLOT, OPS = GemvSlot<F, GROUP, ZEROS>::OPS;
    static constexpr int NS = GemvSlot<F, GROUP, ZEROS>::NS, FRAGS = FewStep<F>::FRAGS;
    static constexpr bool I4 = F == kFewI4;
    static constexpr uint32_t kOnes = 0x3F803F80u;               // bf16
    static constexpr int NG = I4 ? 256 / (I4 ? GROUP : 1) : 1;   // groups of a step
    const GemvArgs &p;
    const FewLane<F, true> ln;       // NVFP4: K a multiple of 32
    const int slice, c0, c1;
    uint8_t *const xs;               // token rows, 16 bytes per fragment, lane group and token
    const int pg, tr;                // INT4: groups of a row; this lane's token

    struct Rows : FewRows {
        size_t group;                // INT4: first group of this lane's row (MFMA row lane % 16)
    };
    struct Operand {
        const uint8_t *x;
        uint32_t lo;                 // MXFP4, NVFP4: address of this lane's scale row modulo 4
        // INT4: byte selectors of the scales in their words, as fp32: of rows 4 g + q, even and odd groups, and of
        // the words this lane loads; bit offset of its zeros in theirs
        uint32_t even[4], odd[4], own, zero;
        FewI4 codes;
    };
    struct I4Data {
        u32x4 c[2], x[1][FRAGS], scale[NG];
        uint32_t own[NS + 1], zero[NS + 1];   // the words this lane loaded: of row lane % 16, group lane / 16 + 4 i
    };
    using Data = std::conditional_t<I4, I4Data, FewData<F>>;

    __device__ __forceinline__ GemvUnits(const GemvArgs &p, int slice, int c0, int c1, uint8_t *xs)
        : p(p), ln(p.K), slice(slice), c0(c0), c1(c1), xs(xs), pg(I4 ? p.K / (I4 ? GROUP : 1) : 0),
          tr(min((int)(threadIdx.x & 15), p.T - 1)) {}
    __device__ __forceinline__ int at(int, int) const { return 0; }
    __device__ __forceinline__ void span(int, int &a, int &b) const {
        a = c0;
        b = c1;
    }
    __device__ __forceinline__ Rows rows(int u, int) const {
        const int top = p.geglu ? 8 * u : 16 * u, low = p.geglu ? p.outs + top : min(top + 8, p.N - 1);
        const int ntop = min(7, (p.geglu ? p.outs : p.N) - 1 - top), nlow = p.geglu ? ntop : min(7, p.N - 1 - low);
        Rows m{ln.rows(p.w + (size_t)top * ln.pitch, p.w + (size_t)low * ln.pitch, p.scales + (size_t)top * ln.spitch,
                       p.scales + (size_t)low * ln.spitch, ntop, nlow), 0};
        if constexpr (I4) m.group = (size_t)gemv_row(p, u, ln.r) * pg;
        return m;
    }
    __device__ __forceinline__ void issue(const Rows &m, int, int st, uint8_t *slot) const {
        const size_t sn = (size_t)p.N * (I4 ? 2 * pg : (int)ln.spitch);
        ln.issue(m, st, slot, p.w, (size_t)p.N * ln.pitch, p.scales, sn);
        if constexpr (I4) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int j = st * NG + ln.g + 4 * i;
                // past the row: another scale of this row, of a group of the same parity if there is one
                const size_t at = m.group + (j < pg ? j : (j & 1) < pg ? j & 1 : 0);
                dma4(MOE_CHECKED(p.scales + 2 * (at & ~(size_t)1), 4, p.scales, (sn + 3) & ~(size_t)3), slot + 2048 + 256 * i);
                if constexpr (ZEROS)
                    dma4(MOE_CHECKED(p.zeros + (at & ~(size_t)3), 4, p.zeros, ((size_t)p.N * pg + 3) & ~(size_t)3),
                         slot + 2048 + 256 * (NS + i));
            }
        }
    }
    __device__ __forceinline__ Operand operand(int u, int) const {
        Operand o;
        o.x = xs + (ln.g * p.T + tr) * 16;
        if constexpr (I4) {
            constexpr uint32_t half[2] = {0x05040c0cu, 0x07060c0cu};   // of the word, in the upper half of an fp32
            // one group in a row: an odd one is past its end, and its word may hold another row's scale
            const uint32_t none = 0x0c0c0c0cu;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t at = (uint32_t)gemv_row(p, u, 4 * ln.g + q) * (uint32_t)pg;
                o.even[q] = half[at & 1];
                o.odd[q] = pg == 1 ? none : half[~at & 1];
            }
            const uint32_t at = (uint32_t)gemv_row(p, u, ln.r) * (uint32_t)pg + ln.g;
            o.own = pg == 1 && (ln.g & 1) ? none : half[at & 1];
            o.zero = 8 * at;
        } else {
            o.lo = (uint32_t)reinterpret_cast<uintptr_t>(p.scales) + (uint32_t)gemv_row(p, u, ln.r) * ln.spitch;
        }
        return o;
    }
    __device__ __forceinline__ Data fetch(const uint8_t *q, int st, int xst, const Operand &o) const {
        Data d;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            d.c[h] = ln.load(q, h);
            if constexpr (!I4) d.sc[h] = ln.scale(q, st, h, o.lo);
        }
        if constexpr (I4) {
#pragma unroll
            for (int j = 0; j < NG; ++j) d.scale[j] = *reinterpret_cast<const u32x4 *>(q + 2048 + 4 * (16 * j + 4 * ln.g));
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const uint32_t *own = reinterpret_cast<const uint32_t *>(q + 2048 + 256 * i + 4 * (threadIdx.x & 63));
                d.own[i] = own[0];
                if constexpr (ZEROS) d.zero[i] = own[64 * NS];
            }
        }
        const uint8_t *x = o.x + (size_t)(WINDOW ? xst : st - c0) * FRAGS * 64 * p.T;
#pragma unroll
        for (int f = 0; f < FRAGS; ++f) d.x[0][f] = *reinterpret_cast<const u32x4 *>(x + f * 64 * p.T);
        return d;
    }
    __device__ __forceinline__ void multiply(const Data &d, int st, const Operand &o, f32x4 (&acc)[2]) const {
        if constexpr (!I4) {
            few_multiply<F, 1>(d, acc);
        } else {
            // group by group: the sums of (16 + code) x, and of x (the ones' rows are alike)
            f32x4 part[NG], tokens[NG];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 c = d.c[h];
                few_transpose(c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int f = 4 * h + i, j = f * 32 / GROUP;
                    if (f * 32 % GROUP == 0) part[j] = tokens[j] = f32x4{0.f, 0.f, 0.f, 0.f};
                    part[j] = mfma16x16x32(o.codes.operand(c[i]), d.x[0][f], part[j]);
                    tokens[j] = mfma16x16x32(u32x4{kOnes, kOnes, kOnes, kOnes}, d.x[0][f], tokens[j]);
                }
            }
            // the groups' offsets, - scale (16 + zero) times the token sums, are an fp32 product over the groups: lane
            // (r, g) has row r's factor and token r's sum of group g.  (Past the row the tokens are zero and the
            // scales this row's, or zero.)
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const float s = __uint_as_float(__builtin_amdgcn_perm(d.own[i], 0u, o.own));
                const float z = ZEROS ? (float)((d.zero[i] >> ((o.zero + 8 * (st * NG + 4 * i)) & 31)) & 0xFFu) : 8.f;
                const bool on = NG > 2 || ln.g < NG;
                float x = 0.f;
#pragma unroll
                for (int j = 0; j < (NG < 4 ? NG : 4); ++j) x = (int)ln.g == j ? tokens[4 * i + j][0] : x;
                acc[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(on ? -s * (16.f + z) : 0.f, x, acc[0], 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < NG; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[1][e] = fmaf(__uint_as_float(__builtin_amdgcn_perm(d.scale[j][e], 0u, j & 1 ? o.odd[e] : o.even[e])),
                                     part[j][e], acc[1][e]);
        }
    }
    __device__ __forceinline__ uint8_t *tokens(int buffer) const { return xs + (size_t)buffer * WINDOW * FRAGS * 64 * p.T; }
    __device__ __forceinline__ void stage(int a, int b, int buffer) const {
        few_request_x<F, kGemvThreads>(p.x, p.ldx, p.T, p.K, a * FRAGS, b * FRAGS, tokens(buffer));
    }
    __device__ __forceinline__ void staged(int a, int b, int buffer) const {
        if constexpr (I4)
            for (int i = threadIdx.x; i < (b - a) * FRAGS * 4 * p.T; i += kGemvThreads) {
                u32x4 *v = reinterpret_cast<u32x4 *>(tokens(buffer) + (size_t)i * 16);
                *v = few_i4_order(*v);
            }
    }
    __device__ __forceinline__ void finish(int u, int, const f32x4 &sum) const {
        if (p.slices == 1) {
            gemv_store<F>(p, u, sum);
        } else if ((int)ln.r < p.T) {
            *reinterpret_cast<f32x4 *>(MOE_CHECKED(p.part + (((size_t)u * p.slices + slice) * p.T + ln.r) * 16 + 4 * ln.g, 16,
                                                   p.part, (size_t)p.units * p.slices * p.T * 64)) = sum;
        }
    }
};

// S: steps in each wave's ring.  WINDOW: of the token rows (FewUnits).
template <int F, int GROUP, bool ZEROS, int S, int WINDOW>
__global__ __launch_bounds__(kGemvThreads) void gemv_w4_kernel(GemvArgs p) {
    __shared__ GemvSmem sm;
    using Src = GemvUnits<F, GROUP, ZEROS, S, WINDOW>;
    const int wave = wave_index(), range = blockIdx.x / p.slices, slice = blockIdx.x % p.slices, T = p.T;
    const int nst = few_steps(F, p.K);
    const int c0 = (int)((long long)slice * nst / p.slices), c1 = (int)((long long)(slice + 1) * nst / p.slices);
    const int u0 = (int)((long long)range * p.units / p.ranges), u1 = (int)((long long)(range + 1) * p.units / p.ranges);
    const Src src(p, slice, c0, c1, sm.area + kGemvWaves * S * Src::SLOT);
    FewUnits<Src> run(src, sm.area, sm.red);
    // the token rows are requested before the weights, so that they arrive first
    if constexpr (WINDOW == 0) src.stage(c0, c1, 0);
    run.start(u0, u1, 0, c1 - c0);
    if constexpr (WINDOW == 0) {
        if (run.more()) few_wait<S * Src::OPS>();   // the ring's S steps are behind them
        else few_wait<0>();
        src.staged(c0, c1, 0);
        __syncthreads();
    }
    run.run();
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
    const int t = min((int)(threadIdx.x & 15), T - 1), g = (threadIdx.x & 63) >> 4;
    for (int u = u0 + wave; u < u1; u += kGemvWaves) {
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < p.slices; ++s)
            sum += *reinterpret_cast<const f32x4 *>(MOE_CHECKED(p.part + (((size_t)u * p.slices + s) * T + t) * 16 + 4 * g, 16,
                                                                p.part, (size_t)p.units * p.slices * T * 64));
        gemv_store<F>(p, u, sum);
    }
}

// Steps in a ring: the deepest that leaves the whole token rows room, else the
// one that leaves room for windows of four steps (which cost barriers: 16
// tokens x 2816 -> 131072 in INT4 58 us with whole rows and three steps, 72
// with windows and four).
constexpr int kGemvDeep = 6, kGemvMiddle = 4, kGemvShallow = 3, kGemvWindow = 4;

template <int F, int GROUP, bool ZEROS>
void launch_format(const GemvArgs &p, hipStream_t st) {
    constexpr int slot = GemvSlot<F, GROUP, ZEROS>::SLOT;
    constexpr int windows = 2 * kGemvWindow * FewStep<F>::FRAGS * 64 * kFewTokens;
    constexpr int S = (kGemvArea - windows) / (kGemvWaves * slot);
    static_assert(S >= 3, "a ring next to the windows");
    const dim3 grid(p.ranges * p.slices), block(kGemvThreads);
    const long long x = (long long)(few_steps(F, p.K) + p.slices - 1) / p.slices * FewStep<F>::FRAGS * 64 * p.T;
    auto fits = [&](int s) { return x + kGemvWaves * s * slot <= kGemvArea; };
    if (fits(kGemvDeep)) gemv_w4_kernel<F, GROUP, ZEROS, kGemvDeep, 0><<<grid, block, 0, st>>>(p);
    else if (fits(kGemvMiddle)) gemv_w4_kernel<F, GROUP, ZEROS, kGemvMiddle, 0><<<grid, block, 0, st>>>(p);
    else if (fits(kGemvShallow)) gemv_w4_kernel<F, GROUP, ZEROS, kGemvShallow, 0><<<grid, block, 0, st>>>(p);
    else gemv_w4_kernel<F, GROUP, ZEROS, S, kGemvWindow><<<grid, block, 0, st>>>(p);
}

}  // namespace

// Workgroups of a product: `ranges` of units times `slices` of K, several
// slices where the token rows do not fit the LDS (next to a shallow ring) and
// there are too few units for all workgroups.
GemvPlan gemv_plan(int T, int N, int K, bool geglu) {
    GemvPlan g;
    g.outs = geglu ? N / 2 : N;
    g.units = geglu ? (g.outs + 7) / 8 : (N - 1) / 16 + 1;
    const int steps = (K - 1) / 256 + 1, fit = (kGemvArea - kGemvWaves * kGemvShallow * 2304) / (512 * T);
    // (to no fewer than 16 steps, two for each wave, beyond what the LDS asks for)
    g.slices = steps <= fit ? 1 : std::max(1, std::min(kGemvBlocks / g.units, std::max((steps + fit - 1) / fit, steps / 16)));
    g.ranges = std::min(g.units, kGemvBlocks / g.slices);
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
    p.y_wide = l.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(l.y) % (l.y_fp32 ? 16 : 8) == 0;
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
