// Building blocks of the few-token kernels (the whole layer for up to 16
// tokens and the 4-bit matrix-vector product): up to 16 token rows are the
// columns of one 16x16x32 MFMA, sixteen weight rows its rows, so a weight
// value is loaded once and multiplied with every token.
//
// Each wave streams its own weights: steps of 16 rows x 128 bytes (whole cache
// lines; 64 K values of bf16, 256 of 4-bit codes) go straight from global
// memory into the slots of a ring in LDS that only this wave uses, so no
// barrier paces the stream and a few instructions, the same for every step,
// keep it running (a ring in registers, its turns unrolled, spent most of a
// one-token call fetching instructions: 42.8 us against 39.8 in bf16; 8 tokens
// 168 against 126).
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

// ODD: scale rows of NVFP4 may start in the middle of a word (K a multiple of
// 32 but not of 64).
template <int F, bool ODD = false>
struct FewStep {
    static constexpr int K = F == kFewBf16 ? 64 : 256;           // K values
    static constexpr int FRAGS = K / 32;                          // MFMAs
    static constexpr int SB = F == kFewMx ? 1 : F == kFewNv ? 2 : 0;   // scale bytes of a piece (8 pieces)
    // Scales (MXFP4, NVFP4): the aligned words that hold a row's 8 or 16 bytes, four to a load of the wave (one
    // load a step rather than each lane its own words: those are half the requests of a step, and take the
    // time of as many cache lines).
    static constexpr int SOPS = SB == 0 ? 0 : ODD && F == kFewNv ? 2 : 1;
    static constexpr int SLOT = 2048 + 256 * SOPS;                // ring slot: 16 rows of 128 bytes, the scale words
    static constexpr int OPS = 2 + SOPS;                          // loads
    // bf16 rows are whole lines that are read once and carry the non-temporal hint: the layer of 8 tokens takes
    // 118 us with it, 129 without.  4-bit rows of a multiple of 16 bytes may straddle lines, whose other part the
    // next step wants (MXFP4, 1 token: 28.3 without, 29.3 with; 8 tokens 63.4 and 61.1).
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

// Where one lane loads the steps of sixteen rows from: 16 bytes of row l / 8
// of each of two blocks of eight consecutive rows, the piece swizzled so that
// the fragment reads have no bank conflicts, and a scale word.  A 4-bit row
// may end inside a step: pieces past its end read the row's last piece, whose
// codes then meet zero token values.
struct FewRows {
    const uint8_t *top, *low;   // of step 0
    const uint8_t *scale;
    uint32_t last_scale;        // offset of the last scale word of the row
};

template <int F, bool ODD = false>
struct FewLane {
    using Step = FewStep<F, ODD>;
    int pieces;                    // of a row
    uint32_t pitch, spitch;        // bytes of a row of weights, of scales
    uint32_t piece;                // loads: this lane's piece within a step
    uint32_t r, g;

    __device__ __forceinline__ explicit FewLane(int k) {
        const uint32_t l = threadIdx.x & 63;
        pitch = F == kFewBf16 ? 2 * k : k / 2;
        spitch = F == kFewMx ? k / 32 : k / 16;
        pieces = k / (F == kFewBf16 ? 8 : 32);
        piece = (l & 7) ^ (l >> 3);
        r = l & 15;
        g = l >> 4;
    }
    // Rows from `top` and `low` on (scales from `stop` and `slow` on); ntop, nlow: the last of each block's
    // eight rows that exists (the others repeat it).
    __device__ __forceinline__ FewRows rows(const uint8_t *top, const uint8_t *low, const uint8_t *stop,
                                            const uint8_t *slow, int ntop = 7, int nlow = 7) const {
        const int l = threadIdx.x & 63, row = l >> 3, q = l >> 2;
        FewRows m{top + min(row, ntop) * (size_t)pitch, low + min(row, nlow) * (size_t)pitch, nullptr, 0};
        if constexpr (Step::SOPS > 0) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(q < 8 ? stop + min(q, ntop) * (size_t)spitch
                                                                   : slow + min(q - 8, nlow) * (size_t)spitch);
            m.scale = reinterpret_cast<const uint8_t *>(at & ~(uintptr_t)3);
            m.last_scale = (((uint32_t)at & 3) + spitch - 1) & ~3u;
        }
        return m;
    }
    // Requests step s into `slot` (wave-uniform).  wb, wn / sb, sn: the extent of the matrices (debug build).
    __device__ __forceinline__ void issue(const FewRows &m, int s, uint8_t *slot, [[maybe_unused]] const void *wb,
                                          [[maybe_unused]] size_t wn, [[maybe_unused]] const void *sb,
                                          [[maybe_unused]] size_t sn) const {
        uint32_t off = 128 * s + 16 * piece;
        if constexpr (F != kFewBf16) off = min(off, 16u * pieces - 16);
        dma16<Step::STREAM>(MOE_CHECKED(m.top + off, 16, wb, wn), slot);
        dma16<Step::STREAM>(MOE_CHECKED(m.low + off, 16, wb, wn), slot + 1024);
        // words l % 4 (and 4 + l % 4) of row l / 4, none past the one that ends the row
#pragma unroll
        for (int h = 0; h < Step::SOPS; ++h)
            dma4(MOE_CHECKED(m.scale + min(8 * Step::SB * s + 16 * h + 4 * (threadIdx.x & 3), m.last_scale), 4, sb,
                             (sn + 3) & ~(size_t)3),
                 slot + 2048 + 256 * h);
    }
    // 16-byte piece 4 h + g of this lane's row in a slot whose loads are complete
    __device__ __forceinline__ u32x4 load(const uint8_t *slot, int h) const {
        return *reinterpret_cast<const u32x4 *>(slot + 128 * r + (((4 * h + g) ^ (r & 7)) << 4));
    }
    // its scales (0 past the row's end); lo: the address of its scale row modulo 4
    __device__ __forceinline__ uint32_t scale(const uint8_t *slot, int s, int h, uint32_t lo) const {
        const uint32_t p = 4 * h + g, at = (lo & 3) + Step::SB * p;
        const uint32_t w = *reinterpret_cast<const uint32_t *>(slot + 2048 + 16 * (at & ~15u) + 16 * r + (at & 12));
        const uint32_t v = (w >> (8 * (at & 3))) & (F == kFewMx ? 0xFFu : 0xFFFFu);
        return (int)(8 * s + p) < pieces ? v : 0u;
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
struct FewI4 {
    // in a vector and a scalar register, so that and-or is one instruction (as constants they take two)
    uint32_t mask = 0x00780078u, base = 0x41804180u;
    __device__ __forceinline__ FewI4() { asm("" : "+v"(mask), "+s"(base)); }
    __device__ __forceinline__ u32x4 operand(uint32_t w) const {
        return u32x4{((w << 3) & mask) | base, ((w >> 1) & mask) | base, ((w >> 5) & mask) | base, ((w >> 9) & mask) | base};
    }
};

// What a step multiplies, out of its slot and the token rows (bf16, MXFP4,
// NVFP4).
//
// PARTS: the token values are sums of that many bf16 values.
template <int F, int PARTS = 1>
struct FewData {
    u32x4 c[2];
    uint32_t sc[2];
    u32x4 x[PARTS][FewStep<F>::FRAGS];
};

template <int F, int PARTS>
__device__ __forceinline__ void few_multiply(const FewData<F, PARTS> &d, f32x4 (&acc)[2]) {
    constexpr int N = FewStep<F>::FRAGS / 2;   // MFMAs of a piece
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < N; ++f) {
            const u32x4 w = few_operand<F>(d.c[h], d.sc[h], f);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) acc[h] = mfma16x16x32(w, d.x[i][N * h + f], acc[h]);
        }
}

// A workgroup's run of units, each an MFMA tile of sixteen weight rows summed
// along its steps.  Whole rounds of eight units go a unit to a wave and need no
// barrier; the units that are left (fewer than eight) are split along K so that
// no wave is longer at work than it must, and their sums joined.  The order of
// each unit's sum depends on the run alone.
//
// Token rows are in LDS, whole, before run() (WINDOW 0), or, where that leaves
// the rings too little room, come in windows of up to WINDOW steps: all waves
// go through the same windows, the next of which is on its way to a second
// buffer meanwhile, and a barrier separates them.  Then all units go a unit to
// a wave.
//
// Src says what the units are: S, SLOT, OPS (steps in a ring, bytes of its
// slots, loads of a step), WINDOW, at(u, v) (the unit's segment of the
// weights, v or a later one), span(v, a, b) (its steps), rows(u, v),
// issue(rows, v, step, slot), operand(u, v) (this lane's token data),
// fetch(slot, step, token step, operand) (out of LDS), multiply(data, step,
// operand, acc), finish(u, v, sums); with windows stage(a, b, buffer) (requests
// the token rows of steps a .. b - 1) and staged(a, b, buffer) (they are here:
// each thread's own).
template <class Src>
struct FewUnits {
    static constexpr int S = Src::S, SLOT = Src::SLOT, OPS = Src::OPS, WAVES = 8;
    const Src &src;
    uint8_t *ring;
    f32x4 (*red)[64];                                 // partial sums of the waves
    int wave, lane;
    int u0 = 0, um = 0, u1 = 0, KW = 1, UG = 1;      // the run; um: the units that are left, UG at a time
    int v0 = 0;                                       // its first segment
    int lu = 0, lv = 0, ls = 0, ls1 = 0, lslot = 0;   // the step to request next (u1: none) and its slot
    int c0 = 0, c1 = 0, NW = 1;                       // windows: of steps c0 .. c1 - 1
    typename Src::Rows rows;

    __device__ __forceinline__ FewUnits(const Src &src, uint8_t *rings, f32x4 (*red)[64])
        : src(src), ring(rings + wave_index() * S * SLOT), red(red), wave(wave_index()), lane(threadIdx.x & 63) {}
    // this wave's steps of unit u of segment v
    __device__ __forceinline__ void part(int u, int v, int &a, int &b) const {
        src.span(v, a, b);
        if (u >= um) {
            const int kw = wave & (KW - 1), n = b - a;
            b = a + (kw + 1) * n / KW;
            a += kw * n / KW;
        }
    }
    // the next unit with steps for this wave: u, or one after it (left: u is one of the units that are left)
    __device__ __forceinline__ void seek(int u, bool left) {
        for (;; u += left ? UG : WAVES) {
            if (!left && u >= um) {
                left = true;
                u = um + wave / KW;
            }
            lu = u1;
            if (u >= u1) return;
            lv = src.at(u, lv);
            part(u, lv, ls, ls1);
            if (ls < ls1) break;   // not where there are more waves than steps
        }
        lu = u;
        rows = src.rows(u, lv);
    }
    __device__ __forceinline__ void request() {
        src.issue(rows, lv, ls, ring + lslot * SLOT);
        lslot = lslot + 1 == S ? 0 : lslot + 1;
        if (++ls == ls1) seek(lu + (lu >= um ? UG : WAVES), lu >= um);
    }
    // Requests the first steps of units a .. b - 1, a of segment v, each of at most `steps` steps.
    __device__ __forceinline__ void start(int a, int b, int v, int steps) {
        u0 = a;
        u1 = b;
        um = Src::WINDOW ? b : b - (b - a) % WAVES;
        KW = Src::WINDOW ? 1 : few_kwaves(b - um, steps);
        if constexpr (Src::WINDOW > 0) {
            src.span(v, c0, c1);
            NW = (c1 - c0 + Src::WINDOW - 1) / Src::WINDOW;
            if (a < b) src.stage(c0, c0 + (c1 - c0) / NW, 0);
        }
        UG = WAVES / KW;
        v0 = lv = v;
        lslot = 0;
        seek(u0 + wave, false);
        for (int i = 0; i < S && lu < u1; ++i) request();
    }
    // whether steps are left to request (after start: the ring is full)
    __device__ __forceinline__ bool more() const { return lu < u1; }
    // Steps a .. b - 1 of this wave's unit, whose token rows begin with token step x0.
    __device__ __forceinline__ void steps(int a, int b, int x0, const typename Src::Operand &x, int &slot, f32x4 (&acc)[2]) {
        for (int st = a; st < b; ++st) {
            // the ring is full but for this step's successors: S - 1 steps may be in flight
            if (lu < u1) few_wait<(S - 1) * OPS>();
            else few_wait<0>();
            // everything of the step into registers at once, then its slot is free for another
            const auto d = src.fetch(ring + slot * SLOT, st, x0 + st - a, x);
            few_lds_done();
            if (lu < u1) request();
            src.multiply(d, st, x, acc);
            slot = slot + 1 == S ? 0 : slot + 1;
        }
    }
    // Window w of a round is here, and all waves are done with the one before; the next is requested (last: no).
    __device__ __forceinline__ void next_window(int n, int w, bool last) const {
        static_assert(S * OPS <= 63 && Src::WINDOW / 2 * OPS <= 63, "the counter of outstanding loads");
        // behind its requests: the ring's S steps, later a step's for each of the window before (no fewer than
        // half a WINDOW: windows are as even as whole steps allow)
        if (lu >= u1) few_wait<0>();
        else if (n == 0) few_wait<S * OPS>();
        else few_wait<Src::WINDOW / 2 * OPS>();
        const int len = c1 - c0;
        src.staged(c0 + w * len / NW, c0 + (w + 1) * len / NW, n & 1);
        __syncthreads();
        if (last) return;
        const int m = w + 1 == NW ? 0 : w + 1;
        src.stage(c0 + m * len / NW, c0 + (m + 1) * len / NW, (n + 1) & 1);
    }
    __device__ __forceinline__ void run() {
        int slot = 0, v = v0;
        [[maybe_unused]] int n = 0;   // windows so far
        for (int i = u0; i < u1;) {
            const bool left = i >= um;
            const int u = i + (left ? wave / KW : wave);
            const bool on = uniform(u < u1);
            f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            if constexpr (Src::WINDOW > 0) {
                typename Src::Operand x = src.operand(on ? u : u0, v = src.at(on ? u : u1 - 1, v));
                for (int w = 0; w < NW; ++w, ++n) {
                    next_window(n, w, w + 1 == NW && i + WAVES >= u1);
                    const int a = c0 + w * (c1 - c0) / NW, b = c0 + (w + 1) * (c1 - c0) / NW;
                    if (on) steps(a, b, (n & 1) * Src::WINDOW, x, slot, acc);
                }
            } else if (on) {
                v = src.at(u, v);
                int a, b;
                part(u, v, a, b);
                steps(a, b, a, src.operand(u, v), slot, acc);
            }
            const f32x4 sum = acc[0] + acc[1];
            if (!left) {
                if (on) src.finish(u, v, sum);
            } else {
                red[wave][lane] = sum;
                __syncthreads();
                if (uniform(wave < UG && i + wave < u1)) {
                    f32x4 all = {0.f, 0.f, 0.f, 0.f};
                    for (int w = 0; w < KW; ++w) all += red[wave * KW + w][lane];
                    src.finish(i + wave, src.at(i + wave, v0), all);
                }
                __syncthreads();
            }
            i += left ? UG : WAVES;
        }
    }
};

// Requests 16-byte pieces of T token rows (row stride ld) for fragments f0 ..
// f1 - 1 into LDS: in fragment, lane group, token order, zero past K.
template <int F, int THREADS>
__device__ __forceinline__ void few_request_x(const uint16_t *x, long long ld, int T, int K, int f0, int f1, uint8_t *dst) {
    [[maybe_unused]] const size_t bytes = (size_t)((T - 1) * ld + K) * 2;
    for (int i = threadIdx.x; i < (f1 - f0) * 4 * T; i += THREADS) {
        const int t = i % T, fg = i / T, k = few_frag_k<F>(f0 + (fg >> 2), fg & 3);
        if (k < K) dma16<false>(MOE_CHECKED(x + t * ld + k, 16, x, bytes), dst + (size_t)(i - (threadIdx.x & 63)) * 16);
        else *reinterpret_cast<u32x4 *>(dst + (size_t)i * 16) = u32x4{0u, 0u, 0u, 0u};
    }
}

}  // namespace moe
