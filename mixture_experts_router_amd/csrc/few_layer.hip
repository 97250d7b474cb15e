// The whole MoE layer for up to 16 tokens in one launch (moe_forward_few).
//
// With few tokens the layer is a stream of expert weights: each touched
// expert's gate/up and down matrices are read once and multiplied with every
// token (few_stream.h), so the bytes bound it and launches and waits are the
// rest of its time.  One persistent grid runs the phases:
//
//   router   logits = x W_r^T (+ b), four experts per work item, summed as
//            moe_route does (fp32 chunks of 256, added in fp64), so both give
//            the same bits
//   gate/up  every workgroup selects the experts itself (top-k of the few
//            tokens from the logits), then h = gelu_tanh(g) * u for its share
//            of the (expert, 8 columns) units
//   down     y[t, e][16 columns] = W_d h in fp32, the units of all touched
//            experts shared evenly; with up to 16 assignments instead
//            out[t][16 columns] = sum over experts of w[t, e] * (W_d h)
//   combine  (where down stored y) out = sum over experts of w[t, e] * y: the
//            routing weights multiply fp32 sums, experts are added in a fixed
//            order, and out is rounded once
//
// Each phase's items are handed out by a ticket counter.  A workgroup takes
// router items while there are any, then gate/up shares, then down items, then
// combine items, and waits only for items of an earlier phase, all of which
// have then been taken by workgroups that are running: every wait ends,
// whatever else runs on the GPU and however few workgroups are resident.
//
// h goes into the down product's MFMAs as two bf16 values, its rounding to bf16
// and the rounding of what that left (16 bits of mantissa): one alone would add
// as much error to out as out's own rounding (2.4e-3 of out's norm against
// 1.65e-3).  It costs 16 tokens with the MLP 4% (189 us against 181), fewer
// tokens nothing.  Nothing else is rounded below fp32 before out.
//
// Measured at hidden 2816, 128 experts, top-8, expert intermediate 704, one
// call after another: 1 token 37 us in bf16 (95.9 MB of weights) and 28 in
// MXFP4 (26.0 MB), 8 tokens 116 (615 MB: 5.3 TB/s) and 62 (164 MB), 5 tokens
// in NVFP4 56 (119 MB), 16 tokens with the dense MLP in bf16 189 (1.02 GB: 5.4
// TB/s).  Of the 8 bf16 tokens' time 13 us pass before the first
// expert weight is requested (start 2, ticket and router 5, top-k 6), 58 in
// gate/up (7.0 TB/s), 9 until h has arrived everywhere, 28 in down (7.3 TB/s,
// first weights requested before h is there), 6 in combine.  What bounds it:
// the bytes, and with one token the chain of dependent trips to memory between
// the phases.
#include <algorithm>

#include "few_stream.h"
#include "moe_launch.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;
constexpr int kFewMaxA = kFewTokens * 32;                 // assignments (k <= 32)
constexpr int kFewArea = 136 * 1024;                      // LDS for the rings and the token rows (the rest: 23 KB)

// Counters in the workspace's zeroed prefix, a line each: tickets (the next
// item of each phase), items done, workgroups left.  A phase's items done are
// counted in one place and, when all are, signalled in kSignals: 256 workgroups
// polling the count itself hold up each other and those that still count.
enum FewPhase { kRouter = 0, kGateUp = 1, kDown = 2, kCombine = 3 };
constexpr int kCtrTicket = 0, kCtrDone = 4, kCtrExit = 7, kCtrSignal = 8, kSignals = 8;
constexpr int kCtrLine = 32, kCtrWords = kCtrLine * (kCtrSignal + 3 * kSignals);
static_assert(kCtrWords * 4 == kFewCounterBytes, "the zeroed prefix");

struct FewArgs {
    const uint16_t *x, *wr;
    const float *bias;
    const uint8_t *wgu, *gus, *wd, *ds;         // experts: weights (or codes) and block scales
    const float *gug, *dg;                      // NVFP4: matrix scales
    const uint8_t *swgu, *sgus, *swd, *sds;     // dense MLP, the same
    const float *sgug, *sdg;
    uint16_t *out;
    int32_t *ids;
    float *wts;
    uint32_t *ctr;
    float *logits;
    uint16_t *h, *h_sh;                         // [T k][part][I], [T][part][I_sh]
    float *y;                                   // [segment of an expert][T k][H], [segment of the MLP][T][H]
    int T, H, E, k, I, I_sh;
    int n_router, n_gu, n_down, n_combine;      // items of each phase
    int columns, PW, ne, ns;                    // down: see FewDown, FewPieces
};

struct FewSmem {
    alignas(1024) uint8_t area[kFewArea];                     // the waves' rings, then x (gate/up) or rows of h (down)
    f32x4 red[kFewWaves][64];                   // partial sums of the waves
    int32_t ids[kFewMaxA];
    float w[kFewMaxA];
    alignas(16) uint8_t slot[kFewMaxA][kFewTokens];   // [touched expert][token]: slot + 1, 0 = not routed there
    int16_t expert[kFewMaxA];                   // touched experts, ascending
    int16_t first[kFewMaxA + 2];                // their first position in expert order; [n_experts] = T k
    int16_t sorted[kFewMaxA];                   // assignments in expert order
    uint32_t mask[32];                          // touched experts
    int n_experts;
    int ticket, down;
};
static_assert(sizeof(FewSmem) <= 160 * 1024, "LDS of one workgroup");

__device__ __forceinline__ uint32_t ctr_add(uint32_t *p) {
    return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What one workgroup computes for others (logits, h) is stored through the
// caches, at agent scope, so that publishing it takes no cache write-back (a
// write-back by every workgroup cost 4 us a phase): once a store is complete,
// every workgroup that loads the line for the first time sees it.
template <typename V>
__device__ __forceinline__ void store_shared(V *p, V v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ uint32_t ctr_ticket(const FewArgs &p, FewPhase phase) {
    return ctr_add(p.ctr + kCtrLine * (kCtrTicket + phase));
}

// One thread counts an item of a phase of n done: its workgroup's stores are complete.
__device__ __forceinline__ void ctr_done(const FewArgs &p, FewPhase phase, int n) {
    if (ctr_add(p.ctr + kCtrLine * (kCtrDone + phase)) != (uint32_t)n - 1) return;
#pragma unroll
    for (int i = 0; i < kSignals; ++i) store_shared(p.ctr + kCtrLine * (kCtrSignal + kSignals * phase + i), 1u);
}

// Counts this workgroup's stored results: every wave's stores are complete,
// then one thread counts.
__device__ __forceinline__ void publish(const FewArgs &p, FewPhase phase, int n) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) ctr_done(p, phase, n);
}

// One thread waits until all items of a phase are done; its workgroup, which
// joins a barrier next, may then load what they stored: the caches'
// invalidation is complete, not merely requested, before the others load.
// The signal comes as long as the counters were zero before the launch;
// the bound only keeps a workspace that was not from holding the GPU (its
// results are then undefined).
__device__ __forceinline__ void wait_done(const FewArgs &p, FewPhase phase) {
    const uint32_t *flag = p.ctr + kCtrLine * (kCtrSignal + kSignals * phase + blockIdx.x % kSignals);
    for (int i = 0; i < (1 << 20); ++i) {
        if (__hip_atomic_load(flag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) break;
        __builtin_amdgcn_s_sleep(1);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Share i of n of `units` units: as even as whole units allow.
__device__ __forceinline__ int share_start(int i, int units, int n) {
    const int q = units / n, r = units - q * n;
    return i * q + min(i, r);
}

// ---------------------------------------------------------------- router
// Four experts, all tokens: wave w takes chunks w, w + 8, ... of 256 K
// values, each summed in fp32 by MFMAs in K order; one thread per (token,
// expert) adds the chunk sums in fp64 in chunk order.
__device__ void few_router(const FewArgs &p, FewSmem &sm, int item) {
    const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
    const int e0 = 4 * item, nchunks = (p.H + 255) / 256;
    const bool on_e = r < 4 && e0 + r < p.E, on_t = r < p.T;
    f32x4(*sum)[kFewTokens] = reinterpret_cast<f32x4(*)[kFewTokens]>(sm.red);   // [16 chunks][token]
    const int et = threadIdx.x >> 4, tt = threadIdx.x & 15;                       // of the adding threads (< 64)
    double total = 0.0;
    for (int c0 = 0; c0 < nchunks; c0 += 2 * kFewWaves) {
        // this wave's two chunks, c0 + wave and c0 + wave + 8: all their loads go out at once
        u32x4 a[2][8], b[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k0 = min(c0 + wave + i * kFewWaves, nchunks - 1) * 256, n = min(256, p.H - k0) / 32;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int k = k0 + 32 * (u < n ? u : 0) + 8 * g;
                a[i][u] = on_e ? *reinterpret_cast<const u32x4 *>(
                                     MOE_CHECKED(p.wr + (size_t)(e0 + r) * p.H + k, 16, p.wr, (size_t)p.E * p.H * 2))
                               : u32x4{0u, 0u, 0u, 0u};
                b[i][u] = on_t ? *reinterpret_cast<const u32x4 *>(
                                     MOE_CHECKED(p.x + (size_t)r * p.H + k, 16, p.x, (size_t)p.T * p.H * 2))
                               : u32x4{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int cc = wave + i * kFewWaves, n = min(256, p.H - (c0 + cc) * 256) / 32;
            if (uniform(c0 + cc < nchunks)) {
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (uniform(u < n)) acc = mfma16x16x32(a[i][u], b[i][u], acc);
                if (g == 0) sum[cc][r] = acc;
            }
        }
        __syncthreads();
        if (threadIdx.x < 64)
            for (int c = 0; c < 2 * kFewWaves && c0 + c < nchunks; ++c) total += (double)sum[c][tt][et];
        __syncthreads();
    }
    if (threadIdx.x < 64 && tt < p.T && e0 + et < p.E) {
        const double b = p.bias ? (double)p.bias[e0 + et] : 0.0;
        store_shared(MOE_CHECKED(p.logits + (size_t)tt * p.E + e0 + et, 4, p.logits, (size_t)p.T * p.E * 4),
                     (float)(total + b));
    }
}

template <int VPL>
__device__ __forceinline__ void few_topk(const FewArgs &p, FewSmem &sm, int t, bool store) {
    const int lane = threadIdx.x & 63;
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 64 * i;
        key[i] = e < p.E ? order_key(*MOE_CHECKED(p.logits + (size_t)t * p.E + e, 4, p.logits, (size_t)p.T * p.E * 4)) : 0u;
    }
    int idx;
    const float w = topk_slots<VPL>(key, p.k, idx);
    if (lane >= p.k) return;
    const int a = t * p.k + lane;
    sm.ids[a] = idx;
    sm.w[a] = w;
    if (store) {
        if (p.ids) *MOE_CHECKED(p.ids + a, 4, p.ids, (size_t)p.T * p.k * 4) = idx;
        if (p.wts) *MOE_CHECKED(p.wts + a, 4, p.wts, (size_t)p.T * p.k * 4) = w;
    }
}

// How many of the first n bytes of a row of `slot` are set (a byte is below 128).
__device__ __forceinline__ int few_count(const u32x4 &row, int n) {
    int c = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int b = min(max(n - 4 * q, 0), 4);
        c += __popc((row[q] + 0x7F7F7F7Fu) & 0x80808080u & (uint32_t)((1ull << (8 * b)) - 1));
    }
    return c;
}

// The routing of every token, by each workgroup for itself: ids and weights,
// the touched experts in ascending order, who goes there, and the assignments
// in (expert, token) order.
__device__ void few_select(const FewArgs &p, FewSmem &sm, bool store) {
    const int wave = wave_index(), A = p.T * p.k, a = threadIdx.x;
    for (int i = threadIdx.x; i < A * kFewTokens / 4; i += kFewThreads) reinterpret_cast<uint32_t *>(sm.slot)[i] = 0u;
    if (threadIdx.x < 32) sm.mask[threadIdx.x] = 0u;
    if (threadIdx.x == 0) wait_done(p, kRouter);
    __syncthreads();
    for (int t = wave; t < p.T; t += kFewWaves) {
        if (p.E <= 64) few_topk<1>(p, sm, t, store);
        else if (p.E <= 128) few_topk<2>(p, sm, t, store);
        else if (p.E <= 256) few_topk<4>(p, sm, t, store);
        else if (p.E <= 512) few_topk<8>(p, sm, t, store);
        else few_topk<16>(p, sm, t, store);
    }
    __syncthreads();
    const int e = a < A ? sm.ids[a] : 0;   // thread a: assignment a (A <= the threads)
    if (a < A) atomicOr(&sm.mask[e >> 5], 1u << (e & 31));
    __syncthreads();
    int u = 0, n = 0;
    for (int i = 0; i < (p.E + 31) / 32; ++i) {
        const uint32_t m = sm.mask[i];
        u += __popc(i < (e >> 5) ? m : i == (e >> 5) ? m & ((1u << (e & 31)) - 1) : 0u);
        n += __popc(m);
    }
    if (a < A) {
        sm.slot[u][a / p.k] = (uint8_t)(a % p.k + 1);
        sm.expert[u] = (int16_t)e;
    }
    if (threadIdx.x == 0) sm.n_experts = n;
    __syncthreads();
    // positions in expert order: a touched expert's count by each thread, then the counts before it
    const int count = a < n ? few_count(*reinterpret_cast<const u32x4 *>(sm.slot[a]), kFewTokens) : 0;
    // inclusive sum over the wave, then over the waves before
    const int lane = threadIdx.x & 63;
    int incl = count;
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(incl, d);
        if (lane >= d) incl += v;
    }
    int *part = reinterpret_cast<int *>(sm.red);
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    int at = incl - count;
    for (int v = 0; v < wave; ++v) at += part[v];
    if (a < n) {
        sm.first[a] = (int16_t)at;
        for (int t = 0; t < p.T; ++t)
            if (const int j = sm.slot[a][t]) sm.sorted[at++] = (int16_t)(t * p.k + j - 1);
        if (a == n - 1) sm.first[n] = (int16_t)at;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- gate/up
template <int F>
__device__ void few_stage_x(const FewArgs &p, uint8_t *xs) {
    const int nfrag = few_steps(F, p.H) * FewStep<F>::FRAGS;
    for (int i = threadIdx.x; i < nfrag * 4 * p.T; i += kFewThreads) {
        const int t = i % p.T, fg = i / p.T, k = few_frag_k<F>(fg >> 2, fg & 3);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (k < p.H)
            v = *reinterpret_cast<const u32x4 *>(MOE_CHECKED(p.x + (size_t)t * p.H + k, 16, p.x, (size_t)p.T * p.H * 2));
        *reinterpret_cast<u32x4 *>(xs + (size_t)i * 16) = v;
    }
    __syncthreads();
}

// A lane's token data of a unit, its row of weights, and the address of that
// row's scales modulo 4 (a unit's first scale row starts at a multiple of 4).
template <int F>
struct FewOperand {
    const uint8_t *x;
    FewLane<F> ln;
    uint32_t lo;
    __device__ __forceinline__ FewOperand(const uint8_t *x, const FewLane<F> &ln)
        : x(x), ln(ln), lo((ln.r & 7) * ln.spitch) {}
};

// A step out of its slot and (token step xst) the token rows of Src.
template <int F, int PARTS, class Src>
__device__ __forceinline__ FewData<F, PARTS> few_fetch(const Src &src, const uint8_t *q, int st, int xst,
                                                       const FewOperand<F> &o) {
    FewData<F, PARTS> d;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        d.c[h] = o.ln.load(q, h);
        d.sc[h] = 0;
        if constexpr (FewStep<F>::SOPS > 0) d.sc[h] = o.ln.scale(q, st, h, o.lo);
    }
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int f = 0; f < FewStep<F>::FRAGS; ++f) d.x[i][f] = src.frag(o.x, xst, f, i);
    return d;
}

// Gate/up units of eight h columns: the MFMA's rows are the unit's eight gate
// rows and the matching eight up rows.
template <int F, int S_, int WINDOW_>
struct FewGateUp {
    static constexpr int S = S_, SLOT = FewStep<F>::SLOT, OPS = FewStep<F>::OPS, WINDOW = WINDOW_;
    using Rows = FewRows;
    using Operand = FewOperand<F>;
    const FewArgs &p;
    FewSmem &sm;
    const bool shared;
    const int I, per;          // units of an expert
    const FewLane<F> ln;

    __device__ __forceinline__ FewGateUp(const FewArgs &p, FewSmem &sm, bool shared)
        : p(p), sm(sm), shared(shared), I(shared ? p.I_sh : p.I), per(I / 8), ln(p.H) {}
    __device__ __forceinline__ int at(int u, int v) const {   // (segment: touched expert)
        while (u >= (v + 1) * per) ++v;
        return v;
    }
    __device__ __forceinline__ const FewLane<F> &lane(int) const { return ln; }
    __device__ __forceinline__ const uint8_t *weights(int) const { return shared ? p.swgu : p.wgu; }
    __device__ __forceinline__ const uint8_t *scales(int) const { return shared ? p.sgus : p.gus; }
    __device__ __forceinline__ size_t weight_bytes(int) const { return (size_t)(shared ? 1 : p.E) * 2 * I * ln.pitch; }
    __device__ __forceinline__ size_t scale_bytes(int) const { return (size_t)(shared ? 1 : p.E) * 2 * I * ln.spitch; }
    __device__ __forceinline__ void span(int, int &a, int &b) const {
        a = 0;
        b = few_steps(F, p.H);
    }
    __device__ __forceinline__ FewRows rows(int u, int v) const {
        const size_t row = (size_t)(shared ? 0 : uniform(sm.expert[v])) * 2 * I + 8 * (u - v * per);
        const uint8_t *w = weights(v) + row * ln.pitch, *s = scales(v) + row * ln.spitch;
        return ln.rows(w, w + (size_t)I * ln.pitch, s, s + (size_t)I * ln.spitch);
    }
    __device__ __forceinline__ void issue(const FewRows &m, int v, int st, uint8_t *slot) const {
        lane(v).issue(m, st, slot, weights(v), weight_bytes(v), scales(v), scale_bytes(v));
    }
    __device__ __forceinline__ FewData<F> fetch(const uint8_t *q, int st, int xst, const FewOperand<F> &o) const {
        return few_fetch<F, 1>(*this, q, st, xst, o);
    }
    __device__ __forceinline__ void multiply(const FewData<F> &d, int, const FewOperand<F> &, f32x4 (&acc)[2]) const {
        few_multiply<F, 1>(d, acc);
    }
    __device__ __forceinline__ uint8_t *tokens(int buffer) const {
        return sm.area + kFewWaves * S * SLOT + (size_t)buffer * WINDOW * FewStep<F>::FRAGS * 64 * p.T;
    }
    __device__ __forceinline__ FewOperand<F> operand(int, int) const {
        return {tokens(0) + (ln.g * p.T + min((int)ln.r, p.T - 1)) * 16, ln};
    }
    __device__ __forceinline__ u32x4 frag(const uint8_t *x, int xst, int i, int) const {
        return *reinterpret_cast<const u32x4 *>(x + 64 * (xst * FewStep<F>::FRAGS + i) * p.T);
    }
    __device__ __forceinline__ void stage(int a, int b, int buffer) const {
        few_request_x<F, kFewThreads>(p.x, p.H, p.T, p.H, a * FewStep<F>::FRAGS, b * FewStep<F>::FRAGS, tokens(buffer));
    }
    __device__ __forceinline__ void staged(int, int, int) const {}
    // Lane 16 g + t, element q of the sums is weight row 4 g + q, token t: gate rows 0..7, up rows 8..15, so a
    // gate's up value is 32 lanes above.
    __device__ __forceinline__ void finish(int u, int v, const f32x4 &acc) const {
        const int t = ln.r;
        const float m = F != kFewNv ? 1.f : shared ? p.sgug[0] : p.gug[uniform(sm.expert[v])];
        float h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t b = __float_as_uint(acc[q]);
            const float up = __uint_as_float(__builtin_amdgcn_permlane32_swap(b, b, false, false)[1]);
            h[q] = gelu_tanh(acc[q] * m) * (up * m);
        }
        const int j = ln.g < 2 && t < p.T ? (shared ? 1 : (int)sm.slot[v][t]) : 0;
        if (j) {
            uint16_t *base = shared ? p.h_sh : p.h;
            const size_t row = shared ? (size_t)t : (size_t)t * p.k + j - 1;
            uint16_t *to = base + 2 * row * I + 8 * (u - v * per) + 4 * ln.g;
#pragma unroll
            for (int part = 0; part < 2; ++part, to += I) {
                const uint32_t b[2] = {pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
                store_shared(reinterpret_cast<uint64_t *>(MOE_CHECKED(to, 8, base, (size_t)p.T * (shared ? 1 : p.k) * I * 4)),
                             b[0] | (uint64_t)b[1] << 32);
                // what the rounding left (nothing where it left the range)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float r = bf16_to_f32(q & 1 ? b[q >> 1] >> 16 : b[q >> 1] & 0xFFFFu);
                    h[q] = __builtin_isinf(r) ? 0.f : h[q] - r;
                }
            }
        }
    }
};

template <int F, int S, int WINDOW>
__device__ __forceinline__ void few_gateup(const FewArgs &p, FewSmem &sm, bool shared, int units, int item) {
    const FewGateUp<F, S, WINDOW> src(p, sm, shared);
    FewUnits<FewGateUp<F, S, WINDOW>> run(src, sm.area, sm.red);
    const int u0 = share_start(item, units, p.n_gu);
    run.start(u0, share_start(item + 1, units, p.n_gu), u0 / src.per, few_steps(F, p.H));
    run.run();
}

// ---------------------------------------------------------------- down
// The K of the down products comes in segments: an expert's row, or pieces of
// it where T rows of h would not fit the LDS, then the dense MLP in
// pieces of the same size.  Units of sixteen output columns of one segment.
//
// COLUMNS: an item is one block of columns, all segments, added in registers
// (out is final).  Otherwise the items share the units evenly, in segment
// order, so that a workgroup needs few rows of h; each product is stored in
// fp32 and added by the combine phase.
//
// h is staged in LDS for as many segments as fit (a pass); the ring's first
// weights of a pass are requested before its h is staged, those of the first
// one before h exists.
//
// The token rows of gate/up are gone by then, so the rings need not be theirs.
// 16 tokens with MLP in bf16 take 189.0 us with three steps, 190.1 with five; 8
// tokens in MXFP4 62.6 with four, 63.1 with five (which leave 16 tokens' rows
// of intermediate 704 no room in one piece).
constexpr int few_down_ring(int f) { return f == kFewBf16 ? 3 : 4; }

template <int F, bool COLUMNS>
struct FewDown {
    static constexpr int S = few_down_ring(F), SLOT = FewStep<F>::SLOT, OPS = FewStep<F>::OPS, WINDOW = 0;
    using Rows = FewRows;
    using Operand = FewOperand<F>;
    static constexpr int KS = FewStep<F>::K;
    static constexpr int H_BYTES = kFewArea - kFewWaves * S * SLOT;   // LDS for rows of h
    const FewArgs &p;
    FewSmem &sm;
    const int ne, PW, pitch;      // segments of an expert, steps of a segment, bytes of one's row of h (two parts)
    const int UE, n, blocks;      // segments of the experts, of all; blocks of columns
    const int r, g;               // this lane's token, its part of a fragment
    uint8_t *hs;
    int item = 0, base = 0;       // COLUMNS: the block; rows of h before the pass
    mutable f32x4 out;            // COLUMNS: sums of this wave's units

    __device__ __forceinline__ FewDown(const FewArgs &p, FewSmem &sm)
        : p(p), sm(sm), ne(p.ne), PW(p.PW), pitch(2 * p.PW * KS * 2 + 16), UE(uniform(sm.n_experts) * p.ne), n(UE + p.ns),
          blocks(p.H / 16), r(threadIdx.x & 15), g((threadIdx.x & 63) >> 4), hs(sm.area + kFewWaves * S * FewStep<F>::SLOT) {}
    __device__ __forceinline__ int at(int u, int v) const {
        if constexpr (COLUMNS) return u;
        while (u >= (v + 1) * blocks) ++v;
        return v;
    }
    __device__ __forceinline__ int seg(int u) const { return COLUMNS ? u : u / blocks; }
    __device__ __forceinline__ int block(int u, int v) const { return COLUMNS ? item : u - v * blocks; }
    // touched expert of segment v, which of its pieces
    __device__ __forceinline__ int expert(int v) const { return ne == 1 ? v : v / ne; }
    __device__ __forceinline__ int piece(int v) const { return v >= UE ? v - UE : ne == 1 ? 0 : v % ne; }
    // rows of h of the segments before v
    __device__ __forceinline__ int rows_before(int v) const {
        if (v >= UE) return p.T * p.k * ne + (v - UE) * p.T;
        const int e = expert(v), q = v - e * ne, f = sm.first[e];
        return f * ne + q * (sm.first[e + 1] - f);
    }
    __device__ __forceinline__ FewLane<F> lane(int v) const { return FewLane<F>(v >= UE ? p.I_sh : p.I); }
    __device__ __forceinline__ const uint8_t *weights(int v) const { return v >= UE ? p.swd : p.wd; }
    __device__ __forceinline__ const uint8_t *scales(int v) const { return v >= UE ? p.sds : p.ds; }
    __device__ __forceinline__ size_t weight_bytes(int v) const {
        return (size_t)(v >= UE ? 1 : p.E) * p.H * lane(v).pitch;
    }
    __device__ __forceinline__ size_t scale_bytes(int v) const {
        return (size_t)(v >= UE ? 1 : p.E) * p.H * lane(v).spitch;
    }
    __device__ __forceinline__ void span(int v, int &a, int &b) const {
        a = piece(v) * PW;
        b = min(few_steps(F, v >= UE ? p.I_sh : p.I), a + PW);
    }
    __device__ __forceinline__ FewRows rows(int u, int v) const {
        const size_t row = (size_t)(v >= UE ? 0 : uniform(sm.expert[expert(v)])) * p.H + 16 * block(u, v);
        const FewLane<F> ln = lane(v);
        const uint8_t *w = weights(v) + row * ln.pitch, *s = scales(v) + row * ln.spitch;
        return ln.rows(w, w + (size_t)8 * ln.pitch, s, s + (size_t)8 * ln.spitch);
    }
    // slot of token t in segment v's expert, + 1 (0: not routed there)
    __device__ __forceinline__ int routed(int v, int t) const { return v >= UE ? t < p.T : (int)sm.slot[expert(v)][t]; }
    __device__ __forceinline__ void issue(const FewRows &m, int v, int st, uint8_t *slot) const {
        lane(v).issue(m, st, slot, weights(v), weight_bytes(v), scales(v), scale_bytes(v));
    }
    __device__ __forceinline__ FewData<F, 2> fetch(const uint8_t *q, int st, int xst, const FewOperand<F> &o) const {
        return few_fetch<F, 2>(*this, q, st, xst, o);
    }
    __device__ __forceinline__ void multiply(const FewData<F, 2> &d, int, const FewOperand<F> &, f32x4 (&acc)[2]) const {
        few_multiply<F, 2>(d, acc);
    }
    // this lane's row of h: its token's, or, where that is not routed here, the first one (left out by finish)
    __device__ __forceinline__ FewOperand<F> operand(int, int v) const {
        const int j = routed(v, r);
        const int rank = v >= UE ? r : few_count(*reinterpret_cast<const u32x4 *>(sm.slot[expert(v)]), r);
        return {hs + (size_t)(rows_before(v) - base + (j ? rank : 0)) * pitch - 2 * KS * PW * piece(v) +
                    2 * few_frag_k<F>(0, g), lane(v)};
    }
    __device__ __forceinline__ u32x4 frag(const uint8_t *x, int st, int i, int part) const {
        return *reinterpret_cast<const u32x4 *>(x + part * 2 * KS * PW + 2 * KS * st + 2 * few_frag_k<F>(i, 0));
    }
    __device__ __forceinline__ void finish(int u, int v, const f32x4 &acc) const {
        const int t = r, j = routed(v, t);
        float f = 1.f;
        if constexpr (F == kFewNv) f = v >= UE ? p.sdg[0] : p.dg[uniform(sm.expert[expert(v)])];
        if constexpr (COLUMNS) {
            if (v < UE) f *= sm.w[j ? t * p.k + j - 1 : 0];
#pragma unroll
            for (int q = 0; q < 4; ++q) out[q] = j ? fmaf(f, acc[q], out[q]) : out[q];
        } else if (j) {
            const int A = p.T * p.k;
            const size_t row = v >= UE ? (size_t)A * ne + (size_t)(v - UE) * p.T + t : (size_t)A * piece(v) + t * p.k + j - 1;
            uint64_t *y = reinterpret_cast<uint64_t *>(
                MOE_CHECKED(p.y + row * p.H + 16 * block(u, v) + 4 * g, 16, p.y, ((size_t)A * ne + p.T * p.ns) * p.H * 4));
#pragma unroll
            for (int q = 0; q < 4; q += 2)
                store_shared(y + q / 2, __float_as_uint(f * acc[q]) | (uint64_t)__float_as_uint(f * acc[q + 1]) << 32);
        }
    }
    // Copies the rows of h of segments va .. vb - 1: segment by segment, its rows in token order.
    __device__ __forceinline__ void stage(int va, int vb, int wave, int lane) const {
        for (int v = va + wave; v < vb; v += kFewWaves) {
            const bool m = v >= UE;
            const int e = expert(v), f = m ? 0 : uniform(sm.first[e]);
            const int nr = m ? p.T : uniform(sm.first[e + 1]) - f, I = m ? p.I_sh : p.I;
            const int a = piece(v) * PW, b = min(few_steps(F, I), a + PW);
            const int valid = (min(I, b * KS) - a * KS) / 8, all = (b - a) * (KS / 8);   // 16-byte pieces of a row
            uint8_t *row = hs + (size_t)(uniform(rows_before(v)) - base) * pitch;
            for (int i = 0; i < 2 * nr; ++i) {   // both parts of each row
                const uint16_t *hb = m ? p.h_sh : p.h;
                const uint16_t *src = hb + (size_t)(2 * (m ? i >> 1 : uniform(sm.sorted[f + (i >> 1)])) + (i & 1)) * I + a * KS;
                uint8_t *dst = row + (i >> 1) * pitch + (i & 1) * 2 * KS * PW;
                for (int c = 0; c < all; c += 64) {
                    if (c + lane < valid)
                        dma16<false>(MOE_CHECKED(src + 8 * (c + lane), 16, hb, (size_t)p.T * (m ? 1 : p.k) * I * 4),
                                     dst + 16 * c);
                    else if (c + lane < all)   // past the row: the codes there count nothing
                        *reinterpret_cast<u32x4 *>(dst + 16 * (c + lane)) = u32x4{0u, 0u, 0u, 0u};
                }
            }
        }
    }
};

template <int F, bool COLUMNS>
__device__ __forceinline__ void few_down_items(const FewArgs &p, FewSmem &sm, int item) {
    using Src = FewDown<F, COLUMNS>;
    const int lane = threadIdx.x & 63, wave = wave_index();
    Src src(p, sm);
    FewUnits<Src> run(src, sm.area, sm.red);
    for (bool have_h = false;;) {
        const int units = COLUMNS ? src.n : src.n * src.blocks;
        const int u0 = COLUMNS ? 0 : share_start(item, units, p.n_down);
        const int u1 = COLUMNS ? units : share_start(item + 1, units, p.n_down);
        src.item = item;
        src.out = f32x4{0.f, 0.f, 0.f, 0.f};
        int next = 0;
        for (int u = u0; u < u1;) {
            // the pass: segments va .. vb - 1, as many as fit
            const int va = src.seg(u), end = src.seg(u1 - 1) + 1, most = Src::H_BYTES / src.pitch;
            src.base = src.rows_before(va);
            int vb = va;
            for (;;) {   // 64 candidates at a time; the rows only grow
                const int v = vb + 1 + lane;
                const int fit = __popcll(__ballot(v <= end && src.rows_before(min(v, end)) - src.base <= most));
                vb += fit;
                if (fit < 64) break;
            }
            vb = uniform(vb);
            const int ub = COLUMNS ? vb : min(u1, vb * src.blocks);
            run.start(u, ub, va, src.PW);
            if (u == u0) {
                if (threadIdx.x == 0) {
                    const uint32_t n = ctr_ticket(p, kDown);   // (on its way while this waits)
                    if (!have_h) wait_done(p, kGateUp);
                    sm.down = (int)n;
                }
                __syncthreads();
                next = uniform(sm.down);
                have_h = true;
            }
            src.stage(va, vb, wave, lane);
            few_wait<0>();
            __syncthreads();
            run.run();
            u = ub;
            if (u < u1) __syncthreads();   // the rows of h are free
        }
        if constexpr (COLUMNS) {
            __syncthreads();
            sm.red[wave][lane] = src.out;
            __syncthreads();
            if (threadIdx.x < 256) {
                const int m = threadIdx.x & 15, t = threadIdx.x >> 4;
                float sum = 0.f;
#pragma unroll
                for (int v = 0; v < kFewWaves; ++v) sum += sm.red[v][16 * (m >> 2) + t][m & 3];
                if (t < p.T)
                    *MOE_CHECKED(p.out + (size_t)t * p.H + 16 * item + m, 2, p.out, (size_t)p.T * p.H * 2) =
                        (uint16_t)f32_to_bf16_rne(sum);
            }
            __syncthreads();   // the sums and the ticket in LDS are free
        } else {
            publish(p, kDown, p.n_down);
            __syncthreads();
        }
        item = next;
        if ((uint32_t)item >= (uint32_t)p.n_down) return;
    }
}

// Combine: out[t][c] = sum over token t's slots of w * y, then the dense MLP's
// segments: in this order, in fp32, rounded once.
__device__ __forceinline__ void few_combine(const FewArgs &p, const FewSmem &sm, int item) {
    const int i = item * kFewThreads + threadIdx.x;
    if (i >= p.T * p.H) return;
    const int t = i / p.H, c = i - t * p.H, A = p.T * p.k;
    [[maybe_unused]] const size_t bytes = ((size_t)A * p.ne + p.T * p.ns) * p.H * 4;
    float sum = 0.f;
    for (int q = 0; q < p.ne; ++q) {
        const float *y = p.y + ((size_t)A * q + t * p.k) * p.H + c;
#pragma unroll 8
        for (int j = 0; j < p.k; ++j) sum = fmaf(sm.w[t * p.k + j], *MOE_CHECKED(y + (size_t)j * p.H, 4, p.y, bytes), sum);
    }
    const float *y = p.y + ((size_t)A * p.ne + t) * p.H + c;
    for (int q = 0; q < p.ns; ++q) sum += *MOE_CHECKED(y + (size_t)q * p.T * p.H, 4, p.y, bytes);
    *MOE_CHECKED(p.out + i, 2, p.out, (size_t)p.T * p.H * 2) = (uint16_t)f32_to_bf16_rne(sum);
}

// S: steps in each wave's ring.  WINDOW: of the token rows in gate/up (FewUnits).
template <int F, int S, int WINDOW>
__global__ __launch_bounds__(kFewThreads) void few_layer_kernel(FewArgs p) {
    __shared__ FewSmem sm;
    if (threadIdx.x == 0) sm.ticket = (int)ctr_ticket(p, kRouter);
    __syncthreads();
    for (int t = uniform(sm.ticket); (uint32_t)t < (uint32_t)p.n_router;) {
        few_router(p, sm, t);
        // (publication and the next ticket in one branch of thread 0, with barriers on either side: two such
        // branches with no barrier between them, as at the end and the start of a loop's body, may be joined by
        // the compiler across the back edge, which lets the other lanes run ahead)
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) {
            ctr_done(p, kRouter, p.n_router);
            sm.ticket = (int)ctr_ticket(p, kRouter);
        }
        __syncthreads();
        t = uniform(sm.ticket);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t a = ctr_ticket(p, kGateUp), b = ctr_ticket(p, kDown);
        sm.ticket = (int)a;
        sm.down = (int)b;
    }
    if constexpr (WINDOW == 0) few_stage_x<F>(p, sm.area + kFewWaves * S * FewStep<F>::SLOT);
    __syncthreads();
    int t = uniform(sm.ticket);
    const int d = uniform(sm.down);
    bool selected = false;
    for (;;) {
        const bool share = (uint32_t)t < (uint32_t)p.n_gu;
        if (share && p.I_sh) {   // needs no routing
            few_gateup<F, S, WINDOW>(p, sm, true, p.I_sh / 8, t);
            __syncthreads();   // the sums in LDS are free
        }
        if (!selected) few_select(p, sm, t == 0);
        selected = true;
        if (!share) break;
        // the next ticket, early: none is left unless a workgroup has not started yet
        if (threadIdx.x == 0) sm.ticket = (int)ctr_ticket(p, kGateUp);
        few_gateup<F, S, WINDOW>(p, sm, false, uniform(sm.n_experts) * (p.I / 8), t);
        publish(p, kGateUp, p.n_gu);
        t = uniform(sm.ticket);
        __syncthreads();
        if ((uint32_t)t >= (uint32_t)p.n_gu) break;
    }
    if ((uint32_t)d < (uint32_t)p.n_down) {
        if (p.columns) few_down_items<F, true>(p, sm, d);
        else few_down_items<F, false>(p, sm, d);
    }
    if (!p.columns) {
        int c = 0;
        for (bool have_y = false;; have_y = true) {
            __syncthreads();
            if (threadIdx.x == 0) {
                sm.ticket = (int)ctr_ticket(p, kCombine);
                if (!have_y && (uint32_t)sm.ticket < (uint32_t)p.n_combine) wait_done(p, kDown);
            }
            __syncthreads();
            c = uniform(sm.ticket);
            if ((uint32_t)c >= (uint32_t)p.n_combine) break;
            few_combine(p, sm, c);
        }
    }
    // the last workgroup to leave clears the counters for the next call
    __syncthreads();
    if (threadIdx.x == 0) sm.ticket = ctr_add(p.ctr + kCtrLine * kCtrExit) == gridDim.x - 1;
    __syncthreads();
    if (sm.ticket && threadIdx.x < kCtrWords / kCtrLine)
        __hip_atomic_store(p.ctr + kCtrLine * threadIdx.x, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Steps in a ring: the deepest that leaves the token rows room (bf16 or 4-bit,
// by slot size), else the one that leaves room for windows of them.  A short
// ring next to whole rows is better than a deep one next to windows, which cost
// a barrier each and leave the last units unsplit: 16 tokens, hidden 2816, bf16
// with MLP 183 us (3 steps) against 190 (6 steps; h in one part); 12 tokens, hidden 4096,
// NVFP4 74 (2) against 83 (4).  Windows against rows read from global memory, 16
// tokens, hidden 5120: bf16 178 us against 230, MXFP4 95 against 153.
constexpr int kRings = 3, kRing[2][kRings + 1] = {{7, 5, 3, 6}, {6, 4, 2, 4}}, kWindow[2] = {8, 4};

struct FewPlan {
    int ring;      // of kRing
    bool columns;
    int PW, ne, ns;
    size_t y;      // floats of the products' workspace
};

int few_slot(int f) { return f == kFewBf16 ? FewStep<kFewBf16>::SLOT : FewStep<kFewMx>::SLOT; }
static_assert(FewStep<kFewMx>::SLOT == FewStep<kFewNv>::SLOT, "one ring for both");

FewPlan few_plan(int f, int T, int H, int k, int I, int I_sh) {
    FewPlan g{};
    const int *rings = kRing[f != kFewBf16], step = f == kFewBf16 ? FewStep<kFewBf16>::K * 2 : FewStep<kFewMx>::K * 2;
    auto rest = [&](int i) { return kFewArea - kFewWaves * rings[i] * few_slot(f); };
    while (g.ring < kRings && (long long)few_steps(f, H) * step * T > rest(g.ring)) ++g.ring;
    // segments of which T rows of h fit
    const int most = ((kFewArea - kFewWaves * few_down_ring(f) * few_slot(f)) / T - 16) / (2 * step), st = few_steps(f, I), want = (st + most - 1) / most;
    g.PW = (st + want - 1) / want;
    g.ne = (st + g.PW - 1) / g.PW;
    g.ns = (few_steps(f, I_sh) + g.PW - 1) / g.PW;
    // Column blocks need all rows of h in every workgroup and use H / 16 of them, but no combine phase: hidden
    // 2816, top-8, one token 36.8 us in bf16 and 28.4 in MXFP4 against 41.4 and 32.5 with shared units, two tokens
    // 49.9 and 37.3 against 51.4 and 38.8; three tokens 66.1 and 42.4 against 63.7 and 39.5.
    g.columns = T * k <= 16;
    g.y = g.columns ? 0 : ((size_t)T * k * g.ne + (size_t)T * g.ns) * H;
    return g;
}

template <int F, int R = 0>
void launch_format(const FewArgs &p, int ring, int blocks, hipStream_t st) {
    constexpr int S = kRing[F != kFewBf16][R], W = R == kRings ? kWindow[F != kFewBf16] : 0;
    static_assert(2 * W * FewStep<F>::FRAGS * 64 * kFewTokens <= kFewArea - kFewWaves * S * FewStep<F>::SLOT, "windows");
    static_assert((kFewArea - kFewWaves * few_down_ring(F) * FewStep<F>::SLOT) / kFewTokens >= 16 + FewStep<F>::K * 4,
                  "a segment is one step or more");
    if (ring == R) {
        few_layer_kernel<F, S, W><<<blocks, kFewThreads, 0, st>>>(p);
        return;
    }
    if constexpr (R < kRings) launch_format<F, R + 1>(p, ring, blocks, st);
}

int few_format(WeightFormat f) { return f == WeightFormat::kBF16 ? kFewBf16 : f == WeightFormat::kMXFP4 ? kFewMx : kFewNv; }

}  // namespace

size_t few_layer_y(WeightFormat fmt, int T, int H, int k, int I, int I_sh) {
    return few_plan(few_format(fmt), T, H, k, I, I_sh).y * sizeof(float);
}

hipError_t launch_few_layer(const FewLayer &l, hipStream_t st) {
    FewArgs p{};
    p.x = l.x;
    p.wr = l.w_router;
    p.bias = l.bias;
    p.wgu = static_cast<const uint8_t *>(l.gate_up.w);
    p.gus = l.gate_up.scales;
    p.gug = l.gate_up.global;
    p.wd = static_cast<const uint8_t *>(l.down.w);
    p.ds = l.down.scales;
    p.dg = l.down.global;
    p.swgu = static_cast<const uint8_t *>(l.sh_gate_up.w);
    p.sgus = l.sh_gate_up.scales;
    p.sgug = l.sh_gate_up.global;
    p.swd = static_cast<const uint8_t *>(l.sh_down.w);
    p.sds = l.sh_down.scales;
    p.sdg = l.sh_down.global;
    p.out = l.out;
    p.ids = l.ids;
    p.wts = l.w;
    p.ctr = l.counters;
    p.logits = l.logits;
    p.h = l.h;
    p.h_sh = l.h_sh;
    p.y = l.y;
    p.T = l.T;
    p.H = l.H;
    p.E = l.E;
    p.k = l.k;
    p.I = l.I;
    p.I_sh = l.I_sh;
    // a workgroup per CU (its LDS fills one), fewer where there are fewer items
    constexpr int kBlocks = 256;
    const long long units = (long long)std::min(l.E, l.T * l.k) * (l.I / 8);   // at most
    p.n_router = (l.E + 3) / 4;
    p.n_gu = (int)std::min<long long>(kBlocks, std::max<long long>(units, l.I_sh / 8));
    const int f = few_format(l.fmt);
    const FewPlan g = few_plan(f, l.T, l.H, l.k, l.I, l.I_sh);
    p.columns = g.columns;
    p.PW = g.PW;
    p.ne = g.ne;
    p.ns = g.ns;
    // (no item is empty: k experts at least are touched)
    p.n_down = g.columns ? l.H / 16 : std::min(kBlocks, (l.k * g.ne + g.ns) * (l.H / 16));
    p.n_combine = (l.T * l.H + kFewThreads - 1) / kFewThreads;
    const int blocks = std::min(kBlocks, std::max(p.n_router, std::max(p.n_gu, p.n_down)));
    switch (f) {
        case kFewBf16: launch_format<kFewBf16>(p, g.ring, blocks, st); break;
        case kFewMx: launch_format<kFewMx>(p, g.ring, blocks, st); break;
        default: launch_format<kFewNv>(p, g.ring, blocks, st);
    }
    return hipGetLastError();
}

#ifdef MOE_DEBUG
MOE_DEBUG_READER(debug_read_few)
#endif

}  // namespace moe
