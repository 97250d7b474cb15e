// The whole MoE layer for up to 16 tokens in one launch (moe_forward_few).
//
// With few tokens the layer is a stream of expert weights: each touched
// expert's gate/up and down matrices are read once and multiplied with every
// token (few_stream.h), so the bytes bound it and launches and waits are the
// rest of its time.  One persistent grid runs three phases:
//
//   router   logits = x W_r^T (+ b), four experts per work item, summed as
//            moe_route does (fp32 chunks of 256, added in fp64), so both give
//            the same bits
//   gate/up  every workgroup selects the experts itself (top-k of the few
//            tokens from the logits), then h = gelu_tanh(g) * u for its share
//            of the (expert, 8 columns) units, rounded to bf16
//   down     out[t][16 columns] = sum over experts of w[t, e] * (W_d h): the
//            routing weights multiply the fp32 sums, experts are added in a
//            fixed order, and out is rounded once
//
// Each phase's items are handed out by a ticket counter.  A workgroup takes
// router items while there are any, then gate/up shares, then down items, and
// waits only for items of an earlier phase, all of which have then been taken
// by workgroups that are running: every wait ends, whatever else runs on the
// GPU and however few workgroups are resident.
#include <algorithm>

#include "few_stream.h"
#include "moe_launch.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;
constexpr int kFewMaxA = kFewTokens * 32;                 // assignments (k <= 32)
constexpr int kFewArea = 136 * 1024;                      // LDS for the rings and the token rows

// Counters in the workspace's zeroed prefix, a line each.
constexpr int kCtrRouterTicket = 0, kCtrGateUpTicket = 32, kCtrDownTicket = 64;   // next item of each phase
constexpr int kCtrRouter = 96, kCtrGateUp = 128, kCtrExit = 160;                    // items done, workgroups left

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
    uint16_t *h, *h_sh;                         // [T k][I], [T][I_sh]
    int T, H, E, k, I, I_sh;
    int n_router, n_gu, n_down;                 // items of each phase
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

// Counts this workgroup's stored results: every wave's stores are complete,
// then one thread counts.
__device__ __forceinline__ void publish(uint32_t *done) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) ctr_add(done);
}

// One thread waits until `n` workgroups have published; its workgroup, which
// joins a barrier next, may then load what they stored: the caches'
// invalidation is complete, not merely requested, before the others load.
// The count is reached as long as the counters were zero before the launch;
// the bound only keeps a workspace that was not from holding the GPU (its
// results are then undefined).
__device__ __forceinline__ void wait_count(uint32_t *ctr, uint32_t n) {
    for (int i = 0; i < (1 << 20); ++i) {
        if (__hip_atomic_load(ctr, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= n) break;
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
    if (threadIdx.x == 0) wait_count(p.ctr + kCtrRouter, p.n_router);
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
// The token operand of MFMA f, lane (r, g): from LDS, where every fragment
// has 16 bytes per (g, token), or from the rows of x.
template <int F, bool XL>
__device__ __forceinline__ u32x4 few_x_frag(const FewArgs &p, const uint8_t *xs, int f, int r, int g) {
    const int t = min(r, p.T - 1);
    if constexpr (XL) return *reinterpret_cast<const u32x4 *>(xs + 64 * f * p.T + (g * p.T + t) * 16);
    const int k = few_frag_k<F>(f, g);
    u32x4 v = *reinterpret_cast<const u32x4 *>(
        MOE_CHECKED(p.x + (size_t)t * p.H + (k < p.H ? k : 0), 16, p.x, (size_t)p.T * p.H * 2));
    return k < p.H ? v : u32x4{0u, 0u, 0u, 0u};
}

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

// Units u0 .. u1 - 1 of eight h columns: the MFMA's rows are the unit's eight
// gate rows and the matching eight up rows.  The workgroup takes 8 / KW units
// at a time, KW waves splitting the K of each.
template <int F, int S, bool XL>
__device__ __forceinline__ void few_gateup(const FewArgs &p, FewSmem &sm, bool shared, int u0, int u1) {
    constexpr int SLOT = FewStep<F>::SLOT, OPS = FewStep<F>::OPS, FRAGS = FewStep<F>::FRAGS;
    const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
    const int I = shared ? p.I_sh : p.I, H = p.H, per = I / 8;
    if (u0 >= u1) return;
    const int ns = few_steps(F, H), KW = few_kwaves(u1 - u0, ns), UG = kFewWaves / KW;
    const int kw = wave % KW, s0 = kw * ns / KW, s1 = (kw + 1) * ns / KW;
    const uint8_t *w = shared ? p.swgu : p.wgu, *s = shared ? p.sgus : p.gus;
    const FewLane<F> ln(H);
    const size_t wn = (size_t)(shared ? 1 : p.E) * 2 * I * ln.pitch, sn = (size_t)(shared ? 1 : p.E) * 2 * I * ln.spitch;
    // (a unit's scale rows start at a multiple of 4 bytes)
    const uint32_t lo = (ln.r & 7) * ln.spitch;
    uint8_t *ring = sm.area + wave * S * SLOT;
    const uint8_t *xs = sm.area + kFewWaves * S * SLOT;

    // the step to request next: of unit lu, and where that unit's rows are
    int lu = u0 + wave / KW, ls = s0, lslot = 0;
    FewRows<F> rows;
    auto point = [&]() {
        const int ue = lu / per;
        const size_t row = (size_t)(shared ? 0 : uniform(sm.expert[ue])) * 2 * I + 8 * (lu - ue * per);
        rows.top = w + row * ln.pitch;
        rows.low = rows.top + (size_t)I * ln.pitch;
        rows.stop = s + row * ln.spitch;
        rows.slow = rows.stop + (size_t)I * ln.spitch;
    };
    auto request = [&]() {
        ln.issue(rows, ls, ring + lslot * SLOT, w, wn, s, sn);
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
    int slot = 0;
    for (int v0 = u0; v0 < u1; v0 += UG) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        if (uniform(v0 + wave / KW < u1)) {
            for (int st = s0; st < s1; ++st) {
                const uint8_t *q = ring + slot * SLOT;
                // the ring is full but for this step's successors: S - 1 steps may be in flight
                if (uniform(lu < u1)) few_wait<(S - 1) * OPS>();
                else few_wait<0>();
                if constexpr (F == kFewBf16) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        acc = mfma16x16x32(ln.load(q, i), few_x_frag<F, XL>(p, xs, st * FRAGS + i, r, g), acc);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const u32x4 c = ln.load(q, h);
                        const uint32_t sc = ln.scale(q, st, h, lo);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc = mfma16x16x32(few_operand<F>(c, sc, i),
                                               few_x_frag<F, XL>(p, xs, st * FRAGS + 4 * h + i, r, g), acc);
                    }
                }
                few_lds_done();
                if (uniform(lu < u1)) request();
                slot = slot + 1 == S ? 0 : slot + 1;
            }
        }
        sm.red[wave][lane] = acc;
        __syncthreads();
        // wave v finishes unit v0 + v: lane 4 t + i has token t and columns 2i, 2i + 1.  Lane 16 (m / 4) + t,
        // element m % 4 of each wave's sums is weight row m, token t: gate rows 0..7, up rows 8..15
        const int u = v0 + wave;
        if (uniform(wave < UG && u < u1)) {
            const int i = 2 * (lane & 3), t = lane >> 2, ue = u / per;
            float gate[2] = {0.f, 0.f}, up[2] = {0.f, 0.f};
            for (int v = 0; v < KW; ++v) {
                const float *a = reinterpret_cast<const float *>(&sm.red[wave * KW + v][16 * (i >> 2) + t]) + (i & 3);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    gate[q] += a[q];
                    up[q] += a[4 * 32 + q];
                }
            }
            if constexpr (F == kFewNv) {
                const float m = shared ? p.sgug[0] : p.gug[uniform(sm.expert[ue])];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    gate[q] *= m;
                    up[q] *= m;
                }
            }
            const uint32_t hv = pack_bf16x2(gelu_tanh(gate[0]) * up[0], gelu_tanh(gate[1]) * up[1]);
            const int j = t < p.T ? (shared ? 1 : (int)sm.slot[ue][t]) : 0;
            if (j) {
                uint16_t *base = shared ? p.h_sh : p.h;
                const size_t row = shared ? (size_t)t : (size_t)t * p.k + j - 1;
                store_shared(reinterpret_cast<uint32_t *>(MOE_CHECKED(base + row * I + 8 * (u - ue * per) + i, 4, base,
                                                                      (size_t)p.T * (shared ? 1 : p.k) * I * 2)), hv);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- down
// Sixteen output columns per item, summed over sub-units: the touched experts
// (or K pieces of them, where sixteen of their rows do not fit the LDS), then
// the dense MLP in pieces of the same size.  The waves take sub-units in turn
// and their sums are added in wave order.  h is staged in LDS for as many
// sub-units as fit (a pass); the ring's first weights of a pass are requested
// before its h is staged, those of the first one before h exists.
template <int F, int S>
struct FewPieces {
    // LDS for rows of h, and the largest piece of which sixteen fit
    static constexpr int H_BYTES = kFewArea - kFewWaves * S * FewStep<F>::SLOT;
    static constexpr int MAX = (H_BYTES / kFewTokens - 16) / (FewStep<F>::K * 2);
    static_assert(MAX >= 1, "one step of sixteen rows fits");
    int PW, pitch, ne, ns, U, T, A, n;   // steps of a piece, bytes of a row of it, pieces of an expert, of the MLP
    __device__ __forceinline__ FewPieces(const FewArgs &p, int n_experts) {
        const int st = few_steps(F, p.I), want = (st + MAX - 1) / MAX;
        PW = (st + want - 1) / want;
        pitch = PW * FewStep<F>::K * 2 + 16;
        ne = (st + PW - 1) / PW;
        ns = p.I_sh ? (few_steps(F, p.I_sh) + PW - 1) / PW : 0;
        U = n_experts;
        T = p.T;
        A = p.T * p.k;
        n = U * ne + ns;
    }
    // rows of h of the sub-units before v
    __device__ __forceinline__ int rows_before(const FewSmem &sm, int v) const {
        if (v >= U * ne) return A * ne + (v - U * ne) * T;
        const int e = v / ne, q = v - e * ne, f = sm.first[e];
        return f * ne + q * (sm.first[e + 1] - f);
    }
};

template <int F, int S>
__device__ __forceinline__ void few_down_items(const FewArgs &p, FewSmem &sm, int item) {
    constexpr int SLOT = FewStep<F>::SLOT, OPS = FewStep<F>::OPS, FRAGS = FewStep<F>::FRAGS, KS = FewStep<F>::K;
    using P = FewPieces<F, S>;
    const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
    const P pc(p, uniform(sm.n_experts));
    const int UE = pc.U * pc.ne;
    uint8_t *ring = sm.area + wave * S * SLOT;
    uint8_t *hs = sm.area + kFewWaves * S * SLOT;

    int va = 0, vb = 0;              // the pass: sub-units va .. vb - 1
    int lv = 0, ls = 0, ls1 = 0, lslot = 0;   // next step to request: of sub-unit lv
    FewRows<F> rows;
    auto steps = [&](int v, int &a, int &b) {   // steps [a, b) of its row that sub-unit v covers
        const int q = v < UE ? v % pc.ne : v - UE;
        a = q * pc.PW;
        b = min(few_steps(F, v < UE ? p.I : p.I_sh), a + pc.PW);
    };
    auto point = [&]() {
        const bool mlp = lv >= UE;
        const size_t row = (size_t)(mlp ? 0 : uniform(sm.expert[lv / pc.ne])) * p.H + 16 * item;
        const FewLane<F> ln(mlp ? p.I_sh : p.I);
        rows.top = (mlp ? p.swd : p.wd) + row * ln.pitch;
        rows.low = rows.top + (size_t)8 * ln.pitch;
        rows.stop = (mlp ? p.sds : p.ds) + row * ln.spitch;
        rows.slow = rows.stop + (size_t)8 * ln.spitch;
        steps(lv, ls, ls1);
    };
    auto request = [&]() {
        uint8_t *q = ring + lslot * SLOT;
        const bool mlp = lv >= UE;
        const FewLane<F> ln(mlp ? p.I_sh : p.I);
        const size_t nr = (size_t)(mlp ? 1 : p.E) * p.H;
        ln.issue(rows, ls, q, mlp ? p.swd : p.wd, nr * ln.pitch, mlp ? p.sds : p.ds, nr * ln.spitch);
        lslot = lslot + 1 == S ? 0 : lslot + 1;
        if (++ls == ls1) {
            lv += kFewWaves;
            if (lv < vb) point();
        }
    };
    // the next pass, as many sub-units as fit, and its first requests
    auto next_pass = [&](int from) {
        va = from;
        const int base = pc.rows_before(sm, va), most = P::H_BYTES / pc.pitch;
        vb = va;
        for (;;) {   // 64 candidates at a time; the rows only grow
            const int v = vb + 1 + lane;
            const int fit = __popcll(__ballot(v <= pc.n && pc.rows_before(sm, min(v, pc.n)) - base <= most));
            vb += fit;
            if (fit < 64) break;
        }
        vb = uniform(vb);
        lv = va + wave;
        lslot = 0;
        if (lv < vb) {
            point();
            for (int i = 0; i < S && lv < vb; ++i) request();
        }
    };
    for (bool have_h = false;;) {
        f32x4 out = {0.f, 0.f, 0.f, 0.f};
        int next = 0;
        for (int from = 0; from < pc.n; from = vb) {
            // wave 0 polls for h, and loads return in order: its first weights only after that
            if (wave != 0 || have_h) next_pass(from);
            if (from == 0) {
                if (threadIdx.x == 0) {
                    if (!have_h) wait_count(p.ctr + kCtrGateUp, p.n_gu);
                    sm.down = (int)ctr_add(p.ctr + kCtrDownTicket);
                }
                __syncthreads();
                next = uniform(sm.down);
                if (wave == 0 && !have_h) next_pass(from);
                have_h = true;
            }
            // stage the pass's rows of h: sub-unit by sub-unit, its rows in token order
            const int base = pc.rows_before(sm, va);
            for (int v = va + wave; v < vb; v += kFewWaves) {
                const bool mlp = v >= UE;
                const int e = v / pc.ne, f = mlp ? 0 : uniform(sm.first[e]);
                const int nr = mlp ? p.T : uniform(sm.first[e + 1]) - f, I = mlp ? p.I_sh : p.I;
                int a, b;
                steps(v, a, b);
                const int valid = (min(I, b * KS) - a * KS) / 8, all = (b - a) * (KS / 8);   // 16-byte pieces of a row
                uint8_t *dst = hs + (size_t)(uniform(pc.rows_before(sm, v)) - base) * pc.pitch;
                for (int i = 0; i < nr; ++i, dst += pc.pitch) {
                    const uint16_t *hb = mlp ? p.h_sh : p.h;
                    const uint16_t *src = hb + (size_t)(mlp ? i : uniform(sm.sorted[f + i])) * I + a * KS;
                    for (int c = 0; c < all; c += 64) {
                        if (c + lane < valid)
                            dma16<false>(MOE_CHECKED(src + 8 * (c + lane), 16, hb, (size_t)p.T * (mlp ? 1 : p.k) * I * 2),
                                         dst + 16 * c);
                        else if (c + lane < all)   // past the row: the codes there count nothing
                            *reinterpret_cast<u32x4 *>(dst + 16 * (c + lane)) = u32x4{0u, 0u, 0u, 0u};
                    }
                }
            }
            few_wait<0>();
            __syncthreads();
            int slot = 0;
            for (int v = va + wave; v < vb; v += kFewWaves) {
                const bool mlp = v >= UE;
                const int e = v / pc.ne;
                int a, b;
                steps(v, a, b);
                // this lane's row: its token's, or, where that is not routed here, the first one (left out below)
                int j = r < p.T, rank = r;
                if (!mlp) {
                    j = sm.slot[e][r];
                    rank = few_count(*reinterpret_cast<const u32x4 *>(sm.slot[e]), r);
                }
                const uint8_t *hr = hs + (size_t)(pc.rows_before(sm, v) - base + (j ? rank : 0)) * pc.pitch;
                const FewLane<F> ln(mlp ? p.I_sh : p.I);
                const uint32_t lo = (ln.r & 7) * ln.spitch;
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
                for (int st = a; st < b; ++st) {
                    const uint8_t *q = ring + slot * SLOT;
                    if (uniform(lv < vb)) few_wait<(S - 1) * OPS>();
                    else few_wait<0>();
                    const uint8_t *hk = hr + 2 * KS * (st - a);
                    if constexpr (F == kFewBf16) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            acc = mfma16x16x32(ln.load(q, i), *reinterpret_cast<const u32x4 *>(hk + 2 * few_frag_k<F>(i, g)),
                                               acc);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const u32x4 c = ln.load(q, h);
                            const uint32_t sc = ln.scale(q, st, h, lo);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc = mfma16x16x32(
                                    few_operand<F>(c, sc, i),
                                    *reinterpret_cast<const u32x4 *>(hk + 2 * few_frag_k<F>(4 * h + i, g)), acc);
                        }
                    }
                    few_lds_done();
                    if (uniform(lv < vb)) request();
                    slot = slot + 1 == S ? 0 : slot + 1;
                }
                float f = mlp ? 1.f : sm.w[j ? r * p.k + j - 1 : 0];
                if constexpr (F == kFewNv) f *= mlp ? p.sdg[0] : p.dg[uniform(sm.expert[e])];
#pragma unroll
                for (int q = 0; q < 4; ++q) out[q] = j ? fmaf(f, acc[q], out[q]) : out[q];
            }
            if (vb < pc.n) __syncthreads();   // the rows of h are free
        }
        sm.red[wave][lane] = out;
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
        item = next;
        if ((uint32_t)item >= (uint32_t)p.n_down) return;
    }
    static_assert(FRAGS * 32 == KS);
}

// S: steps in each wave's ring.  XL: the token rows fit the LDS next to the rings.
template <int F, int S, bool XL>
__global__ __launch_bounds__(kFewThreads) void few_layer_kernel(FewArgs p) {
    __shared__ FewSmem sm;
    if (threadIdx.x == 0) sm.ticket = (int)ctr_add(p.ctr + kCtrRouterTicket);
    __syncthreads();
    for (int t = uniform(sm.ticket); (uint32_t)t < (uint32_t)p.n_router;) {
        few_router(p, sm, t);
        // (publication and the next ticket in one branch of thread 0, with barriers on either side: two such
        // branches with no barrier between them, as at the end and the start of a loop's body, may be joined by
        // the compiler across the back edge, which lets the other lanes run ahead)
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) {
            ctr_add(p.ctr + kCtrRouter);
            sm.ticket = (int)ctr_add(p.ctr + kCtrRouterTicket);
        }
        __syncthreads();
        t = uniform(sm.ticket);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t a = ctr_add(p.ctr + kCtrGateUpTicket), b = ctr_add(p.ctr + kCtrDownTicket);
        sm.ticket = (int)a;
        sm.down = (int)b;
    }
    if constexpr (XL) few_stage_x<F>(p, sm.area + kFewWaves * S * FewStep<F>::SLOT);
    __syncthreads();
    int t = uniform(sm.ticket);
    const int d = uniform(sm.down);
    bool selected = false;
    for (;;) {
        const bool share = (uint32_t)t < (uint32_t)p.n_gu;
        if (share && p.I_sh) {   // needs no routing
            const int units = p.I_sh / 8;
            few_gateup<F, S, XL>(p, sm, true, share_start(t, units, p.n_gu), share_start(t + 1, units, p.n_gu));
        }
        if (!selected) few_select(p, sm, t == 0);
        selected = true;
        if (!share) break;
        // the next ticket, early: none is left unless a workgroup has not started yet
        if (threadIdx.x == 0) sm.ticket = (int)ctr_add(p.ctr + kCtrGateUpTicket);
        const int units = uniform(sm.n_experts) * (p.I / 8);
        few_gateup<F, S, XL>(p, sm, false, share_start(t, units, p.n_gu), share_start(t + 1, units, p.n_gu));
        publish(p.ctr + kCtrGateUp);
        t = uniform(sm.ticket);
        __syncthreads();
        if ((uint32_t)t >= (uint32_t)p.n_gu) break;
    }
    if ((uint32_t)d < (uint32_t)p.n_down) few_down_items<F, S>(p, sm, d);
    // the last workgroup to leave clears the counters for the next call
    if (threadIdx.x == 0 && ctr_add(p.ctr + kCtrExit) == gridDim.x - 1) {
        const int all[6] = {kCtrRouterTicket, kCtrGateUpTicket, kCtrDownTicket, kCtrRouter, kCtrGateUp, kCtrExit};
        for (int c : all) __hip_atomic_store(p.ctr + c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// The deepest of three rings that leaves the token rows room; rows that are
// too long for any are read from global memory.
template <int F, int S0, int S1, int S2>
void launch_format(const FewArgs &p, int blocks, hipStream_t st) {
    const size_t x = (size_t)few_steps(F, p.H) * FewStep<F>::K * 2 * p.T;
    auto fits = [&](int s) { return x <= (size_t)(kFewArea - kFewWaves * s * FewStep<F>::SLOT); };
    const dim3 grid(blocks), block(kFewThreads);
    if (fits(S0)) few_layer_kernel<F, S0, true><<<grid, block, 0, st>>>(p);
    else if (fits(S1)) few_layer_kernel<F, S1, true><<<grid, block, 0, st>>>(p);
    else if (fits(S2)) few_layer_kernel<F, S2, true><<<grid, block, 0, st>>>(p);
    else few_layer_kernel<F, S1, false><<<grid, block, 0, st>>>(p);
}

}  // namespace

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
    p.n_down = l.H / 16;
    const int blocks = std::min(kBlocks, std::max(p.n_router, std::max(p.n_gu, p.n_down)));
    switch (l.fmt) {
        case WeightFormat::kBF16: launch_format<kFewBf16, 7, 5, 3>(p, blocks, st); break;
        case WeightFormat::kMXFP4: launch_format<kFewMx, 5, 4, 2>(p, blocks, st); break;
        default: launch_format<kFewNv, 5, 4, 2>(p, blocks, st);
    }
    return hipGetLastError();
}

#ifdef MOE_DEBUG
MOE_DEBUG_READER(debug_read_few)
#endif

}  // namespace moe
