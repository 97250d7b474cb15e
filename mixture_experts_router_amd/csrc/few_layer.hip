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
#include <type_traits>

#include "few_stream.h"
#include "moe_launch.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;
constexpr int kFewXBytes = 96 * 1024;                     // token rows in LDS
constexpr int kFewBatch = 4;                              // gate/up units reduced together
constexpr int kFewMaxA = kFewTokens * 32;                 // assignments (k <= 32)

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
    uint8_t x[kFewXBytes];                      // token operands, in MFMA order
    f32x4 red[kFewBatch][kFewWaves][64];        // partial sums of the waves
    int32_t ids[kFewMaxA];
    float w[kFewMaxA];
    uint8_t slot[kFewMaxA][kFewTokens];         // [touched expert][token]: slot + 1, 0 = not routed there
    int16_t expert[kFewMaxA];                   // touched experts, ascending
    int16_t index[1024];                        // expert -> touched index (or -1)
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

// The routing of every token, by each workgroup for itself: ids and weights,
// the touched experts in ascending order and who goes there.
__device__ void few_select(const FewArgs &p, FewSmem &sm, bool store) {
    const int wave = wave_index(), lane = threadIdx.x & 63, A = p.T * p.k;
    for (int i = threadIdx.x; i < p.E; i += kFewThreads) sm.index[i] = -1;
    for (int i = threadIdx.x; i < A * kFewTokens / 4; i += kFewThreads) reinterpret_cast<uint32_t *>(sm.slot)[i] = 0u;
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
    for (int a = threadIdx.x; a < A; a += kFewThreads) sm.index[sm.ids[a]] = 0;
    __syncthreads();
    if (wave == 0) {
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 64) {
            const bool on = e0 + lane < p.E && sm.index[e0 + lane] >= 0;
            const uint64_t m = __ballot(on);
            const int at = n + __popcll(m & ((1ull << lane) - 1));
            if (on) {
                sm.index[e0 + lane] = (int16_t)at;
                sm.expert[at] = (int16_t)(e0 + lane);
            }
            n += __popcll(m);
        }
        if (lane == 0) sm.n_experts = n;
    }
    __syncthreads();
    for (int a = threadIdx.x; a < A; a += kFewThreads)
        sm.slot[sm.index[sm.ids[a]]][a / p.k] = (uint8_t)(a % p.k + 1);
    __syncthreads();
}

// ---------------------------------------------------------------- gate/up
// The token operand of MFMA f, lane (r, g): from LDS, where every fragment
// has 16 bytes per (g, token), or from the rows of x.
template <int F, bool XL>
__device__ __forceinline__ u32x4 few_x_frag(const FewArgs &p, const FewSmem &sm, int f, int r, int g) {
    const int t = min(r, p.T - 1);
    if constexpr (XL) return *reinterpret_cast<const u32x4 *>(sm.x + 64 * f * p.T + (g * p.T + t) * 16);
    const int k = few_frag_k<F>(f, g);
    if (k >= p.H) return u32x4{0u, 0u, 0u, 0u};
    return *reinterpret_cast<const u32x4 *>(MOE_CHECKED(p.x + (size_t)t * p.H + k, 16, p.x, (size_t)p.T * p.H * 2));
}

template <int F>
__device__ void few_stage_x(const FewArgs &p, FewSmem &sm) {
    const int nfrag = few_blocks(F, p.H) * FewBlock<F>::STEPS;
    for (int i = threadIdx.x; i < nfrag * 4 * p.T; i += kFewThreads) {
        const int t = i % p.T, fg = i / p.T, k = few_frag_k<F>(fg >> 2, fg & 3);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (k < p.H)
            v = *reinterpret_cast<const u32x4 *>(MOE_CHECKED(p.x + (size_t)t * p.H + k, 16, p.x, (size_t)p.T * p.H * 2));
        *reinterpret_cast<u32x4 *>(sm.x + (size_t)i * 16) = v;
    }
    __syncthreads();
}

// Weight pieces travel from HBM to the MFMAs through a ring of register
// chunks of CB blocks, one consumed while the others are in flight.  Within a
// turn of the ring no branch holds a load (past the end of a row, or of the
// work, the last block is loaded again), so the compiler's waits can count the
// loads and leave the ring full; the last turn loads nothing.
template <int F>
struct FewRing {
    static constexpr int CB = F == kFewBf16 ? 6 : 3;      // blocks of a chunk
    static constexpr int GU = F == kFewBf16 ? 3 : 4;      // chunks in the gate/up's ring
    static constexpr int DN = 4, DH = 2;                  // in the down's: weights, h
};

// Units u0 .. u1 - 1 of eight h columns: the MFMA's rows are the unit's eight
// gate rows and the matching eight up rows; the waves split K.
template <int F, bool XL>
__device__ __forceinline__ void few_gateup(const FewArgs &p, FewSmem &sm, bool shared, int u0, int u1) {
    constexpr int STEPS = FewBlock<F>::STEPS, CB = FewRing<F>::CB, N = FewRing<F>::GU;
    if (u0 >= u1) return;
    const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
    const int I = shared ? p.I_sh : p.I, H = p.H, per = I / 8;
    const int nb = few_blocks(F, H), b0 = wave * nb / kFewWaves, b1 = (wave + 1) * nb / kFewWaves;
    const int nch = ((nb + kFewWaves - 1) / kFewWaves + CB - 1) / CB;   // chunks of a unit, in every wave
    const size_t pitch = F == kFewBf16 ? (size_t)H * 2 : (size_t)H / 2, spitch = F == kFewMx ? H / 32 : H / 16;
    const uint8_t *w = shared ? p.swgu : p.wgu, *s = shared ? p.sgus : p.gus;
    [[maybe_unused]] const size_t rows = (size_t)(shared ? 1 : p.E) * 2 * I;
    const size_t my_row = r < 8 ? r : I + r - 8;

    // the unit being loaded: this lane's weight and scale rows, next chunk
    int lu = u0, lch = 0, le = u0 / per, lc = u0 - le * per;
    const int last = max(b1 - 1, 0);
    const uint8_t *wrow, *srow;
    auto point = [&]() {
        const size_t row = (size_t)(shared ? 0 : uniform(sm.expert[le])) * 2 * I + 8 * lc + my_row;
        wrow = w + row * pitch;
        srow = s + row * spitch;
    };
    u32x4 c[N][CB];
    uint32_t sc[N][CB];
    auto load = [&](int i) {
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            const int b = min(b0 + lch * CB + j, last);
            c[i][j] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4 *>(MOE_CHECKED(wrow + few_piece<F>(b, g, H), 16, w, rows * pitch)));
            if constexpr (F != kFewBf16) sc[i][j] = few_scale<F>(srow, b, g, H, s, rows * spitch);
        }
        if (lch + 1 < nch) {
            ++lch;
        } else if (lu + 1 < u1) {
            lch = 0;
            ++lu;
            if (++lc == per) {
                lc = 0;
                ++le;
            }
            point();
        }
    };
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    int cu = u0, cch = 0, held = 0;   // the unit being summed; units whose sums are in LDS
    auto finish = [&]() {
        sm.red[held][wave][lane] = acc;
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
        if (++held < kFewBatch && cu + 1 < u1) return;
        __syncthreads();
        // wave v finishes held unit v: lane 4 t + i has token t and columns 2i, 2i + 1.  Lane 16 (m / 4) + t,
        // element m % 4 of each wave's sums is weight row m, token t: gate rows 0..7, up rows 8..15
        if (uniform(wave < held)) {
            const int i = 2 * (lane & 3), t = lane >> 2, u = cu + 1 - held + wave, ue = u / per;
            float gate[2] = {0.f, 0.f}, up[2] = {0.f, 0.f};
#pragma unroll
            for (int v = 0; v < kFewWaves; ++v) {
                const float *a = reinterpret_cast<const float *>(&sm.red[wave][v][16 * (i >> 2) + t]) + (i & 3);
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
        held = 0;
        __syncthreads();
    };
    point();
#pragma unroll
    for (int i = 0; i < N; ++i) load(i);
    auto turn = [&](auto more) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int j = 0; j < CB; ++j) {
                const int b = b0 + cch * CB + j;
                if (uniform(b < b1))
#pragma unroll
                    for (int q = 0; q < STEPS; ++q)
                        acc = mfma16x16x32(few_operand<F>(c[i][j], F == kFewBf16 ? 0u : sc[i][j], q),
                                           few_x_frag<F, XL>(p, sm, b * STEPS + q, r, g), acc);
            }
            if constexpr (decltype(more)::value) load(i);
            if (++cch == nch) {
                if (cu < u1) finish();
                cch = 0;
                ++cu;
            }
        }
    };
    for (int left = ((u1 - u0) * nch - 1) / N; left > 0; --left) turn(std::true_type{});
    turn(std::false_type{});
}

// ---------------------------------------------------------------- down
// Sixteen output columns per item: the waves take the touched experts in turn
// (the dense MLP in pieces of about an expert's size), and their sums are
// added in wave order.  The ring's first weights are requested before h
// exists; h (from L2) has a ring of its own.  A lane whose token is not routed
// to the expert multiplies another token's row, whose sums it leaves out.
template <int F>
__device__ __forceinline__ void few_down_items(const FewArgs &p, FewSmem &sm, int item) {
    constexpr int STEPS = FewBlock<F>::STEPS, CB = FewRing<F>::CB, N = FewRing<F>::DN, M = FewRing<F>::DH;
    const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
    const int U = uniform(sm.n_experts), pb = few_blocks(F, p.I);
    const int n = U + (p.I_sh ? (few_blocks(F, p.I_sh) + pb - 1) / pb : 0);   // sub-units: experts, pieces of the dense MLP
    // blocks [b0, b1) of sub-unit v, whose rows are `width` values
    auto span = [&](int v, int &b0, int &b1, int &width) {
        width = v < U ? p.I : p.I_sh;
        b0 = v < U ? 0 : (v - U) * pb;
        b1 = min(few_blocks(F, width), b0 + pb);
    };
    // slot + 1 of this lane's token in sub-unit v (0: not routed there)
    auto route = [&](int v) -> int { return r < p.T ? (v >= U ? 1 : (int)sm.slot[v][r]) : 0; };

    u32x4 c[N][CB], h[M][CB][STEPS];
    uint32_t sc[N][CB];
    // the sub-unit whose weights are being loaded: its next block, its end
    int lv = 0, lb = 0, lb1 = 0, lI = 0;
    const uint8_t *wrow = nullptr, *srow = nullptr;
    [[maybe_unused]] const uint8_t *wbase = nullptr, *sbase = nullptr;
    [[maybe_unused]] size_t wbytes = 0, sbytes = 0;
    auto point = [&]() {
        const bool shared = lv >= U;
        span(lv, lb, lb1, lI);
        const size_t row = (size_t)(shared ? 0 : uniform(sm.expert[lv])) * p.H + 16 * item + r;
        const size_t pitch = F == kFewBf16 ? (size_t)lI * 2 : (size_t)lI / 2, spitch = F == kFewMx ? lI / 32 : lI / 16;
        wbase = shared ? p.swd : p.wd;
        sbase = shared ? p.sds : p.ds;
        wbytes = (size_t)(shared ? 1 : p.E) * p.H * pitch;
        sbytes = (size_t)(shared ? 1 : p.E) * p.H * spitch;
        wrow = wbase + row * pitch;
        srow = sbase + row * spitch;
    };
    auto load = [&](int i) {
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            const int b = min(lb + j, lb1 - 1);
            c[i][j] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4 *>(MOE_CHECKED(wrow + few_piece<F>(b, g, lI), 16, wbase, wbytes)));
            if constexpr (F != kFewBf16) sc[i][j] = few_scale<F>(srow, b, g, lI, sbase, sbytes);
        }
        if (lb + CB < lb1) {
            lb += CB;
        } else if (lv + kFewWaves < n) {
            lv += kFewWaves;
            point();
        }
    };
    auto start = [&]() {
        lv = wave;
        if (lv >= n) return;
        point();
#pragma unroll
        for (int i = 0; i < N; ++i) load(i);
    };
    // the sub-unit whose h is being loaded, and this lane's h row (where its
    // token is not routed there, the row of one that is)
    int hv = 0, hb = 0, hb1 = 0, hI = 0;
    const uint16_t *hrow = nullptr;
    [[maybe_unused]] const uint16_t *hbase = nullptr;
    [[maybe_unused]] size_t hbytes = 0;
    auto point_h = [&]() {
        const bool shared = hv >= U;
        span(hv, hb, hb1, hI);
        const int j = route(hv), mine = shared ? r : r * p.k + j - 1;
        const int other = __builtin_amdgcn_readlane(mine, (int)__builtin_ctzll(__ballot(j != 0) | (1ull << 63)));
        hbase = shared ? p.h_sh : p.h;
        hbytes = (size_t)p.T * (shared ? 1 : p.k) * hI * 2;
        hrow = hbase + (size_t)(j ? mine : other) * hI;
    };
    auto load_h = [&](int i) {
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            const int b = min(hb + j, hb1 - 1);
#pragma unroll
            for (int q = 0; q < STEPS; ++q) {
                const int k = few_frag_k<F>(b * STEPS + q, g);
                h[i][j][q] = *reinterpret_cast<const u32x4 *>(MOE_CHECKED(hrow + (k < hI ? k : 0), 16, hbase, hbytes));
            }
        }
        if (hb + CB < hb1) {
            hb += CB;
        } else if (hv + kFewWaves < n) {
            hv += kFewWaves;
            point_h();
        }
    };

    for (bool have_h = false;;) {
        // wave 0 polls for h, and loads return in order: its weights only after that
        if (wave != 0) start();
        if (threadIdx.x == 0) {
            if (!have_h) wait_count(p.ctr + kCtrGateUp, p.n_gu);
            sm.down = (int)ctr_add(p.ctr + kCtrDownTicket);
        }
        have_h = true;
        __syncthreads();
        if (wave == 0) start();
        const int next = uniform(sm.down);
        f32x4 out = {0.f, 0.f, 0.f, 0.f};
        if (wave < n) {
            hv = wave;
            point_h();
#pragma unroll
            for (int i = 0; i < M; ++i) load_h(i);
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
            int cv = wave, cb, cb1, cI;
            span(cv, cb, cb1, cI);
            auto turn = [&](auto more) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
#pragma unroll
                    for (int j = 0; j < CB; ++j) {
                        if (uniform(cb + j < cb1)) {
                            u32x4 cw = c[i][j];
                            if constexpr (F != kFewBf16) {
                                // codes past the row (the last block of an odd number of half blocks) count as zero
                                if (128 * (cb + j) + 32 * g >= cI) cw = u32x4{0u, 0u, 0u, 0u};
                            }
#pragma unroll
                            for (int q = 0; q < STEPS; ++q)
                                acc = mfma16x16x32(few_operand<F>(cw, F == kFewBf16 ? 0u : sc[i][j], q), h[i % M][j][q], acc);
                        }
                    }
                    if constexpr (decltype(more)::value) load(i);
                    if (decltype(more)::value || i + M < N) load_h(i % M);
                    cb += CB;
                    if (cb >= cb1 && cv < n) {
                        const int j = route(cv);
                        float f = cv >= U ? 1.f : sm.w[j ? r * p.k + j - 1 : 0];
                        if constexpr (F == kFewNv) f *= cv >= U ? p.sdg[0] : p.dg[uniform(sm.expert[cv])];
#pragma unroll
                        for (int q = 0; q < 4; ++q) out[q] = j ? fmaf(f, acc[q], out[q]) : out[q];
                        acc = f32x4{0.f, 0.f, 0.f, 0.f};
                        cv += kFewWaves;
                        if (cv < n) span(cv, cb, cb1, cI);
                    }
                }
            };
            int chunks = 0;
            for (int v = wave; v < n; v += kFewWaves) {
                int v0, v1, vI;
                span(v, v0, v1, vI);
                chunks += (v1 - v0 + CB - 1) / CB;
            }
            for (int left = (chunks - 1) / N; left > 0; --left) turn(std::true_type{});
            turn(std::false_type{});
        }
        sm.red[0][wave][lane] = out;
        __syncthreads();
        if (threadIdx.x < 256) {
            const int m = threadIdx.x & 15, t = threadIdx.x >> 4;
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < kFewWaves; ++v) sum += sm.red[0][v][16 * (m >> 2) + t][m & 3];
            if (t < p.T)
                *MOE_CHECKED(p.out + (size_t)t * p.H + 16 * item + m, 2, p.out, (size_t)p.T * p.H * 2) =
                    (uint16_t)f32_to_bf16_rne(sum);
        }
        __syncthreads();   // the sums and the ticket in LDS are free
        item = next;
        if ((uint32_t)item >= (uint32_t)p.n_down) return;
    }
}

// XL: the token rows fit the LDS.
template <int F, bool XL>
__global__ __launch_bounds__(kFewThreads) void few_layer_kernel(FewArgs p) {
    __shared__ FewSmem sm;
    const int wave = wave_index();
    // tickets: a router item (then more, while there are any), then a gate/up
    // share and a down item together
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
    if constexpr (XL) few_stage_x<F>(p, sm);
    __syncthreads();
    int t = uniform(sm.ticket);
    const int d = uniform(sm.down);
    if (p.I_sh && (uint32_t)t < (uint32_t)p.n_gu) {   // needs no routing
        const int units = p.I_sh / 8;
        few_gateup<F, XL>(p, sm, true, share_start(t, units, p.n_gu), share_start(t + 1, units, p.n_gu));
    }
    few_select(p, sm, t == 0);
    for (bool first = true; (uint32_t)t < (uint32_t)p.n_gu; first = false) {
        // the next ticket, early: none is left unless a workgroup has not started yet
        if (threadIdx.x == 0) sm.ticket = (int)ctr_add(p.ctr + kCtrGateUpTicket);
        if (!first && p.I_sh) {
            const int units = p.I_sh / 8;
            few_gateup<F, XL>(p, sm, true, share_start(t, units, p.n_gu), share_start(t + 1, units, p.n_gu));
        }
        const int units = uniform(sm.n_experts) * (p.I / 8);
        few_gateup<F, XL>(p, sm, false, share_start(t, units, p.n_gu), share_start(t + 1, units, p.n_gu));
        publish(p.ctr + kCtrGateUp);
        t = uniform(sm.ticket);
        __syncthreads();
    }
    if ((uint32_t)d < (uint32_t)p.n_down) few_down_items<F>(p, sm, d);
    // the last workgroup to leave clears the counters for the next call
    if (threadIdx.x == 0 && ctr_add(p.ctr + kCtrExit) == gridDim.x - 1) {
        const int all[6] = {kCtrRouterTicket, kCtrGateUpTicket, kCtrDownTicket, kCtrRouter, kCtrGateUp, kCtrExit};
        for (int c : all) __hip_atomic_store(p.ctr + c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
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
    const dim3 grid(blocks), block(kFewThreads);
    const bool fits = ((size_t)l.H + 127) / 128 * 256 * l.T <= kFewXBytes;
    switch (l.fmt) {
        case WeightFormat::kBF16:
            if (fits) few_layer_kernel<kFewBf16, true><<<grid, block, 0, st>>>(p);
            else few_layer_kernel<kFewBf16, false><<<grid, block, 0, st>>>(p);
            break;
        case WeightFormat::kMXFP4:
            if (fits) few_layer_kernel<kFewMx, true><<<grid, block, 0, st>>>(p);
            else few_layer_kernel<kFewMx, false><<<grid, block, 0, st>>>(p);
            break;
        default:
            if (fits) few_layer_kernel<kFewNv, true><<<grid, block, 0, st>>>(p);
            else few_layer_kernel<kFewNv, false><<<grid, block, 0, st>>>(p);
    }
    return hipGetLastError();
}

#ifdef MOE_DEBUG
MOE_DEBUG_READER(debug_read_few)
#endif

}  // namespace moe
