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
// Work items are handed out by a ticket counter, router items first, then
// gate/up, then down.  A workgroup waits only for items of an earlier phase,
// and all of those have been taken by workgroups that are running when a
// later ticket is handed out: every wait ends, whatever else runs on the GPU
// and however few workgroups are resident.
#include <algorithm>

#include "few_stream.h"
#include "moe_launch.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int kFewWaves = 8;
constexpr int kFewXBytes = 128 * 1024;                    // token rows in LDS
constexpr int kFewMaxA = kFewTokens * 32;                 // assignments (k <= 32)

// Counters in the workspace's zeroed prefix, a line each.
constexpr int kCtrTicket = 0, kCtrRouter = 32, kCtrGateUp = 64, kCtrExit = 96;

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
    int n_router, n_gu_sh, n_gu, n_down;        // tickets of each kind
};

struct FewSmem {
    uint8_t x[kFewXBytes];                      // token operands, in MFMA order
    f32x4 red[2][kFewWaves][64];                // partial sums of the waves
    int32_t ids[kFewMaxA];
    float w[kFewMaxA];
    uint8_t slot[kFewMaxA][kFewTokens];         // [touched expert][token]: slot + 1, 0 = not routed there
    int16_t expert[kFewMaxA];                   // touched experts, ascending
    int16_t index[1024];                        // expert -> touched index (or -1)
    int n_experts;
    int ticket;
};
static_assert(sizeof(FewSmem) <= 160 * 1024, "LDS of one workgroup");

__device__ __forceinline__ uint32_t ctr_add(uint32_t *p) {
    return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Publishes what this workgroup has written: every wave's stores are
// complete, then one thread makes them visible device-wide and counts.
__device__ __forceinline__ void publish(uint32_t *ctr) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        ctr_add(ctr);
    }
}

// Waits until `n` workgroups have published.  The count is reached as long as
// the counters were zero before the launch; the bound only keeps a workspace
// that was not from holding the GPU (its results are then undefined).
__device__ __forceinline__ void wait_for(uint32_t *ctr, uint32_t n) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < (1 << 22); ++i) {
            if (__hip_atomic_load(ctr, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= n) break;
            __builtin_amdgcn_s_sleep(1);
        }
        __threadfence();
    }
    __syncthreads();
}

// ---------------------------------------------------------------- router
// Four experts, all tokens: wave w takes chunks w, w + 8, ... of 256 K
// values, each summed in fp32 by MFMAs in K order; one thread per (token,
// expert) adds the chunk sums in fp64 in chunk order.
__device__ void few_router(const FewArgs &p, FewSmem &sm, int item) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int e0 = 4 * item, nchunks = (p.H + 255) / 256;
    const bool on_e = r < 4 && e0 + r < p.E, on_t = r < p.T;
    f32x4(*sum)[kFewTokens] = reinterpret_cast<f32x4(*)[kFewTokens]>(sm.red);   // [16 chunks][token]
    const int et = threadIdx.x >> 4, tt = threadIdx.x & 15;                       // of the adding threads (< 64)
    double total = 0.0;
    for (int c0 = 0; c0 < nchunks; c0 += 2 * kFewWaves) {
        for (int cc = wave; cc < 2 * kFewWaves && c0 + cc < nchunks; cc += kFewWaves) {
            const int k0 = (c0 + cc) * 256, n = min(256, p.H - k0) / 32;
            u32x4 a[8], b[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int k = k0 + 32 * (u < n ? u : 0) + 8 * g;
                a[u] = on_e ? *reinterpret_cast<const u32x4 *>(
                                  MOE_CHECKED(p.wr + (size_t)(e0 + r) * p.H + k, 16, p.wr, (size_t)p.E * p.H * 2))
                            : u32x4{0u, 0u, 0u, 0u};
                b[u] = on_t ? *reinterpret_cast<const u32x4 *>(
                                  MOE_CHECKED(p.x + (size_t)r * p.H + k, 16, p.x, (size_t)p.T * p.H * 2))
                            : u32x4{0u, 0u, 0u, 0u};
            }
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (u < n) acc = mfma16x16x32(a[u], b[u], acc);
            if (g == 0) sum[cc][r] = acc;
        }
        __syncthreads();
        if (threadIdx.x < 64)
            for (int c = 0; c < 2 * kFewWaves && c0 + c < nchunks; ++c) total += (double)sum[c][tt][et];
        __syncthreads();
    }
    if (threadIdx.x < 64 && tt < p.T && e0 + et < p.E) {
        const double b = p.bias ? (double)p.bias[e0 + et] : 0.0;
        *MOE_CHECKED(p.logits + (size_t)tt * p.E + e0 + et, 4, p.logits, (size_t)p.T * p.E * 4) = (float)(total + b);
    }
    publish(p.ctr + kCtrRouter);
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
    wait_for(p.ctr + kCtrRouter, p.n_router);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, A = p.T * p.k;
    for (int i = threadIdx.x; i < 1024; i += blockDim.x) sm.index[i] = -1;
    for (int i = threadIdx.x; i < kFewMaxA * kFewTokens / 4; i += blockDim.x) reinterpret_cast<uint32_t *>(sm.slot)[i] = 0u;
    for (int t = wave; t < p.T; t += kFewWaves) {
        if (p.E <= 64) few_topk<1>(p, sm, t, store);
        else if (p.E <= 128) few_topk<2>(p, sm, t, store);
        else if (p.E <= 256) few_topk<4>(p, sm, t, store);
        else if (p.E <= 512) few_topk<8>(p, sm, t, store);
        else few_topk<16>(p, sm, t, store);
    }
    __syncthreads();
    for (int a = threadIdx.x; a < A; a += blockDim.x) sm.index[sm.ids[a]] = 0;
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
    for (int a = threadIdx.x; a < A; a += blockDim.x)
        sm.slot[sm.index[sm.ids[a]]][a / p.k] = (uint8_t)(a % p.k + 1);
    __syncthreads();
}

// ---------------------------------------------------------------- gate/up
// The token operand of MFMA f, lane (r, g): from LDS, where every fragment
// has 16 bytes per (g, token), or from the rows of x.
template <int F>
__device__ __forceinline__ u32x4 few_x_frag(const FewArgs &p, const FewSmem &sm, bool in_lds, int f, int r, int g) {
    const int t = min(r, p.T - 1);
    if (in_lds) return *reinterpret_cast<const u32x4 *>(sm.x + ((size_t)(f * 4 + g) * p.T + t) * 16);
    const int k = few_frag_k<F>(f, g);
    if (k >= p.H) return u32x4{0u, 0u, 0u, 0u};
    return *reinterpret_cast<const u32x4 *>(MOE_CHECKED(p.x + (size_t)t * p.H + k, 16, p.x, (size_t)p.T * p.H * 2));
}

template <int F>
__device__ void few_stage_x(const FewArgs &p, FewSmem &sm) {
    const int nfrag = few_blocks(F, p.H) * FewBlock<F>::STEPS;
    for (int i = threadIdx.x; i < nfrag * 4 * p.T; i += blockDim.x) {
        const int t = i % p.T, fg = i / p.T, k = few_frag_k<F>(fg >> 2, fg & 3);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (k < p.H)
            v = *reinterpret_cast<const u32x4 *>(MOE_CHECKED(p.x + (size_t)t * p.H + k, 16, p.x, (size_t)p.T * p.H * 2));
        *reinterpret_cast<u32x4 *>(sm.x + (size_t)i * 16) = v;
    }
    __syncthreads();
}

// Units u0 .. u1 - 1 of eight h columns: the MFMA's rows are the unit's eight
// gate rows and the matching eight up rows; the waves split K.
template <int F>
__device__ void few_gateup(const FewArgs &p, FewSmem &sm, bool shared, bool in_lds, int u0, int u1) {
    constexpr int STEPS = FewBlock<F>::STEPS;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int I = shared ? p.I_sh : p.I, H = p.H;
    const int nb = few_blocks(F, H), b0 = wave * nb / kFewWaves, b1 = (wave + 1) * nb / kFewWaves;
    const size_t pitch = F == kFewBf16 ? (size_t)H * 2 : (size_t)H / 2, spitch = F == kFewMx ? H / 32 : H / 16;
    const uint8_t *w = shared ? p.swgu : p.wgu, *s = shared ? p.sgus : p.gus;
    [[maybe_unused]] const size_t rows = (size_t)(shared ? 1 : p.E) * 2 * I;
    for (int u = u0; u < u1; ++u) {
        const int ue = u / (I / 8), c0 = (u - ue * (I / 8)) * 8;
        const int e = shared ? 0 : sm.expert[ue];
        const size_t row = (size_t)e * 2 * I + (r < 8 ? c0 + r : I + c0 + r - 8);
        const uint8_t *wrow = w + row * pitch, *srow = s + row * spitch;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int b = b0; b < b1; ++b) {
            const u32x4 c = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4 *>(MOE_CHECKED(wrow + few_piece<F>(b, g, H), 16, w, rows * pitch)));
            const uint32_t sc = few_scale<F>(srow, b, g, H, s, rows * spitch);
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
                acc = mfma16x16x32(few_operand<F>(c, sc, i), few_x_frag<F>(p, sm, in_lds, b * STEPS + i, r, g), acc);
        }
        f32x4(*red)[64] = sm.red[u & 1];
        red[wave][lane] = acc;
        few_lds_barrier();
        // lane 16 (m / 4) + t, element m % 4 of each wave's sums: weight row m, token t
        if (threadIdx.x < 128) {
            const int c = threadIdx.x & 7, t = threadIdx.x >> 3;
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int v = 0; v < kFewWaves; ++v) {
                gate += red[v][16 * (c >> 2) + t][c & 3];
                up += red[v][16 * (2 + (c >> 2)) + t][c & 3];
            }
            if constexpr (F == kFewNv) {
                const float m = (shared ? p.sgug : p.gug)[e];
                gate *= m;
                up *= m;
            }
            const uint16_t hv = (uint16_t)f32_to_bf16_rne(gelu_tanh(gate) * up);
            if (t < p.T) {
                if (shared) {
                    *MOE_CHECKED(p.h_sh + (size_t)t * I + c0 + c, 2, p.h_sh, (size_t)p.T * I * 2) = hv;
                } else if (const int j = sm.slot[ue][t]) {
                    *MOE_CHECKED(p.h + ((size_t)t * p.k + j - 1) * I + c0 + c, 2, p.h, (size_t)p.T * p.k * I * 2) = hv;
                }
            }
        }
    }
    publish(p.ctr + kCtrGateUp);
}

// ---------------------------------------------------------------- down
// Sixteen output columns: the waves take the touched experts in turn (the
// dense MLP in pieces of about an expert's size), and their sums are added in
// wave order.
template <int F>
__device__ void few_down(const FewArgs &p, FewSmem &sm, int item) {
    constexpr int STEPS = FewBlock<F>::STEPS, KB = FewBlock<F>::K;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int U = sm.n_experts;
    const int pb = few_blocks(F, p.I), np = p.I_sh ? (few_blocks(F, p.I_sh) + pb - 1) / pb : 0;   // blocks of a piece, pieces
    f32x4 out = {0.f, 0.f, 0.f, 0.f};
    for (int v = wave; v < U + np; v += kFewWaves) {
        const bool shared = v >= U;
        const int I = shared ? p.I_sh : p.I, e = shared ? 0 : sm.expert[v], nb = few_blocks(F, I);
        const int b0 = shared ? (v - U) * pb : 0, b1 = shared ? min(nb, b0 + pb) : nb;
        const size_t pitch = F == kFewBf16 ? (size_t)I * 2 : (size_t)I / 2, spitch = F == kFewMx ? I / 32 : I / 16;
        const uint8_t *w = shared ? p.swd : p.wd, *s = shared ? p.sds : p.ds;
        const size_t row = (size_t)e * p.H + 16 * item + r;
        [[maybe_unused]] const size_t rows = (size_t)(shared ? 1 : p.E) * p.H;
        const uint8_t *wrow = w + row * pitch, *srow = s + row * spitch;
        const int j = shared ? 1 : sm.slot[v][r];             // lane (r, g)'s token r: its slot + 1
        const bool on = r < p.T && j;
        const uint16_t *hb = shared ? p.h_sh : p.h;
        const uint16_t *hrow = hb + (on ? (shared ? (size_t)r : (size_t)r * p.k + j - 1) * I : 0);
        [[maybe_unused]] const size_t hbytes = (size_t)p.T * (shared ? 1 : p.k) * I * 2;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int b = b0; b < b1; ++b) {
            const u32x4 c = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4 *>(MOE_CHECKED(wrow + few_piece<F>(b, g, I), 16, w, rows * pitch)));
            const uint32_t sc = few_scale<F>(srow, b, g, I, s, rows * spitch);
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int k = few_frag_k<F>(b * STEPS + i, g);
                u32x4 hv = {0u, 0u, 0u, 0u};
                if (on && (KB == 32 || k < I))
                    hv = *reinterpret_cast<const u32x4 *>(MOE_CHECKED(hrow + k, 16, hb, hbytes));
                acc = mfma16x16x32(few_operand<F>(c, sc, i), hv, acc);
            }
        }
        float f = shared ? 1.f : sm.w[on ? r * p.k + j - 1 : 0];
        if constexpr (F == kFewNv) f *= (shared ? p.sdg : p.dg)[e];
        if (on)
#pragma unroll
            for (int q = 0; q < 4; ++q) out[q] = fmaf(f, acc[q], out[q]);
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
}

template <int F>
__global__ __launch_bounds__(64 * kFewWaves) void few_layer_kernel(FewArgs p) {
    __shared__ FewSmem sm;
    const int n1 = p.n_router, n2 = n1 + p.n_gu_sh, n3 = n2 + p.n_gu, n4 = n3 + p.n_down;
    const bool in_lds = (size_t)few_blocks(F, p.H) * FewBlock<F>::K * 2 * p.T <= kFewXBytes;
    bool staged = false, selected = false, have_h = false;
    for (;;) {
        __syncthreads();   // the LDS of the previous item is free
        if (threadIdx.x == 0) sm.ticket = (int)ctr_add(p.ctr + kCtrTicket);
        __syncthreads();
        const int t = sm.ticket;
        if (t >= n4 || t < 0) break;
        if (t < n1) {
            few_router(p, sm, t);
            continue;
        }
        if (t < n3 && !staged && in_lds) {
            few_stage_x<F>(p, sm);
            staged = true;
        }
        if (t >= n2 && !selected) {
            few_select(p, sm, t == n2);
            selected = true;
        }
        if (t < n3) {
            const bool shared = t < n2;
            const int i = shared ? t - n1 : t - n2, n = shared ? p.n_gu_sh : p.n_gu;
            const int units = shared ? p.I_sh / 8 : sm.n_experts * (p.I / 8);
            few_gateup<F>(p, sm, shared, in_lds, (int)((long long)i * units / n), (int)((long long)(i + 1) * units / n));
            continue;
        }
        if (!have_h) {
            wait_for(p.ctr + kCtrGateUp, p.n_gu_sh + p.n_gu);
            have_h = true;
        }
        few_down<F>(p, sm, t - n3);
    }
    // the last workgroup to leave clears the counters for the next call
    if (threadIdx.x == 0 && ctr_add(p.ctr + kCtrExit) == gridDim.x - 1) {
        const int all[4] = {kCtrTicket, kCtrRouter, kCtrGateUp, kCtrExit};
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
    p.n_gu_sh = l.I_sh ? std::min(kBlocks, l.I_sh / 8) : 0;
    p.n_gu = (int)std::min<long long>(kBlocks, units);
    p.n_down = l.H / 16;
    const int blocks = std::min(kBlocks, std::max(std::max(p.n_router, p.n_gu), std::max(p.n_gu_sh, p.n_down)));
    switch (l.fmt) {
        case WeightFormat::kBF16: few_layer_kernel<kFewBf16><<<blocks, 64 * kFewWaves, 0, st>>>(p); break;
        case WeightFormat::kMXFP4: few_layer_kernel<kFewMx><<<blocks, 64 * kFewWaves, 0, st>>>(p); break;
        default: few_layer_kernel<kFewNv><<<blocks, 64 * kFewWaves, 0, st>>>(p); break;
    }
    return hipGetLastError();
}

#ifdef MOE_DEBUG
MOE_DEBUG_READER(debug_read_few)
#endif

}  // namespace moe
