// moe_layer.cu -- a whole mixture-of-experts layer for a few tokens (decoding).
//
//   l = Wr x         s = softmax(l) or logistic(l)      the topk experts by s (+ bias)
//   u_e = g1_e W1_e x     h_e = act(u_e)  or  act(gate) * up      y = sum_e w_e g2_e W2_e h_e
//
// Weights are NVFP4 (E2M1 codes, E4M3 scales per 16, one fp32 scale per expert), tokens
// bf16.  Bound by reading the chosen experts' weights once, 4.5 bits each.  Launches: the
// router, the first and the second projection, the weighted sum.
//
// A code times its block scale has at most 6 significant bits and lies in 2^-10 ..
// 2688: exact in fp16, which the hardware decodes two codes at a time.  The activations
// are held in fp16 too, each row scaled by a power of two to a maximum in [2^14, 2^15):
// bf16 rows then lose nothing above 2^-32 of their maximum.  The fp32 rows between the
// projections are split, v = hi + 2^-11 lo with hi = fp16(v) and lo = fp16(2^11 (v - hi)):
// 2^-22 of a value, or 2^-50 of its row's maximum, is all that is lost (hi alone: 2^-11,
// which showed in y as a relative difference of 9e-4).  The products go through mma.m16n8k16
// with 16 weight rows as M and 8 columns as N, accumulated in fp32; a column is a token, in
// the second projection one of a token's two parts, side by side, so that one thread holds
// both sums.
//
// Measured (calls in a graph): 64 experts of 2048 x 1024, top 4: 22 us for 1 token, 54 us for
// 16 (146 MB of weights: 22 us at 6.5 TB/s); 128 experts of 4096 x 2048, top 8, 64 tokens:
// 404 us for 1.8 GB (274 us), the projections 233 and 137 us at 5.1 and 4.3 TB/s; 8 such
// experts, top 2, 64 tokens: 142 us.  What bounds it: few tokens, the chain of four launches;
// many, issue slots (56% busy with four warps a scheduler, the latencies of decoding and MMA
// covered in part); more tokens an expert than shared memory holds rows, further passes over
// its weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cmath>

#include "activation.cuh"

namespace nvfp4 {

__device__ __forceinline__ void grid_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------- router
constexpr int kRouteCluster = 8;  // CTAs that share a group of tokens
constexpr int kRouteThreads = 256, kRouteWarps = kRouteThreads / 32;

__device__ __forceinline__ void store_remote_f64(const void* local, uint32_t cta, double v) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(local)), "r"(cta));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at), "d"(v) : "memory");
}

// The cluster's barrier for warps whose lanes may be apart (a loop or a store that not all
// lanes took comes before): without .aligned each thread arrives for itself.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// An integer whose order is the number's, both zeros alike, NaN below -infinity.
__device__ __forceinline__ long long order_of(double v) {
    const long long b = __double_as_longlong(v + 0.0);
    return v != v ? LLONG_MIN : b < 0 ? b ^ LLONG_MAX : b;
}

// A cluster takes TC tokens.  Logits: a warp takes an expert and the cluster's tokens;
// products of eight elements are added in fp32, those sums in fp64, so that the choice
// does not hang on the order of the additions or on the batch.  The logits of token r go
// to CTA r, which picks its experts after a cluster barrier: an expert's place is the
// number of experts before it (larger key, or equal and of lower index; NaN comes last).
template <int TC>
__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads)
    moe_route_kernel(const MoeLayerParams p) {
    __shared__ double logit[kMaxGroups];
    __shared__ long long key[kMaxGroups];
    __shared__ int chosen[kMoeMaxTopk];
    __shared__ double red[kRouteWarps];
    __shared__ uint32_t amax;
    const int rank = blockIdx.x % kRouteCluster, t0 = blockIdx.x / kRouteCluster * TC;
    const int nt = p.T - t0 < TC ? p.T - t0 : TC;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    cluster_arrive();  // this CTA runs
    grid_dependents();
    if (threadIdx.x == 0) amax = 0;
    for (int i = blockIdx.x * kRouteThreads + threadIdx.x; i < p.T * p.topk; i += gridDim.x * kRouteThreads)
        p.h_amax[i] = 0;
    bool joined = false;
    for (int e = rank * kRouteWarps + warp; e < p.E; e += kRouteCluster * kRouteWarps) {
        double acc[TC];
#pragma unroll
        for (int t = 0; t < TC; ++t) acc[t] = 0.0;
        const uint16_t* w = p.router + (int64_t)e * p.K;
        const uint16_t* x = p.x + (int64_t)t0 * p.K;
#pragma unroll 4
        for (int k = lane * 8; k < p.K; k += 256) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(w + k));
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int t = 0; t < TC; ++t) {
                // tokens past the batch repeat the last one; their sums are not stored
                const uint4 b = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)(t < nt ? t : nt - 1) * p.K + k));
                const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s = fmaf(bf16_lo(aw[i]), bf16_lo(bw[i]), s);
                    s = fmaf(bf16_hi(aw[i]), bf16_hi(bw[i]), s);
                }
                acc[t] += (double)s;
            }
        }
#pragma unroll
        for (int t = 0; t < TC; ++t)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xFFFFFFFFu, acc[t], o);
        if (!joined) {
            cluster_wait();
            joined = true;
        }
#pragma unroll
        for (int t = 0; t < TC; ++t)
            if (t < nt && lane == t) store_remote_f64(logit + e, (uint32_t)t, acc[t]);
    }
    if (!joined) cluster_wait();
    cluster_arrive();
    cluster_wait();
    if (rank >= nt) return;
    const int t = t0 + rank;
    uint32_t big = 0;  // the row's largest |x|, as integers: their order, NaN largest
    for (int k = threadIdx.x * 8; k < p.K; k += kRouteThreads * 8) {
        const uint4 b = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.K + k));
        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) big = max(big, max((bw[i] << 16) & 0x7FFF0000u, bw[i] & 0x7FFF0000u));
    }
    big = __reduce_max_sync(0xFFFFFFFFu, big);
    if (lane == 0) atomicMax(&amax, big);
    double sum = 0.0, top = 0.0;
    if (!p.sigmoid && (p.sel_bias != nullptr || !p.renormalize)) {  // the softmax over all experts
        top = -INFINITY;
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) top = fmax(top, logit[e]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (lane == 0) red[warp] = top;
        __syncthreads();
        for (int i = 0; i < kRouteWarps; ++i) top = fmax(top, red[i]);
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) sum += exp(logit[e] - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) red[warp] = sum;
        __syncthreads();
        sum = 0.0;
        for (int i = 0; i < kRouteWarps; ++i) sum += red[i];
    }
    // without a bias the logits themselves give the order
    bool nan = false;
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
        double k = logit[e];
        nan |= k != k;
        if (p.sel_bias != nullptr)
            k = (p.sigmoid ? 1.0 / (1.0 + exp(-k)) : exp(k - top) / sum) + (double)p.sel_bias[e];
        key[e] = order_of(k);
    }
    const bool any_nan = __syncthreads_or(nan);
    int parts = 1;  // threads that count for one expert
    while (parts < 32 && p.E * parts * 2 <= kRouteThreads) parts *= 2;
    for (int e0 = 0; e0 < p.E; e0 += kRouteThreads / parts) {
        const int e = e0 + threadIdx.x / parts;
        const long long k = e < p.E ? key[e] : 0;
        int place = 0;
        for (int o = threadIdx.x % parts; o < p.E; o += parts) place += key[o] > k || (key[o] == k && o < e) ? 1 : 0;
        for (int o = 1; o < parts; o <<= 1) place += __shfl_xor_sync(0xFFFFFFFFu, place, o);
        if (e < p.E && place < p.topk) chosen[place] = e;
    }
    __syncthreads();
    if (threadIdx.x == 0) p.x_amax[t] = amax;
    if (threadIdx.x < p.topk) {
        const int j = threadIdx.x, e = chosen[j];
        double first = logit[chosen[0]];  // the largest chosen logit
        for (int i = 1; i < p.topk; ++i) first = fmax(first, logit[chosen[i]]);
        // The weights go through fp32 exponentials of logits (softmax: of their differences)
        // rounded to fp32: off by 2^-24 of the exponent and a few ulp, far below y's 2^-8.
        // Scores that are to be renormalized may share a factor: the softmax's total, and
        // e^first where the largest logistic is below a half, or all could vanish in fp32.
        const bool low = p.sigmoid && p.renormalize && first < 0.0;
        auto score = [&](int c) {
            const float l = (float)logit[c];
            if (p.sigmoid && !low) return 1.0f / (1.0f + expf(-l));
            const float r = expf((float)(logit[c] - first));
            return low ? r / (1.0f + expf(l)) : r;
        };
        float s = score(e);
        if (p.renormalize) {
            float total = 0.0f;
            for (int i = 0; i < p.topk; ++i) total += score(chosen[i]);
            s /= total;
        } else if (!p.sigmoid) {
            s = (float)(exp(logit[e] - top) / sum);
        }
        if (!p.sigmoid && any_nan) s = __uint_as_float(0x7FFFFFFFu);  // one NaN spoils a softmax
        p.idx[t * p.topk + j] = e;
        p.weight[t * p.topk + j] = s * p.route_scale;
    }
}

// ---------------------------------------------------------------- expert projections
// A persistent CTA per SM, sixteen warps.  Its work is a contiguous range of (expert,
// tile) pairs (kCountedItems says how long), a tile being 32 weight rows (gated: 16 gate rows and the 16 up rows they
// multiply); the part of the range that lies in one expert is a segment, walked once per
// pass of up to `cap` tokens, whose rows are held in shared memory.  A warp takes a whole
// tile, 128 columns at a time: two 16-row MMA tiles, which share the tokens' fragments.
// Each lane copies the codes that it will read itself (and two scale words that its warp
// shares) into a ring of stages with asynchronous copies, a ring's depth ahead, over the
// borders of tiles, passes and segments: nothing is handed over between warps, so a
// stage is refilled the moment it is in registers.  When fewer tiles than warps are left,
// ks warps split a tile's columns and join their sums in order.
//   First projection of 64 tokens, 128 experts of 4096 x 2048: 233 us; 378 while every CTA had
// as many (expert, tile) pairs whatever the experts' tokens, against which: refilled after the
// arithmetic: 397.  Stages filled by TMA from producer threads, four warps to a stage: 434
// (264 with the arithmetic left out, but the way from use to refill is longer).  Weights
// decoded into tensor memory for tcgen05 fp16 MMAs: 536 (130 cycles for each M = 128, N =
// 16 MMA).  All warps on one tile, for contiguous reads: above 560 (a join per tile).
constexpr int kExpWarps = 16, kExpThreads = kExpWarps * 32;
constexpr int kMaxTiles = 4;            // 8-column tiles of one pass
// Share of the work.  From this many items a CTA on, where experts have unlike numbers of
// tokens, an item counts as its passes over the weights plus its 8-column tiles; with fewer,
// what counts is how many tiles a CTA's warps have to split at a time, and every item counts
// alike.  Measured, alike and counted (us): 64 tokens, 128 experts of 4096 x 2048, top 8
// (110 items a CTA) 633 and 400; 128 tokens, 64 of 1024 x 1024, top 8 (14 to 28) 110 and 93;
// 64 tokens, 8 of 4096 x 2048, top 2 (7) 178 and 143; 32 tokens, 16 of 2048 x 1024, top 4 (7)
// 53.3 and 51.3; 48 tokens, 12 of 2048 x 1536, top 3 (5 to 8) 67.8 and 69.4; 128 tokens, 4 of
// 4096 x 2048, top 2 (3.5) 215 and 294; 100 tokens, 10 of 1536 x 1536 without gate, top 2 (3) 66
// and 75; 128 tokens, 8 of 1024 x 512, top 2 (2) 43 and 57.
constexpr int kCountedItems = 6;
constexpr int kMaxDepth = 5;            // stages of a warp's ring
constexpr int kMoeMaxGrid = 256;        // CTAs of a projection
constexpr int kScaleBytes = 2 * 40 * 4;  // two atoms' words of 32 rows, padded apart
constexpr int kStageBytes = 4 * 512 + kScaleBytes;  // of one warp: 32 rows x 64 bytes, scales

// Shared memory of a launch: byte offsets after the rings (which start at 0).
struct ExpPlan {
    int depth;       // stages of a warp's ring
    int cap, cols;   // tokens of a pass; columns of a tile (8, or those of cap tokens if that is less)
    int tiles;       // the most tiles of a pass
    int x, red, lists, bytes;
};

__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&o)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// two E4M3 scales as fp16 pairs (s, s)
__device__ __forceinline__ void scales2(uint32_t sf16, uint32_t& s0, uint32_t& s1) {
    uint32_t h;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(sf16));
    s0 = __byte_perm(h, h, 0x1010);
    s1 = __byte_perm(h, h, 0x3232);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One stage of a warp: two 16-row MMA tiles by 128 columns.  Lane (g, t) holds rows g and
// g + 8 of a tile at columns 32 t .. 32 t + 31 (16 bytes of codes, two scales); MMA j takes
// elements 4 j .. 4 j + 3 of each of the four lanes t.
//   code: this lane's 16 bytes of row (tile, half) (2 tile + half) * 512 on; sc: its two
//   scales, 32 bytes on per row.  xb: the tokens' 16-byte units of this lane, `xstep`
//   apart for consecutive eights of the reduction, `xtile` for tiles of columns.
struct StageRegs {
    uint4 w[2][2];
    uint32_t s[2][2];
};
__device__ __forceinline__ void stage_load(StageRegs& r, uint32_t code, uint32_t sc) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            r.w[i][h] = lds128(code + i * 1024 + h * 512);
            r.s[i][h] = lds16(sc + i * 64 + h * 32);
        }
}
template <int NT, int MT>
__device__ __forceinline__ void stage_mma(float (&acc)[2][MT][4], const StageRegs& r, uint32_t xb, uint32_t xstep,
                                          uint32_t xtile) {
    uint32_t s[2][2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) scales2(r.s[i][h], s[i][h][0], s[i][h][1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint4 x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n] = lds128(xb + j * xstep + n * xtile);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t u[4], v[4];
            decode8(j == 0 ? r.w[i][0].x : j == 1 ? r.w[i][0].y : j == 2 ? r.w[i][0].z : r.w[i][0].w, u);
            decode8(j == 0 ? r.w[i][1].x : j == 1 ? r.w[i][1].y : j == 2 ? r.w[i][1].z : r.w[i][1].w, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                u[q] = mul2(u[q], s[i][0][j >> 1]);
                v[q] = mul2(v[q], s[i][1][j >> 1]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_f16(acc[i][n], u[0], v[0], u[1], v[1], x[n].x, x[n].y);
                mma_f16(acc[i][n], u[2], v[2], u[3], v[3], x[n].z, x[n].w);
            }
        }
    }
}

__device__ __forceinline__ float act_any(int act, float z) {
    switch (act) {
        case kActRelu2: return act_value<kActRelu2>(z);
        case kActGelu: return act_value<kActGelu>(z);
        case kActSilu: return act_value<kActSilu>(z);
        default: return z;
    }
}

// The power of two that brings a row with this largest |x| to [2^14, 2^15), and its inverse.
__device__ __forceinline__ void row_scales(float amax, float& down, float& up) {
    int e = (int)(__float_as_uint(amax) >> 23) - 127 - 14;  // amax in [2^(e+14), 2^(e+15))
    if (amax == 0.0f) e = 0;
    e = e < -126 ? -126 : e > 113 ? 113 : e;  // Inf and NaN rows: any scale, they stay so
    down = __uint_as_float((uint32_t)(127 - e) << 23);
    up = __uint_as_float((uint32_t)(127 + e) << 23);
}

// Where a warp stands in its CTA's work.
struct Cursor {
    int it;             // first pair of the segment
    int e, j0, nj;      // expert, its first tile here, tiles of the segment
    int p0, done;       // first token of the pass, tiles of earlier rounds
    int ks, taken;      // warps per tile, tiles of this round
    int j, step, step1; // this warp's tile, its next and last stage of the round
    bool on, end;
};

// Columns of the MMA that a token takes, and what its second one (v - hi) is scaled by.
template <bool DOWN>
constexpr int kParts = DOWN ? 2 : 1;
constexpr float kLowUp = 2048.0f, kLowDown = 1.0f / 2048.0f;

// MT: the most tiles of columns of a pass (registers for their sums).
template <bool DOWN, int MT>
__global__ void __launch_bounds__(kExpThreads, 1) moe_expert_kernel(const MoeLayerParams p, const ExpPlan pl) {
    extern __shared__ __align__(16) uint8_t sm[];
    constexpr int P = kParts<DOWN>;
    __shared__ float row_scale[8 * MT / P];
    __shared__ int nactive, even;
    const int nslots = p.T * p.topk;
    uint32_t* const count = reinterpret_cast<uint32_t*>(sm + pl.lists);  // tokens of each expert
    uint16_t* const start = reinterpret_cast<uint16_t*>(count + p.E);    // first entry in slots
    uint16_t* const active = start + p.E;                                // experts with tokens, ascending
    uint16_t* const slots = active + p.E;                                // token * topk + choice, by expert
    uint16_t* const place = slots + nslots;                              // a slot's place among its expert's
    uint16_t* const load0 = place + nslots;                              // sum of the loads of the experts before
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int kdim = DOWN ? p.F : p.K;                    // reduction length
    const int rows_e = DOWN ? p.K : p.F * (1 + p.gated);  // weight rows of an expert
    const bool gated = !DOWN && p.gated;
    const int tiles = DOWN ? p.K / 32 : gated ? p.F / 16 : p.F / 32;
    const int katoms = kdim / 64, steps = kdim / 128;
    const uint8_t* const codes = DOWN ? p.w2 : p.w1;
    const uint8_t* const sf = DOWN ? p.w2_sf : p.w1_sf;
    const float* const gs = DOWN ? p.w2_g : p.w1_g;
    for (int e = threadIdx.x; e < p.E; e += kExpThreads) count[e] = 0;
    // The second projection may start before the first has ended: by then the first has
    // seen the router's end, so the choices can be read, and the weights fetched; its
    // results are waited for before the rows are.
    if (!DOWN) grid_wait();
    grid_dependents();
    // ---- which experts are taken, and by which slots.  Their order inside an expert
    // does not matter: a token's column of the MMA does not touch the others.
    __syncthreads();
    for (int i = threadIdx.x; i < nslots; i += kExpThreads) place[i] = (uint16_t)atomicAdd(&count[__ldcg(p.idx + i)], 1u);
    __syncthreads();
    if (warp == 0) {
        int slot = 0, nact = 0;
        uint32_t most = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < p.E ? (int)count[e] : 0;
            const uint32_t on = __ballot_sync(0xFFFFFFFFu, c > 0);
            if (on == 0) continue;
            most = max(most, (uint32_t)c);
            int s = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
                if (lane >= o) s += v;
            }
            if (c > 0) {
                start[e] = (uint16_t)(slot + s - c);
                active[nact + __popc(on & ((1u << lane) - 1u))] = (uint16_t)e;
            }
            slot += __shfl_sync(0xFFFFFFFFu, s, 31);
            nact += __popc(on);
        }
        // Experts with more tokens than a tile or a pass holds cost more per weight tile.
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        const bool uneven = (int)most * P > pl.cols && nact * tiles >= kCountedItems * (int)gridDim.x;
        if (uneven) {
            int load = 0;
            __syncwarp();
            for (int a0 = 0; a0 < nact; a0 += 32) {
                const int a = a0 + lane, c = a < nact ? (int)count[active[a]] : 0;
                const int passes = (c + pl.cap - 1) / pl.cap;
                const int own = c > 0 ? passes + max(passes, (c * P + 7) / 8) : 0;
                int s = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
                    if (lane >= o) s += v;
                }
                if (a < nact) load0[a] = (uint16_t)(load + s - own);
                load += __shfl_sync(0xFFFFFFFFu, s, 31);
            }
            if (lane == 0) load0[nact] = (uint16_t)load;
        }
        if (lane == 0) {
            nactive = nact;
            even = !uneven;
        }
    }
    __syncthreads();
    // CTA b's first item: an equal share of the items, or of the experts' loads in whole tiles.
    // 32 bits hold both products: an expert has at most F / 16 = 2^10 tiles (gated), there are
    // 2^10 experts, and a token counts at most twice (a pass and a tile of its own), so the loads
    // are 2^12 in all; b goes up to the grid's size.
    static_assert((uint64_t)kMaxGroups * (kMoeMaxDim / 16) * kMoeMaxGrid < 1ull << 31 &&
                      2ull * kMoeMaxTokens * kMoeMaxTopk * (kMoeMaxDim / 16) * kMoeMaxGrid < 1ull << 32,
                  "the shares' products fit in 32 bits");
    static_assert(2 * kMoeMaxTokens * kMoeMaxTopk < 1 << 16 && kMaxGroups < 1 << 16, "the lists hold 16 bits");
    auto share = [&](uint32_t b) -> int {
        if (even || b == gridDim.x) return (int)((uint32_t)(nactive * tiles) * b / gridDim.x);
        const uint32_t u = (uint32_t)load0[nactive] * (uint32_t)tiles * b / gridDim.x;
        int lo = 0, hi = nactive - 1;  // the expert that holds unit u of the loads
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((uint32_t)load0[mid] * (uint32_t)tiles <= u) lo = mid; else hi = mid - 1;
        }
        return lo * tiles + (int)((u - (uint32_t)load0[lo] * (uint32_t)tiles) / (uint32_t)(load0[lo + 1] - load0[lo]));
    };
    const int it_begin = share(blockIdx.x), it_end = share(blockIdx.x + 1);
    if (it_begin >= it_end) return;

    auto enter = [&](Cursor& c) {  // the segment that starts at c.it
        const int a = c.it / tiles;
        c.e = active[a];
        c.j0 = c.it - a * tiles;
        c.nj = min(it_end - c.it, tiles - c.j0);
        c.p0 = c.done = 0;
    };
    auto settle = [&](Cursor& c) {  // this warp's part of the round
        const int rem = c.nj - c.done;
        int lks = 0;
        while ((rem << (lks + 1)) <= kExpWarps && (2 << lks) <= steps) ++lks;
        const int part = warp & ((1 << lks) - 1), jj = warp >> lks;
        c.ks = 1 << lks;
        c.taken = rem < (kExpWarps >> lks) ? rem : kExpWarps >> lks;
        c.on = jj < c.taken;
        c.j = c.j0 + c.done + jj;
        c.step = steps * part >> lks;
        c.step1 = steps * (part + 1) >> lks;
    };
    auto next_round = [&](Cursor& c) {
        c.done += c.taken;
        if (c.done >= c.nj) {
            c.done = 0;
            c.p0 += pl.cap;
            if (c.p0 >= (int)count[c.e]) {
                c.it += c.nj;
                if (c.it >= it_end) {
                    c.end = true;
                    return;
                }
                enter(c);
            }
        }
        settle(c);
    };
    // First row of the lane in a tile: lines of a 128-row scale atom, whose 16-byte lines
    // hold the scales of rows l, l + 32, l + 64, l + 96.  From there, row g + 8 of an MMA
    // tile and the second MMA tile are a fixed number of rows on.
    auto first_row = [&](int j) {
        return gated ? 16 * j + g : 32 * j + g;
    };
    const int half_rows = gated ? p.F : 8, tile_rows = gated ? 8 : 16;
    const int64_t pitch = kdim / 2;
    // ---- the copies: lane (g, t) fetches its codes of the four rows (tile i, half h), and
    // the scale words of row (t / 2, t % 2) in the stage's two atoms
    const uint32_t ring = smem_addr(sm) + (uint32_t)warp * (uint32_t)(pl.depth * kStageBytes);
    const uint32_t sc_dst = 4 * 512 + (uint32_t)(t * 8 + g) * 4u;
    const uint8_t *src = nullptr, *ssrc = nullptr;
    Cursor ld{};
    auto aim = [&]() {
        const int64_t R = (int64_t)ld.e * rows_e + first_row(ld.j);
        src = codes + R * pitch + ld.step * 64 + t * 16;
        const int64_t S = R + (t >> 1) * tile_rows + (t & 1) * half_rows;
        ssrc = sf + ((S >> 7) * katoms + 2 * ld.step) * 512 + (S & 31) * 16 + ((S >> 5) & 3) * 4;
    };
    auto fetch = [&](uint32_t stage) {  // one stage, and the cursor on
        if (!ld.end) {
            const uint32_t dst = stage + (uint32_t)lane * 16u;
            copy16(dst, src);
            copy16(dst + 512u, src + half_rows * pitch);
            copy16(dst + 1024u, src + tile_rows * pitch);
            copy16(dst + 1536u, src + (tile_rows + half_rows) * pitch);
            copy4(stage + sc_dst, ssrc);
            copy4(stage + sc_dst + 160u, ssrc + 512);
            src += 64;
            ssrc += 1024;
            if (++ld.step >= ld.step1) {
                do next_round(ld);
                while (!ld.end && !ld.on);
                if (!ld.end) aim();
            }
        }
        copy_commit();  // a group per stage, empty ones too: their number is what is waited for
    };
    ld.it = it_begin;
    ld.end = false;
    enter(ld);
    settle(ld);
    Cursor cp = ld;
    while (!ld.end && !ld.on) next_round(ld);
    if (!ld.end) aim();
    for (int i = 0; i < pl.depth; ++i) fetch(ring + (uint32_t)(i * kStageBytes));
    for (int i = threadIdx.x; i < nslots; i += kExpThreads) slots[start[__ldcg(p.idx + i)] + place[i]] = (uint16_t)i;

    float* const red = reinterpret_cast<float*>(sm + pl.red);
    const uint32_t xs = smem_addr(sm + pl.x);
    const uint32_t xstep = (uint32_t)pl.cols * 64u, xtile = (uint32_t)steps * 4u * xstep;
    // (columns past a tile's repeat its first; their sums are not used)
    const uint32_t xlane = xs + (g < pl.cols ? (uint32_t)g * 64u : 0u) + (uint32_t)t * 16u;
    const uint32_t sc_off = 4 * 512 + (uint32_t)(t >> 1) * 160u + (uint32_t)g * 4u + (uint32_t)(t & 1) * 2u;
    uint32_t stage = ring;
    if (DOWN) grid_wait();
    bool fresh = true;
    while (!cp.end) {
        const int n_e = (int)count[cp.e];
        const int np = n_e - cp.p0 < pl.cap ? n_e - cp.p0 : pl.cap;
        const int nt = (np * P + 7) / 8;
        const uint16_t* const my_slots = slots + start[cp.e] + cp.p0;
        if (fresh) {
            // ---- the tokens' rows as scaled fp16 in fragment order: 16-byte unit
            // (column, k / 8) at [tile][k / 128][(k % 32) / 8][column][(k % 128) / 32]
            __syncthreads();  // the slots are in place; the previous pass has read its rows
            const int rows_pad = (pl.cols < 8 ? pl.cols : nt * 8) / P;
            for (int u = threadIdx.x; u < rows_pad * steps * 16; u += kExpThreads) {
                const int i = u / (steps * 16), w = u - i * (steps * 16), k = w * 8;
                const int col = i * P;
                const uint32_t dst = xs + (uint32_t)(col >> 3) * xtile + (uint32_t)((w >> 4) * 4 + (w & 3)) * xstep +
                                     (uint32_t)(col & 7) * 64u + (uint32_t)((w >> 2) & 3) * 16u;
                uint32_t o[4] = {0, 0, 0, 0}, low[4] = {0, 0, 0, 0};
                if (i < np) {
                    const int slot = my_slots[i];
                    float down, up;
                    row_scales(__uint_as_float(DOWN ? __ldcg(p.h_amax + slot) : __ldcg(p.x_amax + slot / p.topk)), down, up);
                    if (w == 0) row_scale[i] = up;
                    float v[8];
                    if (DOWN) {
                        const float* const row = p.h + (int64_t)slot * p.F + k;
                        const float4 lo = __ldcg(reinterpret_cast<const float4*>(row));
                        const float4 hi = __ldcg(reinterpret_cast<const float4*>(row + 4));
                        v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
                        v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
                    } else {
                        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(slot / p.topk) * p.K + k));
                        v[0] = bf16_lo(x.x); v[1] = bf16_hi(x.x); v[2] = bf16_lo(x.y); v[3] = bf16_hi(x.y);
                        v[4] = bf16_lo(x.z); v[5] = bf16_hi(x.z); v[6] = bf16_lo(x.w); v[7] = bf16_hi(x.w);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float a = v[2 * q] * down, b = v[2 * q + 1] * down;  // exact: |a|, |b| < 2^15
                        const __half2 h = __floats2half2_rn(a, b);
                        o[q] = *reinterpret_cast<const uint32_t*>(&h);
                        if (DOWN) {
                            const float2 f = __half22float2(h);
                            float da = a - f.x, db = b - f.y;  // infinities stay in the first part alone
                            da = da == da ? da : 0.0f;
                            db = db == db ? db : 0.0f;
                            const __half2 l = __floats2half2_rn(da * kLowUp, db * kLowUp);
                            low[q] = *reinterpret_cast<const uint32_t*>(&l);
                        }
                    }
                }
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                             : "memory");
                if (DOWN)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 64u), "r"(low[0]), "r"(low[1]),
                                 "r"(low[2]), "r"(low[3])
                                 : "memory");
            }
            __syncthreads();
        }
        const float g_e = __ldg(gs + cp.e);
        float acc[2][MT][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < MT; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][n][q] = 0.0f;
        if (cp.on) {
            uint32_t xb = xlane + (uint32_t)cp.step * 4u * xstep;
            for (int step = cp.step; step < cp.step1; ++step) {
                switch (pl.depth) {  // the oldest stage has landed
                    case 2: copy_wait<1>(); break;
                    case 3: copy_wait<2>(); break;
                    case 4: copy_wait<3>(); break;
                    default: copy_wait<4>(); break;
                }
                __syncwarp();  // the scales that other lanes fetched
                StageRegs r;
                stage_load(r, stage + (uint32_t)lane * 16u, stage + sc_off);
                __syncwarp();  // every lane has read the stage: it is refilled while this one is used
                fetch(stage);
                stage += kStageBytes;
                if (stage == ring + (uint32_t)(pl.depth * kStageBytes)) stage = ring;
                if (MT == 1 || nt == 1) stage_mma<1, MT>(acc, r, xb, xstep, xtile);
                else if (MT == 2 || nt == 2) stage_mma<(MT > 1 ? 2 : 1), MT>(acc, r, xb, xstep, xtile);
                else if (nt == 3) stage_mma<(MT > 2 ? 3 : 1), MT>(acc, r, xb, xstep, xtile);
                else stage_mma<MT, MT>(acc, r, xb, xstep, xtile);
                xb += 4u * xstep;
            }
        }
        const int part = warp & (cp.ks - 1);
        if (cp.ks > 1 && cp.on) {
            // Join the parts of a tile, in order.  Such a round is the last of its pass, so
            // the next use of `red` comes after a barrier of the whole CTA.
            float* const mine = red + warp * (nt * 256) + lane * 4;
            if (part != 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < MT; ++n) {
                        if (n >= nt) break;
                        *reinterpret_cast<float4*>(mine + (i * nt + n) * 128) =
                            make_float4(acc[i][n][0], acc[i][n][1], acc[i][n][2], acc[i][n][3]);
                    }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / cp.ks), "r"(cp.ks * 32) : "memory");
            if (part == 0) {
                for (int w = 1; w < cp.ks; ++w)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < MT; ++n) {
                            if (n >= nt) break;
                            const float4 v = *reinterpret_cast<const float4*>(mine + ((w * 2 + i) * nt + n) * 128);
                            acc[i][n][0] += v.x; acc[i][n][1] += v.y; acc[i][n][2] += v.z; acc[i][n][3] += v.w;
                        }
            }
        }
        if (cp.on && part == 0) {
            const int row = first_row(cp.j);
#pragma unroll
            for (int n = 0; n < MT; ++n) {
                if (n >= nt) break;
#pragma unroll
                for (int c = 0; c < 2 / P; ++c) {
                    const int m = (n * 8 + 2 * t) / P + c;
                    const bool in = m < np;
                    const float scale = in ? row_scale[m] : 0.0f;
                    const int slot = in ? my_slots[m] : 0;
                    uint32_t big = 0;  // the row's largest |h| of this lane
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float s0 = DOWN ? fmaf(acc[i][n][1], kLowDown, acc[i][n][0]) : acc[i][n][c];
                        const float s1 = DOWN ? fmaf(acc[i][n][3], kLowDown, acc[i][n][2]) : acc[i][n][2 + c];
                        const float v0 = s0 * scale * g_e, v1 = s1 * scale * g_e;
                        const int r0 = row + i * tile_rows;
                        if (DOWN) {
                            if (in) {
                                float* const z = p.z + (int64_t)slot * p.K + r0;
                                z[0] = v0;
                                z[8] = v1;
                            }
                        } else {
                            float* const h = p.h + (int64_t)slot * p.F + r0;
                            float h0 = act_any(p.act, v0), h1 = 0.0f;
                            if (gated) {
                                h0 *= v1;
                            } else {
                                h1 = act_any(p.act, v1);
                                if (in) h[8] = h1;
                            }
                            if (in) h[0] = h0;
                            big = max(big, max(__float_as_uint(h0) & 0x7FFFFFFFu, __float_as_uint(h1) & 0x7FFFFFFFu));
                        }
                    }
                    if (!DOWN) {  // over the eight lanes of a column
                        big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 4));
                        big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 8));
                        big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 16));
                        if (in && g == 0) atomicMax(p.h_amax + slot, big);
                    }
                }
            }
        }
        const int p0 = cp.p0;
        const int it = cp.it;
        next_round(cp);
        fresh = cp.it != it || cp.p0 != p0;
    }
    copy_wait<0>();
}

// y = the tokens' weighted sums over their choices, in order.  (Inside the second projection
// instead, by the last expert to finish 32 columns of a token: 1 token of 64 experts of 2048 x
// 1024 21.9 us as with this kernel, 16 tokens 56.8 against 56.4, 7 of 10 of 384 x 256 19.0
// against 17.2, 64 of 128 of 1024 x 512 72 against 62: the fences weigh more than a launch.)
__global__ void __launch_bounds__(256) moe_sum_kernel(const MoeLayerParams p) {
    grid_wait();
    const int per = p.K / 4;
    const int u = blockIdx.x * 256 + threadIdx.x;
    if (u >= p.T * per) return;
    const int tok = u / per, col = (u - tok * per) * 4;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int q = 0; q < p.topk; ++q) {
        const float w = __ldcg(p.weight + tok * p.topk + q);
        const float4 z = __ldcg(reinterpret_cast<const float4*>(p.z + (int64_t)(tok * p.topk + q) * p.K + col));
        y.x = fmaf(w, z.x, y.x); y.y = fmaf(w, z.y, y.y);
        y.z = fmaf(w, z.z, y.z); y.w = fmaf(w, z.w, y.w);
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
    *reinterpret_cast<uint2*>(p.y + (int64_t)tok * p.K + col) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// ---------------------------------------------------------------- host side
// Shared memory of a launch.  A pass takes as many tokens as an expert is likely to have
// (its mean and two standard deviations), in tiles of 8 columns, while the rings keep 3
// stages; for as many as it has usually (one deviation) 2 stages do, as a second pass costs
// more.  3 and 2 there (us): 128 tokens, 32 experts of 2048 x 1024, top 4 105 and 94; 64 of 64
// of 4096 x 2048, top 8 319 and 310; 128 of 64 of 1024 x 1024, top 8 98 and 94; 2 stages for the
// likely number too: 64 tokens, 128 of 4096 x 2048, top 8 399 and 406.  Very long rows leave
// room for fewer than 8 columns.
static bool plan_expert(const MoeLayerParams& p, bool down, int smem_max, ExpPlan* pl) {
    const int parts = down ? kParts<true> : kParts<false>;
    const int row_bytes = 2 * (down ? p.F : p.K);
    const int lists = (4 * p.E + 2 * 2 * p.E + 2 * 2 * p.T * p.topk + 2 * (p.E + 1) + 15) / 16 * 16;
    const int room = smem_max - lists;
    const double mean = (double)p.T * p.topk / p.E;
    int likely = (int)(mean + 2.0 * sqrt(mean)) + 1;
    likely = likely > p.T ? p.T : likely;
    int nt = (likely * parts + 7) / 8;
    nt = nt > kMaxTiles ? kMaxTiles : nt;
    auto depth = [&](int columns, int tiles) {
        const int n = (room - columns * row_bytes - tiles * kExpWarps * 1024) / (kExpWarps * kStageBytes);
        return n > kMaxDepth ? kMaxDepth : n;
    };
    const int usual = ((int)(mean + sqrt(mean)) + 1) * parts;
    while (nt > 1 && depth(nt * 8, nt) < (nt * 8 - 8 < usual ? 2 : 3)) --nt;
    int columns = nt * 8;
    pl->cols = 8;
    while (columns > parts && depth(columns, nt) < 2) pl->cols = columns = columns / 2;
    pl->cap = columns / parts;
    pl->tiles = nt;
    pl->depth = depth(columns, nt);
    if (pl->depth < 2) return false;
    pl->x = kExpWarps * pl->depth * kStageBytes;
    pl->red = pl->x + columns * row_bytes;
    pl->lists = pl->red + nt * kExpWarps * 1024;
    pl->bytes = pl->lists + lists;
    return true;
}

template <class... Args>
static cudaError_t launch_dependent(void (*kernel)(Args...), int grid, int threads, int smem, cudaStream_t st,
                                    const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool DOWN, int MT>
static cudaError_t launch_expert_mt(const MoeLayerParams& p, const ExpPlan& pl, int dev, int room, int sms,
                                    cudaStream_t st) {
    static bool configured[64] = {};
    if (!configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(moe_expert_kernel<DOWN, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    return launch_dependent(moe_expert_kernel<DOWN, MT>, sms < kMoeMaxGrid ? sms : kMoeMaxGrid, kExpThreads, pl.bytes, st, p, pl);
}

template <bool DOWN>
static cudaError_t launch_expert(const MoeLayerParams& p, int sms, cudaStream_t st) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static int most[64] = {};
    if (most[dev] == 0 &&
        (e = cudaDeviceGetAttribute(&most[dev], cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess)
        return e;
    const int room = most[dev] - 1024;  // beside the static arrays
    ExpPlan pl;
    if (!plan_expert(p, DOWN, room, &pl)) return cudaErrorInvalidValue;
    if (pl.tiles == 1) return launch_expert_mt<DOWN, 1>(p, pl, dev, room, sms, st);
    if (pl.tiles == 2) return launch_expert_mt<DOWN, 2>(p, pl, dev, room, sms, st);
    return launch_expert_mt<DOWN, 4>(p, pl, dev, room, sms, st);
}

template <int TC>
static cudaError_t launch_route(const MoeLayerParams& p, cudaStream_t st) {
    const unsigned clusters = (unsigned)((p.T + TC - 1) / TC);
    moe_route_kernel<TC><<<clusters * kRouteCluster, kRouteThreads, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_moe_layer(const MoeLayerParams& p, int sms, cudaStream_t st) {
    // as few tokens per cluster as keep the clusters resident at once
    const int most = sms / kRouteCluster;
    cudaError_t e = p.T <= most ? launch_route<1>(p, st) : p.T <= 2 * most ? launch_route<2>(p, st)
                  : p.T <= 4 * most ? launch_route<4>(p, st) : launch_route<8>(p, st);
    if (e == cudaSuccess) e = launch_expert<false>(p, sms, st);
    if (e == cudaSuccess) e = launch_expert<true>(p, sms, st);
    if (e == cudaSuccess) e = launch_dependent(moe_sum_kernel, (p.T * (p.K / 4) + 255) / 256, 256, 0, st, p);
    return e;
}

}  // namespace nvfp4
