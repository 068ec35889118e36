// adamw.cu -- AdamW step over a list of tensors, moments in 32 or in 8 bits.
//
// Per element, with g the gradient times *grad_scale, t the step:
//   m = b1 m + (1 - b1) g        v = b2 v + (1 - b2) g^2        r = sqrt(v)
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (r / sqrt(1 - b2^t) + eps)
// Every product and sum is rounded on its own (no contraction), so that the result
// is the formula's, operation by operation, in fp32.
//
// 8-bit moments hold m and r = sqrt(v) as E4M3 codes with one E8M0 scale per 32
// consecutive elements (8.25 bits each), rounded stochastically: with beta2 near 1 a
// step moves v by less than half a code, and round-to-nearest would never move it.
// r is stored instead of v because its exponent range is half of v's.  A nonzero r
// never rounds to the zero code: m / (0 + eps) would be a huge step.
//
// Bound by memory with 32-bit moments: 28 bytes an element (bf16 gradients and copies), 210M
// elements in 860 us = 6.8 TB/s (a plain copy on the same machine moves 6.5).  With
// 8-bit moments, 16 bytes, 101M elements in 354 us = 4.6 TB/s, short of both memory and issue
// slots: 94 instructions an element (the draws are 11) keep those 74% busy, and the longest
// stall is the wait for memory, one pass of loads being in flight.  Fewer instructions alone
// (78, packed) gained nothing; those and the next pass's loads ahead 2%, which was not
// worth the code.  Step and rate on the device cost two powers in fp64 per CTA before its
// first load: 899 us against 863, and 373 against 356 with 8 bits.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace nvfp4 {

constexpr int kAdamThreads = 256;
constexpr int kAdamVec = 8;                              // elements per thread and pass
constexpr int kAdamPass = kAdamThreads * kAdamVec;       // elements per CTA and pass

template <int CAP>
struct AdamTable {
    AdamWEntry t[CAP];
    uint32_t chunk0[CAP + 1];  // first chunk of each tensor, then the number of chunks
    int count;
};

struct AdamScalars {
    float b1, omb1, b2, omb2, eps, inv_sqrt_bc2, step_size, gscale;
    double lr;
    uint32_t step;
};

// Four E4M3 codes -> fp32 (exact; NaN codes give NaN).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t codes, float* x) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
__device__ __forceinline__ float e8m0_to_f32(uint32_t code) {
    return __uint_as_float(code == 0 ? 0x00400000u : code == 255 ? 0x7FC00000u : code << 23);
}

// The E8M0 code of a block whose largest |x| has these bits: 2^e with e the smallest
// exponent that keeps the block at or below 448 (255: the block holds Inf or NaN).
__device__ __forceinline__ uint32_t block_scale_code(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return 255u;
    if (amax_bits == 0) return 0u;
    int e = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = e < -127 ? -127 : e;
    return (uint32_t)(e + 127);
}

// |x| times 2^-e as an E4M3 code in bits 20 .. 26, rounded up iff R + floor(p 2^16) >= 2^16
// with p the position between the two neighbours: in the fp32 whose bias makes bit 20 the
// code's last bit (subnormals included), that is an addition below it.
__device__ __forceinline__ uint32_t e4m3_sr_bits(float ax, float inv, uint32_t r16_at_4) {
    return __float_as_uint(__fmul_rn(__fmul_rn(ax, inv), 0x1p-120f)) + r16_at_4;
}
// the bytes in bits 20 .. 27 of four words, as one word
__device__ __forceinline__ uint32_t gather_codes(const uint32_t (&w)[4]) {
    return __byte_perm(__byte_perm(w[0] << 4, w[1] << 4, 0x0073), __byte_perm(w[2] << 4, w[3] << 4, 0x0073), 0x5410);
}

template <int BITS, bool GRAD_F32, int CAP>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamTable<CAP> tab,
                                                             const AdamWArgs a, const int tensor0, const int passes) {
    __shared__ AdamScalars sc;
    if (a.skip != nullptr && *a.skip != 0) return;  // the whole grid sees the same word
    if (threadIdx.x == 0) {
        sc.b1 = (float)a.beta1;
        sc.omb1 = (float)(1.0 - a.beta1);
        sc.b2 = (float)a.beta2;
        sc.omb2 = (float)(1.0 - a.beta2);
        sc.eps = (float)a.eps;
        sc.lr = a.dev_lr ? (double)*a.dev_lr : a.lr;
        sc.gscale = a.grad_scale ? *a.grad_scale : 1.0f;
        double bc1 = a.bc1, bc2 = a.bc2;
        int64_t step = a.step;
        if (a.dev_step) {
            step = *a.dev_step < 1 ? 1 : *a.dev_step;
            bc1 = 1.0 - pow(a.beta1, (double)step);
            bc2 = 1.0 - pow(a.beta2, (double)step);
        }
        sc.step = (uint32_t)step;
        sc.inv_sqrt_bc2 = (float)(1.0 / sqrt(bc2));
        sc.step_size = (float)(sc.lr / bc1);
    }
    __syncthreads();
    const AdamScalars s = sc;
    const uint32_t c = blockIdx.x;
    int lo = 0, hi = tab.count - 1;  // the tensor of chunk c
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.chunk0[mid] <= c) lo = mid; else hi = mid - 1;
    }
    const AdamWEntry& T = tab.t[lo];
    const float decay = (float)(1.0 - s.lr * T.weight_decay);
    const int64_t chunk_begin = (int64_t)(c - tab.chunk0[lo]) * passes * kAdamPass;
    for (int pass = 0; pass < passes; ++pass) {
        const int64_t begin = chunk_begin + (int64_t)pass * kAdamPass;
        if (begin >= T.n) break;
        const int64_t i0 = begin + threadIdx.x * kAdamVec;
        const int cnt = T.n - i0 >= kAdamVec ? kAdamVec : T.n > i0 ? (int)(T.n - i0) : 0;
        const bool full = cnt == kAdamVec;
        float p[8], g[8], m[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = g[i] = m[i] = v[i] = 0.0f;
        auto load_f32 = [&](const float* src, float (&x)[8]) {
            if (full) {
                const float4 a4 = __ldcs(reinterpret_cast<const float4*>(src + i0));
                const float4 b4 = __ldcs(reinterpret_cast<const float4*>(src + i0 + 4));
                x[0] = a4.x; x[1] = a4.y; x[2] = a4.z; x[3] = a4.w;
                x[4] = b4.x; x[5] = b4.y; x[6] = b4.z; x[7] = b4.w;
            } else {
                for (int i = 0; i < 8; ++i)
                    if (i < cnt) x[i] = src[i0 + i];
            }
        };
        load_f32(T.p, p);
        if (GRAD_F32) {
            load_f32(static_cast<const float*>(T.grad), g);
        } else if (full) {
            const uint4 w = ld_stream_v4(static_cast<const uint16_t*>(T.grad) + i0);
            g[0] = bf16_lo(w.x); g[1] = bf16_hi(w.x); g[2] = bf16_lo(w.y); g[3] = bf16_hi(w.y);
            g[4] = bf16_lo(w.z); g[5] = bf16_hi(w.z); g[6] = bf16_lo(w.w); g[7] = bf16_hi(w.w);
        } else {
            for (int i = 0; i < 8; ++i)
                if (i < cnt) g[i] = bf16_lo(static_cast<const uint16_t*>(T.grad)[i0 + i]);
        }
        uint8_t* const m8 = static_cast<uint8_t*>(T.m);
        uint8_t* const v8 = static_cast<uint8_t*>(T.v);
        if (BITS == 32) {
            load_f32(static_cast<const float*>(T.m), m);
            load_f32(static_cast<const float*>(T.v), v);
        } else {
            uint32_t mc[2] = {0, 0}, vc[2] = {0, 0};
            float ms = 0.0f, vs = 0.0f;
            if (cnt > 0) {
                ms = e8m0_to_f32(T.m_scale[i0 >> 5]);
                vs = e8m0_to_f32(T.v_scale[i0 >> 5]);
            }
            if (full) {
                const uint2 a2 = *reinterpret_cast<const uint2*>(m8 + i0), b2 = *reinterpret_cast<const uint2*>(v8 + i0);
                mc[0] = a2.x; mc[1] = a2.y; vc[0] = b2.x; vc[1] = b2.y;
            } else {
                for (int i = 0; i < 8; ++i)
                    if (i < cnt) {
                        mc[i >> 2] |= (uint32_t)m8[i0 + i] << (8 * (i & 3));
                        vc[i >> 2] |= (uint32_t)v8[i0 + i] << (8 * (i & 3));
                    }
            }
            e4m3x4_to_f32(mc[0], m);
            e4m3x4_to_f32(mc[1], m + 4);
            e4m3x4_to_f32(vc[0], v);
            e4m3x4_to_f32(vc[1], v + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] = __fmul_rn(m[i], ms);
                const float r = __fmul_rn(v[i], vs);
                v[i] = __fmul_rn(r, r);
            }
        }
        float r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gi = a.grad_scale ? __fmul_rn(g[i], s.gscale) : g[i];
            m[i] = __fadd_rn(__fmul_rn(m[i], s.b1), __fmul_rn(gi, s.omb1));
            v[i] = __fadd_rn(__fmul_rn(v[i], s.b2), __fmul_rn(__fmul_rn(gi, gi), s.omb2));
            r[i] = __fsqrt_rn(v[i]);
            const float den = __fadd_rn(__fmul_rn(r[i], s.inv_sqrt_bc2), s.eps);
            // the quotient to 2 ulp: far below what p's own rounding keeps of the update
            p[i] = __fsub_rn(__fmul_rn(p[i], decay), __fmul_rn(__fdividef(m[i], den), s.step_size));
        }
        auto store_f32 = [&](float* dst, const float (&x)[8]) {
            if (full) {
                __stcs(reinterpret_cast<float4*>(dst + i0), make_float4(x[0], x[1], x[2], x[3]));
                __stcs(reinterpret_cast<float4*>(dst + i0 + 4), make_float4(x[4], x[5], x[6], x[7]));
            } else {
                for (int i = 0; i < 8; ++i)
                    if (i < cnt) dst[i0 + i] = x[i];
            }
        };
        store_f32(T.p, p);
        if (T.w) {
            __nv_bfloat16* w = static_cast<__nv_bfloat16*>(T.w);
            if (full) {
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(p[2 * i], p[2 * i + 1]);
                    o[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
                __stcs(reinterpret_cast<uint4*>(w + i0), make_uint4(o[0], o[1], o[2], o[3]));
            } else {
                for (int i = 0; i < 8; ++i)
                    if (i < cnt) w[i0 + i] = __float2bfloat16_rn(p[i]);
            }
        }
        if (BITS == 32) {
            store_f32(static_cast<float*>(T.m), m);
            store_f32(static_cast<float*>(T.v), v);
        } else {
            // block maxima over the four threads of a 32-element block (elements past
            // the tensor's end are zero); integer order is |x|'s order, NaN largest
            if (!full) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= cnt) m[i] = r[i] = 0.0f;
            }
            uint32_t am = 0, av = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                am = max(am, __float_as_uint(m[i]) & 0x7FFFFFFFu);
                av = max(av, __float_as_uint(r[i]) & 0x7FFFFFFFu);
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
                av = max(av, __shfl_xor_sync(0xFFFFFFFFu, av, o));
            }
            const uint32_t cm = block_scale_code(am), cv = block_scale_code(av);
            const float im = e8m0_to_f32(254u - (cm == 255u ? 0u : cm)), iv = e8m0_to_f32(254u - (cv == 255u ? 0u : cv));
            uint32_t mc[2], vc[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint64_t q = (uint64_t)(i0 >> 2) + h;
                const Philox4 d = philox4x32_10_rk((uint32_t)q, (uint32_t)(q >> 32), (uint32_t)(tensor0 + lo), s.step, a.rk);
                const uint32_t dr[4] = {d.x, d.y, d.z, d.w};
                uint32_t km[4], kv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = 4 * h + j;
                    km[j] = e4m3_sr_bits(fabsf(m[i]), im, (dr[j] & 0xFFFFu) << 4);
                    // bit 27 is the code's sign: the fp32's, four places down
                    km[j] = (km[j] & 0x07FFFFFFu) | ((__float_as_uint(m[i]) >> 4) & 0x08000000u);
                    // above zero (a square root is 0 or at least 2^-75): never the zero code
                    kv[j] = max(e4m3_sr_bits(r[i], iv, (dr[j] >> 12) & 0xFFFF0u), min(__float_as_uint(r[i]), 1u << 20));
                }
                mc[h] = cm == 255u ? 0x7F7F7F7Fu : gather_codes(km);
                vc[h] = cv == 255u ? 0x7F7F7F7Fu : gather_codes(kv);
            }
            if (full) {
                *reinterpret_cast<uint2*>(m8 + i0) = make_uint2(mc[0], mc[1]);
                *reinterpret_cast<uint2*>(v8 + i0) = make_uint2(vc[0], vc[1]);
            } else {
                for (int i = 0; i < 8; ++i)
                    if (i < cnt) {
                        m8[i0 + i] = (uint8_t)(mc[i >> 2] >> (8 * (i & 3)));
                        v8[i0 + i] = (uint8_t)(vc[i >> 2] >> (8 * (i & 3)));
                    }
            }
            if (cnt > 0 && (threadIdx.x & 3) == 0) {
                T.m_scale[i0 >> 5] = (uint8_t)cm;
                T.v_scale[i0 >> 5] = (uint8_t)cv;
            }
        }
    }
}

template <int BITS, bool GRAD_F32, int CAP>
static cudaError_t launch_cap(const AdamWEntry* e, int count, const AdamWArgs& a, int sms, cudaStream_t st) {
    AdamTable<CAP> tab;
    // One CTA per chunk, in the tensors' order: a grid of resident CTAs that walk the
    // chunks instead reads and writes many places of DRAM at once (210M parameters,
    // 32-bit moments: 985 us against 855 us).  With 8-bit moments, where the start of a
    // CTA weighs more, four passes a chunk once that leaves every SM several CTAs
    // (101M parameters: 476 us with one pass, 386 with two, 351 with four, 347 with
    // eight; 32-bit: 855 us with one, 870 with two, 879 with four).
    uint64_t total = 0;
    for (int i = 0; i < count; ++i) total += (uint64_t)e[i].n;
    const int passes = BITS == 8 && total >= (uint64_t)kAdamPass * 4 * 16 * (uint64_t)sms ? 4 : 1;
    const int64_t chunk = (int64_t)kAdamPass * passes;
    int done = 0;
    while (done < count) {
        const int first = done;
        uint64_t chunks = 0;
        tab.count = 0;
        // as many tensors as the table holds; chunk numbers stay within a grid's
        while (done < count && tab.count < CAP) {
            const uint64_t c = (uint64_t)((e[done].n + chunk - 1) / chunk);
            if (tab.count > 0 && chunks + c > 0x7FFFFFFFull) break;
            tab.t[tab.count] = e[done];
            tab.chunk0[tab.count] = (uint32_t)chunks;
            chunks += c;
            ++tab.count;
            ++done;
        }
        tab.chunk0[tab.count] = (uint32_t)chunks;
        if (chunks == 0) continue;
        adamw_kernel<BITS, GRAD_F32, CAP><<<(unsigned)chunks, kAdamThreads, 0, st>>>(tab, a, first, passes);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

template <int BITS, bool GRAD_F32>
static cudaError_t launch_bits(const AdamWEntry* e, int count, const AdamWArgs& a, int sms, cudaStream_t st) {
    return count <= 32 ? launch_cap<BITS, GRAD_F32, 32>(e, count, a, sms, st)
                       : launch_cap<BITS, GRAD_F32, 384>(e, count, a, sms, st);
}

cudaError_t launch_adamw(const AdamWEntry* e, int count, const AdamWArgs& a, int state_bits, bool grad_f32,
                         int sms, cudaStream_t st) {
    if (state_bits == 32)
        return grad_f32 ? launch_bits<32, true>(e, count, a, sms, st) : launch_bits<32, false>(e, count, a, sms, st);
    return grad_f32 ? launch_bits<8, true>(e, count, a, sms, st) : launch_bits<8, false>(e, count, a, sms, st);
}

}  // namespace nvfp4
