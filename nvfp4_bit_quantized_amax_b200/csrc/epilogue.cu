// epilogue.cu -- backward pass of the GEMM's fused epilogue D = act(Z) + R, Z = A B^T + bias.
//
//   dZ[m][n] = dY[m][n] act'(Z[m][n])      dbias[n] = sum over m of dZ[m][n]
// (the residual's gradient is dY itself).  Memory-bound: 4 bytes read and 2 written per
// element; 8192 x 20480 with GELU take 177 us in a replayed graph (5.7 TB/s), 184 to 188 called
// with caches cleared.  A CTA takes 32 or 128 rows of 256 columns, 8 columns and every eighth
// row per thread, four rows' loads in flight at a time (one row's: 246 us).  The column sums
// of the unrounded products, in fp32: the eight CTAs of a cluster add theirs through
// distributed shared memory; with more rows than a cluster has, its sums are a partial row,
// and a second kernel adds those up.  Every order is fixed by M and N, so the sums do not
// depend on timing.
#include <cuda_bf16.h>

#include "activation.cuh"

namespace nvfp4 {

constexpr int kBwdCols = 256;
constexpr int kBwdCluster = 8;

// Rows per CTA: 32 while those CTAs are at most 1024, so that small problems spread and end
// soon; else 128, which pays the cluster's barriers once per 16 rows of a thread.  1024 is
// where the two meet as measured (registers allow four or five CTAs per SM, some 600 to 740 at
// once, so the last of them run in a second wave).  GELU with sums, 32 and 128 rows (us): 250 x
// 264 3.4 and 7.5, 4096 x 1024 7.9 and 11.5, 512 x 16384 (1024 CTAs) 12.3 and 16.7, 2048 x 4096
// (1024) 12.2 and 12.1, 4096 x 4096 23.4 and 20.0, 8192 x 20480 208 and 177.
static inline int64_t bwd_rows(int64_t M, int64_t N) {
    return (N + kBwdCols - 1) / kBwdCols * ((M + 31) / 32) <= 1024 ? 32 : 128;
}

template <int ACT>
__global__ void __cluster_dims__(kBwdCluster, 1, 1) __launch_bounds__(256) epilogue_backward_kernel(const uint16_t* dY,
                                                                const uint16_t* Z, int64_t M,
                                                                int64_t N, uint16_t* dZ,
                                                                float* __restrict__ sums, const int rows) {
    __shared__ float part[8][kBwdCols];
    __shared__ float total[kBwdCols];
    const int rank = blockIdx.x % kBwdCluster;
    const unsigned strips = (unsigned)((N + kBwdCols - 1) / kBwdCols), cid = blockIdx.x / kBwdCluster;
    const int64_t strip = cid % strips, cluster = cid / strips;  // columns fastest: whole rows together
    const int64_t col = strip * kBwdCols + (threadIdx.x & 31) * 8;
    const int64_t row0 = (cluster * kBwdCluster + rank) * rows;
    const int64_t row1 = row0 + rows < M ? row0 + rows : M;
    f32x2 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = both(0.0f);
    if (col < N) {
        for (int64_t r = row0 + (threadIdx.x >> 5); r < row1; r += 32) {
            uint4 dy[4], z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                dy[k] = z[k] = make_uint4(0, 0, 0, 0);
                if (r + 8 * k < row1) {
                    dy[k] = __ldcs(reinterpret_cast<const uint4*>(dY + (r + 8 * k) * N + col));
                    z[k] = __ldcs(reinterpret_cast<const uint4*>(Z + (r + 8 * k) * N + col));
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (r + 8 * k >= row1) break;
                const uint32_t aw[4] = {dy[k].x, dy[k].y, dy[k].z, dy[k].w}, bw[4] = {z[k].x, z[k].y, z[k].z, z[k].w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x2 d = mul2f(pack2(bf16_lo(aw[i]), bf16_hi(aw[i])),
                                          act_slope2<ACT>(pack2(bf16_lo(bw[i]), bf16_hi(bw[i]))));
                    acc[i] = add2f(acc[i], d);
                    float lo, hi;
                    unpack2(d, lo, hi);
                    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                    o[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
                __stcs(reinterpret_cast<uint4*>(dZ + (r + 8 * k) * N + col), make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
    }
    if (sums == nullptr) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(acc[i], lo, hi);
        part[threadIdx.x >> 5][(threadIdx.x & 31) * 8 + 2 * i] = lo;
        part[threadIdx.x >> 5][(threadIdx.x & 31) * 8 + 2 * i + 1] = hi;
    }
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += part[w][threadIdx.x];
    total[threadIdx.x] = t;
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    // CTA r of the cluster adds columns 32 r .. 32 r + 31: thread (w, l) fetches CTA w's
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(&total[rank * 32 + l])), "r"(w));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(t) : "r"(at) : "memory");
    part[w][l] = t;
    // this CTA has read its peers' sums; it ends only when they have read its own
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    __syncthreads();
    const int64_t c = strip * kBwdCols + rank * 32 + threadIdx.x;
    if (threadIdx.x < 32 && c < N) {
        t = 0.0f;
#pragma unroll
        for (int q = 0; q < kBwdCluster; ++q) t += part[q][threadIdx.x];
        sums[cluster * N + c] = t;
    }
    // (not .aligned: where N % 32 is not 0 the store above has parted the lanes)
    asm volatile("barrier.cluster.wait;" ::: "memory");
}

// dbias[n] = sum of the partial rows, in row order by eight threads of a column.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ partials, int64_t rows, int64_t N,
                                                         float* __restrict__ out) {
    __shared__ float part[8][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    float t = 0.0f;
    if (c < N)
        for (int64_t r = threadIdx.x >> 5; r < rows; r += 8) t += partials[r * N + c];
    part[threadIdx.x >> 5][threadIdx.x & 31] = t;
    __syncthreads();
    if (threadIdx.x < 32 && c < N) {
        t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += part[w][threadIdx.x];
        out[c] = t;
    }
}

static int64_t row_clusters(int64_t M, int64_t N) {
    const int64_t rows = bwd_rows(M, N) * kBwdCluster;
    return (M + rows - 1) / rows;
}

int64_t epilogue_backward_partials(int64_t M, int64_t N) {
    const int64_t rc = row_clusters(M, N);
    return rc > 1 ? rc * N : 0;
}

template <int ACT>
static cudaError_t launch_bwd(const uint16_t* dY, const uint16_t* Z, int64_t M, int64_t N, uint16_t* dZ,
                              float* dbias, float* partials, cudaStream_t st) {
    const int64_t rc = row_clusters(M, N);
    float* sums = dbias == nullptr ? nullptr : rc > 1 ? partials : dbias;
    const int64_t grid = (N + kBwdCols - 1) / kBwdCols * rc * kBwdCluster;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    epilogue_backward_kernel<ACT><<<(unsigned)grid, 256, 0, st>>>(dY, Z, M, N, dZ, sums, (int)bwd_rows(M, N));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || dbias == nullptr || rc == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((N + 31) / 32));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, column_sum_kernel, (const float*)partials, rc, N, dbias);
}

cudaError_t launch_epilogue_backward(const uint16_t* dY, const uint16_t* Z, int act, int64_t M, int64_t N,
                                     uint16_t* dZ, float* dbias, float* partials, cudaStream_t st) {
    switch (act) {
        case kActRelu2: return launch_bwd<kActRelu2>(dY, Z, M, N, dZ, dbias, partials, st);
        case kActGelu: return launch_bwd<kActGelu>(dY, Z, M, N, dZ, dbias, partials, st);
        case kActSilu: return launch_bwd<kActSilu>(dY, Z, M, N, dZ, dbias, partials, st);
        default: return launch_bwd<kActNone>(dY, Z, M, N, dZ, dbias, partials, st);
    }
}

}  // namespace nvfp4
