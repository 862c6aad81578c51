// moe_linear.hip -- C = A B^T with the linear epilogue (bias, activation,
// residual, pre-activation kept), and the elementwise steps around the dense
// products: fp32 activations as three bf16 terms, the gradient through the
// activation with the bias gradient's column sums.
#include "moe_dense.h"

namespace moe {

// fp32 [n] -> three bf16 planes [n] (n a multiple of 8): one pass, bound by
// its 10 bytes per value (8192 x 4096: 53 us, 6.3 TB/s of reads and writes
// that partly stay in the last-level cache).
__global__ __launch_bounds__(256) void k_dense_split3(const float *x, uint16_t *out, int64_t n) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
        float v[8];
        dn_load_f32<8>(x + i, v);
        dn_store_split3<8>(out + i, (size_t)n, v);
    }
}

// dz = dy act'(z) for 256 columns (32 threads of 8) and one chunk of rows (8
// at a time), and the chunk's column sums (from the unrounded values: eight
// row lanes in fp32, then joined in order).  Bound by its reads and writes (8192 x 4096, SiLU:
// 201 MB in 44 us, 4.6 TB/s; 777 x 2048 7.6 us, launch and one trip to memory).
__global__ __launch_bounds__(256) void k_dense_dz(DzParams P) {
    __shared__ float s_sum[8][256 + 8];
    const int tid = threadIdx.x, cl = tid & 31, rl = tid >> 5;
    const int n = blockIdx.x * 256 + cl * 8;
    const int64_t r0 = (int64_t)blockIdx.y * P.rows_per_chunk;
    const int64_t r1 = min((int64_t)P.T, r0 + P.rows_per_chunk);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n < P.N) {
        constexpr int Q = 4;  // rows in flight per thread (loaded before the first is stored)
        for (int64_t t0 = r0 + rl; t0 < r1; t0 += 8 * Q) {
            u32x4 dy[Q], z[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int64_t t = min(t0 + 8 * q, r1 - 1);
                dy[q] = *(const u32x4 *)(P.dy + t * P.N + n);
                if (P.z) z[q] = *(const u32x4 *)(P.z + t * P.N + n);
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int64_t t = t0 + 8 * q;
                if (t >= r1) break;
                float v[8];
                dn_unpack<8>(dy[q], v);
                if (P.z) {
                    float zv[8];
                    dn_unpack<8>(z[q], zv);
                    dn_times_slope<8>(P.act, zv, v);
                }
                if (P.dz) dn_store_bf<8>(P.dz + t * P.N + n, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += v[i];
            }
        }
    }
    if (!P.part) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) s_sum[rl][cl * 8 + i] = sum[i];
    __syncthreads();
    const int c = blockIdx.x * 256 + tid;
    if (c < P.N) {
        float v = s_sum[0][tid];
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s_sum[i][tid];
        P.part[(int64_t)blockIdx.y * P.N + c] = v;
    }
}

__global__ __launch_bounds__(256) void k_dense_colsum(ColsumParams P) {
    __shared__ float s_sum[256 / DN_SUM_COLS][DN_SUM_COLS + 1];
    dn_colsum<256>(P, blockIdx.x, &s_sum[0][0]);
}

hipError_t dense_split3_launch(const float *x, uint16_t *out, int64_t n, hipStream_t st) {
    const int64_t blocks = (n / 8 + 255) / 256;
    hipLaunchKernelGGL(k_dense_split3, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, st, x, out, n);
    return hipGetLastError();
}
hipError_t dense_dz_launch(const DzParams &P, hipStream_t st) {
    hipLaunchKernelGGL(k_dense_dz, dim3((unsigned)((P.N + 255) / 256), (unsigned)P.nchunks), dim3(256), 0, st, P);
    return hipGetLastError();
}
hipError_t dense_colsum_launch(const ColsumParams &P, hipStream_t st) {
    hipLaunchKernelGGL(k_dense_colsum, dim3((unsigned)((P.N + DN_SUM_COLS - 1) / DN_SUM_COLS)), dim3(256), 0, st, P);
    return hipGetLastError();
}
hipError_t dense_linear_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_NT, DN_EPI_LINEAR>(P, tile, st);
}

}  // namespace moe
