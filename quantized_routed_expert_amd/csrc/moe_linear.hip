// moe_linear.hip -- C = A B^T with the linear epilogue (bias, activation,
// residual, pre-activation kept), and the elementwise steps around the dense
// products: fp32 activations as three bf16 terms, the gradient through the
// activation with the bias gradient's column sums.
#include "moe_dense.h"

namespace moe {

// fp32 [n] -> three bf16 planes [n] (n a multiple of 8): one pass, bound by
// its 10 bytes per value.
__global__ __launch_bounds__(256) void k_dense_split3(const float *x, uint16_t *out, int64_t n) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
        float v[8];
        dn_load_f32<8>(x + i, v);
        dn_store_split3<8>(out + i, (size_t)n, v);
    }
}

__device__ __forceinline__ void dn_store_sum(void *out, int c, float v, int out_f32, int accumulate) {
    if (out_f32) {
        float *o = (float *)out + c;
        *o = accumulate ? *o + v : v;
    } else {
        uint16_t *o = (uint16_t *)out + c;
        if (accumulate) v += dn_bf(*o);
        *o = (uint16_t)(dn_pack(v, 0.f) & 0xFFFFu);
    }
}

// dz = dy act'(z) for 256 columns (32 threads of 8) and one chunk of rows (8
// at a time), and the chunk's column sums (from the unrounded values: eight
// row lanes in fp32, then joined in order).  Bound by its reads and writes.
__global__ __launch_bounds__(256) void k_dense_dz(DzParams P) {
    __shared__ float s_sum[8][256 + 8];
    const int tid = threadIdx.x, cl = tid & 31, rl = tid >> 5;
    const int n = blockIdx.x * 256 + cl * 8;
    const int64_t r0 = (int64_t)blockIdx.y * P.rows_per_chunk;
    const int64_t r1 = min((int64_t)P.T, r0 + P.rows_per_chunk);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n < P.N) {
#pragma unroll 4
        for (int64_t t = r0 + rl; t < r1; t += 8) {
            float v[8];
            dn_load_bf<8>(P.dy + t * P.N + n, v);
            if (P.z) {
                float z[8];
                dn_load_bf<8>(P.z + t * P.N + n, z);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float d;
                    dn_act1<true>(P.act, z[i], d);
                    v[i] *= d;
                }
            }
            if (P.dz) dn_store_bf<8>(P.dz + t * P.N + n, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += v[i];
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
        if (P.out)
            __hip_atomic_store(&P.part[(int64_t)blockIdx.y * P.N + c], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        else
            P.part[(int64_t)blockIdx.y * P.N + c] = v;
    }
    // the last workgroup of these columns adds the chunks, in order
    __shared__ uint32_t s_last;
    if (!P.out || !dn_last(P.counters + (int64_t)blockIdx.x * DEC_CSTRIDE, (uint32_t)P.nchunks, &s_last) || c >= P.N) return;
    float v = 0.f;
#pragma unroll 8
    for (int i = 0; i < P.nchunks; ++i)
        v += __hip_atomic_load(&P.part[(int64_t)i * P.N + c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    dn_store_sum(P.out, c, v, P.out_f32, P.accumulate);
}

// bias gradient where k_dense_dz does not finish it (no rows, or more columns
// than counters): the chunks' sums.  32 columns a workgroup; eight chunk lanes
// add every eighth chunk, then are joined in order (nchunks 0: zero).
__global__ __launch_bounds__(256) void k_dense_colsum(ColsumParams P) {
    __shared__ float s_sum[8][33];
    const int cl = threadIdx.x & 31, l = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cl;
    float v = 0.f;
    if (c < P.N) {
#pragma unroll 8
        for (int i = l; i < P.nchunks; i += 8) v += P.part[(int64_t)i * P.N + c];
    }
    s_sum[l][cl] = v;
    __syncthreads();
    if (l > 0 || c >= P.N) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s_sum[i][cl];
    dn_store_sum(P.out, c, v, P.out_f32, P.accumulate);
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
    hipLaunchKernelGGL(k_dense_colsum, dim3((unsigned)((P.N + 31) / 32)), dim3(256), 0, st, P);
    return hipGetLastError();
}
hipError_t dense_linear_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_NT, DN_EPI_LINEAR>(P, tile, st);
}

}  // namespace moe
