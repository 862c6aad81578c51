// moe_rows.hip -- C = A B^T for few rows (M <= 256): the weights
// are read once, straight into the registers that the MFMA takes, and nothing
// else costs: bound by the weights' bytes and, below some 10 MB, by the launch
// and one round trip to memory.
//
// One workgroup takes 16 weight rows (8 with HALVES = 2), its 8 waves a part
// of K each, for MT blocks of 16 activation rows (8 with HALVES = 2).  v_mfma_f32_16x16x32_bf16: the weight rows are the row operand,
// the activation rows the column operand.  With HALVES = 2 operand
// rows 8..15 are the same 8 weight rows at another part of K and columns
// 8..15 the same activations there; the two diagonal blocks of the result are
// the two parts' sums, so no lane loads a byte twice and twice as many
// workgroups share a small matrix.  Parts are summed in LDS in their order.
//
// A bf16 activation is an operand as it is; an fp32 one enters as its three
// exact bf16 terms (three MFMAs on one weight fragment).
//
// Measured (MI355X, kernel alone in a graph): 1 x 2048 x 2048 3.6 us, 16 rows
// 5.2, 64 rows 7.9; 1 x 4096 x 22016 35 us (5.1 TB/s of weights); fp32 37 x
// 1000 x 520 4.5 us (8.4 with all rows in one workgroup, which then splits
// them all).  Tiles take over where a
// workgroup's activation reads outweigh its weights (moe_dense.hip).
#include "moe_dense.h"

namespace moe {

constexpr int RW_WAVES = 8;
// 32-k loads of a set in flight per wave (two such sets), for MT blocks of 16
// activation rows: what the registers hold
template <int XF32, int MT>
constexpr int RW_U = MT == 1 ? 6 : MT == 2 ? (XF32 ? 3 : 4) : (XF32 ? 2 : 3);

template <int XF32, int MT>
struct RwSet {
    u32x4 w[RW_U<XF32, MT>], x[RW_U<XF32, MT>][MT][XF32 ? 2 : 1];
};

template <int EPI, int XF32, int HALVES, int MT>
__global__ __launch_bounds__(RW_WAVES * 64) void k_dense_rows(DenseRowsParams P) {
    constexpr bool GATED = EPI == DN_EPI_GATED;
    constexpr int R = 16 / HALVES;             // weight rows per workgroup
    constexpr int RN = GATED ? R / 2 : R;      // output columns per workgroup
    constexpr int PARTS = RW_WAVES * HALVES;
    constexpr int U = RW_U<XF32, MT>;
    __shared__ __align__(16) float s_part[PARTS][MT * 16 / HALVES][R + 4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int half = HALVES == 2 ? li >> 3 : 0, r = HALVES == 2 ? li & 7 : li;
    const int n0 = blockIdx.x * RN, m0 = blockIdx.y * (MT * 16 / HALVES);
    // rows past the end read a valid row and are never stored
    const int n = min(n0 + (GATED ? r % RN : r), P.N - 1);
    const uint16_t *wr = (GATED && r >= RN ? P.b2 : P.b) + (int64_t)n * P.K;
    // this lane's part of K: 32-k pieces from k0 on
    const int pieces = (P.K + 31) / 32, per = (pieces + PARTS - 1) / PARTS;
    const int k0 = (wave * HALVES + half) * per * 32 + 8 * lg;

    auto load = [&](RwSet<XF32, MT> &s, int i0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = k0 + (i0 + i) * 32;
            // (a piece past the part or past K is zero in both operands)
            const bool in = i0 + i < per && k < P.K;
            const u32x4 z = {0u, 0u, 0u, 0u};
            s.w[i] = z;
#pragma unroll
            for (int q = 0; q < MT; ++q) {
                s.x[i][q][0] = z;
                if (XF32) s.x[i][q][XF32] = z;
            }
            if (in) {
                s.w[i] = *(const u32x4 *)(wr + k);
#pragma unroll
                for (int q = 0; q < MT; ++q) {
                    const int64_t at = (int64_t)min(m0 + 16 / HALVES * q + r, P.M - 1) * P.K + k;
                    if constexpr (XF32) {
                        s.x[i][q][0] = *(const u32x4 *)((const float *)P.a + at);
                        s.x[i][q][1] = *(const u32x4 *)((const float *)P.a + at + 4);
                    } else {
                        s.x[i][q][0] = *(const u32x4 *)((const uint16_t *)P.a + at);
                    }
                }
            }
        }
    };
    float4v acc[MT];
#pragma unroll
    for (int q = 0; q < MT; ++q) acc[q] = float4v{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const RwSet<XF32, MT> &s, int i0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i0 + i >= per) break;  // (uniform: a short part)
            const bf16x8 w = __builtin_bit_cast(bf16x8, s.w[i]);
#pragma unroll
            for (int q = 0; q < MT; ++q) {
                const u32x4 x0 = s.x[i][q][0];
                if constexpr (XF32) {
                    const u32x4 x1 = s.x[i][q][1];
                    const uint32_t f[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                    uint32_t p[8][3];
#pragma unroll
                    for (int e = 0; e < 8; ++e) dn_split3(__builtin_bit_cast(float, f[e]), p[e]);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const u32x4 v = {dn_high2(p[0][k], p[1][k]), dn_high2(p[2][k], p[3][k]), dn_high2(p[4][k], p[5][k]),
                                         dn_high2(p[6][k], p[7][k])};
                        acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, v), acc[q], 0, 0, 0);
                    }
                } else {
                    acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, x0), acc[q], 0, 0, 0);
                }
            }
        }
    };
    RwSet<XF32, MT> a, b;
    load(a, 0);
    for (int i0 = 0; i0 < per; i0 += 2 * U) {
        if (i0 + U < per) load(b, i0 + U);
        multiply(a, i0);
        if (i0 + U < per) {
            if (i0 + 2 * U < per) load(a, i0 + 2 * U);
            multiply(b, i0 + U);
        }
    }
    // D: rows 4 lg + v (weight rows), column li (activation row)
    if (HALVES == 1 || (li >> 3) == (lg >> 1)) {
#pragma unroll
        for (int q = 0; q < MT; ++q)
            *(float4v *)&s_part[wave * HALVES + half][16 / HALVES * q + r][HALVES == 2 ? 4 * (lg & 1) : 4 * lg] = acc[q];
    }
    __syncthreads();
    constexpr int Q = RN / 4;  // four columns per thread
    const int ml = tid / Q, m = m0 + ml, c = tid % Q * 4;
    if (ml >= MT * 16 / HALVES || m >= P.M || n0 + c >= P.N) return;
    float v[4], u[4];
    auto sum = [&](float(&o)[4], int col) {
        float4v q = *(const float4v *)&s_part[0][ml][col];
#pragma unroll
        for (int p = 1; p < PARTS; ++p) q += *(const float4v *)&s_part[p][ml][col];
        o[0] = q.x;
        o[1] = q.y;
        o[2] = q.z;
        o[3] = q.w;
    };
    sum(v, c);
    if constexpr (GATED) {
        sum(u, RN + c);
        dn_epi_gated<4>(P.e, P.M, P.N, m, n0 + c, v, u);
    } else {
        dn_epi_linear<4>(P.e, P.N, m, n0 + c, v);
    }
}

template <int EPI>
static hipError_t rows_t(const DenseRowsParams &P, hipStream_t st) {
    const int64_t rows = EPI == DN_EPI_GATED ? 2 * (int64_t)P.N : P.N;
    const DenseRowsShape S = dense_rows_shape(P.M, rows);
    const dim3 grid((unsigned)S.wgs, (unsigned)S.blocks), block(RW_WAVES * 64);
#define RW_LAUNCH(HALVES, MT)                                                                        \
    if (P.a_f32)                                                                                     \
        hipLaunchKernelGGL((k_dense_rows<EPI, 1, HALVES, MT>), grid, block, 0, st, P);                 \
    else                                                                                             \
        hipLaunchKernelGGL((k_dense_rows<EPI, 0, HALVES, MT>), grid, block, 0, st, P)
    if (S.halves && S.mt == 1) {
        RW_LAUNCH(2, 1);
    } else if (S.halves) {
        RW_LAUNCH(2, 2);
    } else if (S.mt == 1) {
        RW_LAUNCH(1, 1);
    } else if (S.mt == 2) {
        RW_LAUNCH(1, 2);
    } else {
        RW_LAUNCH(1, 4);
    }
#undef RW_LAUNCH
    return hipGetLastError();
}

hipError_t dense_rows_linear_launch(const DenseRowsParams &P, hipStream_t st) { return rows_t<DN_EPI_LINEAR>(P, st); }
hipError_t dense_rows_gated_launch(const DenseRowsParams &P, hipStream_t st) { return rows_t<DN_EPI_GATED>(P, st); }

}  // namespace moe
