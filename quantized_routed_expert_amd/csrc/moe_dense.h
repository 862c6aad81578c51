// moe_dense.h -- the tiled bf16 product under the dense operators (linear and
// the gated feed-forward block, forward and backward).
//
// One workgroup computes a BM x BN tile of C over a range of 64-k steps.  Both
// operands' slices of a step stream into LDS with 16-byte direct-to-LDS buffer
// loads, two steps or more ahead of their use.  Loads past an operand's edge return zero (the buffer's range
// check by rows, a per-lane mask along the contiguous axis), so every size
// that is a multiple of 8 along the contiguous axes runs the same code and no
// out-of-range value (a NaN next to the matrix) enters a sum.
//
// The weight side (N) feeds the MFMA's row operand, the activation side (M)
// its column operand: D's rows are n, four consecutive per lane, so a lane
// holds runs along the output's contiguous axis (joined to eight, dn_join).
//
// An operand whose rows run along k is read as 16-byte fragments (8 k); one
// whose rows run along m or n ("transposed") with ds_read_b64_tr_b16, which
// hands 16 lanes the columns of a 4 x 16 block.  Both give a lane of k-group
// g the k values 8g .. 8g+7 in order.
//
// LDS placement.  k-rows: 128 bytes (8 pieces of 16) per row, piece c of row r
// at c ^ s(r); the eight rows a quarter wave reads together have eight
// different s, so they touch all banks once.  Transposed: R*2 bytes per k,
// the 32-byte column block p of row k at p ^ g(k) within each 256 bytes; the
// eight k rows half a wave reads together have eight different g.  Direct
// loads write LDS in lane order, so the permutation is applied to the global
// address (within 128 or 256 contiguous bytes: the same cache lines).
//
// Measured (MI355X, 8192 x 4096 x 4096, bf16): A B^T 188 to 200 us (1.37 to
// 1.46 PFLOP/s, the library's kernel 171), A B 190 to 202 (library 200),
// A^T B 186 to 200 (library 229).  Large tiles keep the matrix cores busy 65
// to 75% of the cycles: a 256 x 256 tile's step is 2048 cycles of MFMA, 1536
// of LDS reads and 1024 of loads into LDS, and the clock falls to 1.9 GHz
// under that power.  Small ones wait for the path from L2.
#pragma once
#include "moe_device.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;

constexpr uint32_t DN_OOB = 0x80000000u;  // past every buffer's range (< 2^31 bytes)

// Buffer of `bytes` bytes from p (raw, stride 0): loads past it return zero.
__device__ __forceinline__ u32x4 dn_rsrc(const void *p, int bytes) {
    const uint64_t a = (uint64_t)p;
    return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, (uint32_t)max(bytes, 0), 0x00027000u};
}
// 16 bytes per lane from buffer offset `off` to LDS: lane l writes dst + 16 l.
// Counts in vmcnt.  As an instruction of its own and not the builtin: with
// that, the compiler waits for all such loads before every transposed LDS
// read, though they go to the other buffer.  It has no register result; LDS
// is read only after wait_vm and a barrier.
__device__ __forceinline__ void dn_load_lds(u32x4 rsrc, uint32_t dst, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(dst), "v"(off), "s"(rsrc)
                 : "memory", "m0");
}

// a constant as an argument
template <int N>
struct DnInt {
    static constexpr int value = N;
};

// ---------------------------------------------------------------------------
// Values and types
// ---------------------------------------------------------------------------
__device__ __forceinline__ float dn_bf(uint32_t bits16) { return __builtin_bit_cast(float, bits16 << 16); }
// two floats -> two bf16, round to nearest even (NaN kept)
__device__ __forceinline__ uint32_t dn_pack(float a, float b) {
    const __bf16 x = (__bf16)a, y = (__bf16)b;
    return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
}

// V consecutive bf16 / fp32 (16-byte aligned when V is 8, 8-byte for bf16 V = 4)
template <int V>
__device__ __forceinline__ void dn_load_bf(const uint16_t *p, float (&v)[V]) {
    if constexpr (V == 8) {
        const u32x4 q = *(const u32x4 *)p;
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = dn_bf(w[i] & 0xFFFFu);
            v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
        }
    } else {
        const u32x2 q = *(const u32x2 *)p;
        v[0] = dn_bf(q.x & 0xFFFFu);
        v[1] = __builtin_bit_cast(float, q.x & 0xFFFF0000u);
        v[2] = dn_bf(q.y & 0xFFFFu);
        v[3] = __builtin_bit_cast(float, q.y & 0xFFFF0000u);
    }
}
template <int V>
__device__ __forceinline__ void dn_load_f32(const float *p, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4v q = *(const float4v *)(p + i);
        v[i] = q.x;
        v[i + 1] = q.y;
        v[i + 2] = q.z;
        v[i + 3] = q.w;
    }
}
template <int V>
__device__ __forceinline__ void dn_store_bf(uint16_t *p, const float (&v)[V]) {
    if constexpr (V == 8)
        *(u32x4 *)p = u32x4{dn_pack(v[0], v[1]), dn_pack(v[2], v[3]), dn_pack(v[4], v[5]), dn_pack(v[6], v[7])};
    else
        *(u32x2 *)p = u32x2{dn_pack(v[0], v[1]), dn_pack(v[2], v[3])};
}
template <int V>
__device__ __forceinline__ void dn_store_f32(float *p, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) *(float4v *)(p + i) = float4v{v[i], v[i + 1], v[i + 2], v[i + 3]};
}

// An fp32 value as three bf16 terms (each in the high half of t[i]): 8
// significant bits each, cut toward zero, so the terms sum to the value
// exactly (24 bits) unless the last ones underflow.  An infinity or NaN stays
// in the first term alone (canonicalized: a NaN keeps its high mantissa bit).
__device__ __forceinline__ void dn_split3(float v, uint32_t (&t)[3]) {
    v = __builtin_canonicalizef(v);
    t[0] = __builtin_bit_cast(uint32_t, v);
    float r = v - __builtin_bit_cast(float, t[0] & 0xFFFF0000u);  // exact
    r = __builtin_fabsf(v) < __builtin_inff() ? r : 0.0f;
    t[1] = __builtin_bit_cast(uint32_t, r);
    t[2] = __builtin_bit_cast(uint32_t, r - __builtin_bit_cast(float, t[1] & 0xFFFF0000u));  // exact, at most 8 bits
}
// the high halves of a and b: two bf16
__device__ __forceinline__ uint32_t dn_high2(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }
template <int V>
__device__ __forceinline__ void dn_store_split3(uint16_t *p, size_t plane, const float (&v)[V]) {
    uint32_t t[V][3];
#pragma unroll
    for (int i = 0; i < V; ++i) dn_split3(v[i], t[i]);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if constexpr (V == 8)
            *(u32x4 *)(p + k * plane) = u32x4{dn_high2(t[0][k], t[1][k]), dn_high2(t[2][k], t[3][k]),
                                              dn_high2(t[4][k], t[5][k]), dn_high2(t[6][k], t[7][k])};
        else
            *(u32x2 *)(p + k * plane) = u32x2{dn_high2(t[0][k], t[1][k]), dn_high2(t[2][k], t[3][k])};
    }
}

// ---------------------------------------------------------------------------
// Activations in fp32.  The logistic function 1 / (1 + exp(-v)): exp
// overflows to infinity for large -v, which gives 0, its limit.
// GELU (tanh) uses (1 + tanh(q)) / 2 = logistic(2 q).
// ---------------------------------------------------------------------------
__device__ __forceinline__ float dn_sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }
constexpr float DN_GELU_C = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float DN_GELU_A = 0.044715f;

// act(v); with D, its derivative too
template <bool D>
__device__ __forceinline__ float dn_act1(int act, float v, float &d) {
    switch (act) {
        case DN_ACT_SILU: {
            const float s = dn_sigmoid(v);
            if (D) d = s * (1.0f + v * (1.0f - s));
            return v * s;
        }
        case DN_ACT_GELU: {
            const float c = 0.5f * (1.0f + erff(v * 0.70710678118654752f));
            if (D) d = c + v * 0.3989422804014327f * __expf(-0.5f * v * v);
            return v * c;
        }
        case DN_ACT_GELU_TANH: {
            const float s = dn_sigmoid(2.0f * DN_GELU_C * (v + DN_GELU_A * v * v * v));
            if (D) d = s + 2.0f * v * s * (1.0f - s) * DN_GELU_C * (1.0f + 3.0f * DN_GELU_A * v * v);
            return v * s;
        }
        case DN_ACT_RELU:
            if (D) d = v > 0.0f ? 1.0f : 0.0f;
            return v > 0.0f ? v : (v != v ? v : 0.0f);
        default:
            if (D) d = 1.0f;
            return v;
    }
}
// V values at once: f(constant activation) for a run-time one, so that one
// activation's code runs straight through
template <class F>
__device__ __forceinline__ void dn_for_act(int act, F f) {
    switch (act) {
        case DN_ACT_SILU: f(DnInt<DN_ACT_SILU>()); break;
        case DN_ACT_GELU: f(DnInt<DN_ACT_GELU>()); break;
        case DN_ACT_GELU_TANH: f(DnInt<DN_ACT_GELU_TANH>()); break;
        case DN_ACT_RELU: f(DnInt<DN_ACT_RELU>()); break;
        default: break;
    }
}
template <int V>
__device__ __forceinline__ void dn_act(int act, float (&v)[V]) {
    dn_for_act(act, [&](auto a) {
        float d;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = dn_act1<false>(decltype(a)::value, v[i], d);
    });
}
// v *= act'(z)
template <int V>
__device__ __forceinline__ void dn_times_slope(int act, const float (&z)[V], float (&v)[V]) {
    dn_for_act(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float d;
            dn_act1<true>(decltype(a)::value, z[i], d);
            v[i] *= d;
        }
    });
}

// ---------------------------------------------------------------------------
// Sums handed from workgroup to workgroup: device-scope accesses (they bypass
// the caches that XCDs do not share), counted on a counter that is zero
// between calls.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void dn_store_dev(float4v *p, float4v v) {
    uint64_t q[2];
    __builtin_memcpy(q, &v, 16);
    __hip_atomic_store((uint64_t *)p, q[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store((uint64_t *)p + 1, q[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float4v dn_load_dev(const float4v *p) {
    uint64_t q[2];
    q[0] = __hip_atomic_load((const uint64_t *)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    q[1] = __hip_atomic_load((const uint64_t *)p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    float4v v;
    __builtin_memcpy(&v, q, 16);
    return v;
}
// After a workgroup's dn_store_dev: whether it is the last of n (all threads
// get the answer; the last sets the counter back to zero).  s_last: LDS.
// The order needs no write-back of a whole L2 (an acquire-release count, 3 to
// 5 us a call): the sums alone are handed over, their stores are device-scope
// and complete (waited for by every wave) before the count, their loads
// device-scope after it.
__device__ __forceinline__ bool dn_last(uint32_t *counter, uint32_t n, uint32_t *s_last) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);  // this wave's stores have arrived
    __syncthreads();                // every wave's have
    if (threadIdx.x == 0) {
        const uint32_t before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *s_last = before == n - 1;
        if (before == n - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return *s_last != 0;
}

// ---------------------------------------------------------------------------
// Results: V consecutive columns.  The few-row kernel's go through pointers,
// a tile's through buffers whose range is the tile's rows: what lies past the
// last row or column is neither read nor written, without a branch, so a
// tile's loads stay in flight (with branches every wait was for all of them).
// ---------------------------------------------------------------------------
// two bf16 in each of V / 2 words
template <int V>
__device__ __forceinline__ void dn_unpack(u32x4 q, float (&v)[V]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        v[2 * i] = dn_bf(w[i] & 0xFFFFu);
        v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
}
template <int V>
__device__ __forceinline__ u32x4 dn_packed(const float (&v)[V]) {
    if constexpr (V == 8)
        return u32x4{dn_pack(v[0], v[1]), dn_pack(v[2], v[3]), dn_pack(v[4], v[5]), dn_pack(v[6], v[7])};
    else
        return u32x4{dn_pack(v[0], v[1]), dn_pack(v[2], v[3]), 0u, 0u};
}

// z = v + bias (kept in bf16 if asked); y = act(z) + residual
template <int V>
__device__ __forceinline__ void dn_epi_linear(const DenseEpi &e, int N, int64_t m, int n, float (&v)[V]) {
    const int64_t at = m * N + n;
    if (e.bias) {
        float b[V];
        dn_load_bf<V>(e.bias + n, b);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += b[i];
    }
    if (e.z) dn_store_bf<V>(e.z + at, v);
    if (e.act != DN_ACT_NONE) dn_act<V>(e.act, v);
    if (e.res) {
        float r[V];
        if (e.res_f32)
            dn_load_f32<V>((const float *)e.res + at, r);
        else
            dn_load_bf<V>((const uint16_t *)e.res + at, r);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += r[i];
    }
    if (e.y_f32)
        dn_store_f32<V>((float *)e.y + at, v);
    else
        dn_store_bf<V>((uint16_t *)e.y + at, v);
}
// h = act(g) u.  h enters the down product in bf16; for an fp32 y exactly, as
// fp32 (h_terms = 0: split where it is read) or three bf16 terms, so that y is
// as good as its type.  g and u kept for the backward pass are rounded to
// bf16 (the type that pass reads).
template <int V>
__device__ __forceinline__ void dn_epi_gated(const DenseEpi &e, int64_t M, int N, int64_t m, int n, float (&g)[V],
                                             float (&u)[V]) {
    if (e.gu) {
        dn_store_bf<V>(e.gu + m * (2 * (int64_t)N) + n, g);
        dn_store_bf<V>(e.gu + m * (2 * (int64_t)N) + N + n, u);
    }
    dn_act<V>(e.act, g);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] *= u[i];
    if (e.h_terms == 0)
        dn_store_f32<V>((float *)e.h + m * N + n, g);
    else if (e.h_terms == 3)
        dn_store_split3<V>(e.h + m * N + n, (size_t)M * N, g);
    else
        dn_store_bf<V>(e.h + m * N + n, g);
}

#ifdef __HIP_DEVICE_COMPILE__
// A tile's rows of a matrix of `ld` columns: element offsets from its first
// row; a null matrix is empty.
constexpr int DN_NO_COLUMN = 1 << 29;  // past the range of every tile, in elements of 2 and of 4 bytes
struct DnRows {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ DnRows(const void *p, int64_t m0, int rows, int64_t ld, int size) {
        r = __builtin_amdgcn_make_buffer_rsrc((uint8_t *)const_cast<void *>(p) + (p ? m0 * ld * size : 0), (short)0,
                                              p ? rows * (int)ld * size : 0, 0x00027000);
    }
    __device__ __forceinline__ u32x4 load16(int off) const { return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0); }
    __device__ __forceinline__ u32x4 load8(int off) const {
        const u32x2 q = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
        return u32x4{q.x, q.y, 0u, 0u};
    }
    __device__ __forceinline__ void store16(u32x4 v, int off) const { __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 0); }
    __device__ __forceinline__ void store8(u32x4 v, int off) const {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{v.x, v.y}, r, off, 0, 0);
    }
    // (an absent column's offset may pass 2^31: an unsigned number, past every range)
    __device__ __forceinline__ static int bytes(int at, int size) { return (int)((uint32_t)at * (uint32_t)size); }
    // V bf16 from element `at` on
    template <int V>
    __device__ __forceinline__ u32x4 load_bf(int at) const {
        return V == 8 ? load16(bytes(at, 2)) : load8(bytes(at, 2));
    }
    template <int V>
    __device__ __forceinline__ void store_bf(const float (&v)[V], int at) const {
        if (V == 8)
            store16(dn_packed<V>(v), bytes(at, 2));
        else
            store8(dn_packed<V>(v), bytes(at, 2));
    }
    template <int V>
    __device__ __forceinline__ void store_words(const uint32_t (&w)[V], int at) const {
#pragma unroll
        for (int i = 0; i < V; i += 4) store16(u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]}, bytes(at + i, 4));
    }
};
#endif

// ---------------------------------------------------------------------------
// Streaming one operand's slices into LDS
// ---------------------------------------------------------------------------
// g(k) of a transposed slice of R columns (a 64-column row is 128 bytes: its
// four blocks and the row's parity make the eight places)
template <int R>
__device__ __forceinline__ int dn_swap(int k) {
    return R >= 128 ? (k & 3) | (((k >> 3) & 1) << 2) : ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
}

// KC: R rows of 64 k, s(r) = r % 8.  Otherwise: 64 k of R columns.
template <int R, bool KC, int NW>
struct DnStream {
    static constexpr int NL = R * 128 / 1024 / NW;  // loads per wave and step
    static constexpr int BYTES = R * 128;
    static_assert(NL * NW * 1024 == BYTES, "whole wave loads");
    uint32_t voff[NL];
    int kpiece;  // k-rows: the first k of the 16-byte piece that this lane loads of each of its rows

    // row of the tile whose piece (k-rows) the lane loads with load j
    __device__ __forceinline__ static int row(int j, int wave, int lane) { return (j * NW + wave) * 8 + (lane >> 3); }
    // ld in elements; cols: columns left from the tile's first (transposed).
    // pair != 0 (gated): the tile's rows are groups of `pair` rows of one
    // matrix and the same rows of another
    __device__ __forceinline__ void setup(int wave, int lane, int64_t ld, int64_t cols, int pair) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            if constexpr (KC) {
                const int r = row(j, wave, lane);
                const int c = (lane & 7) ^ (r & 7);
                kpiece = c * 8;
                voff[j] = (uint32_t)((pair ? r / (2 * pair) * pair + r % pair : r) * (int)ld * 2 + c * 16);
            } else {
                const int at = (j * NW + wave) * 1024 + lane * 16;
                const int k = at / (R * 2), p = (at % (R * 2)) / 16;
                const int c = p ^ (dn_swap<R>(k) << 1);
                voff[j] = c * 8 < cols ? (uint32_t)(k * (int)ld * 2 + c * 16) : DN_OOB;
            }
        }
    }
    // load j; past: OR-ed into the offset (DN_OOB: this lane's k is past K)
    __device__ __forceinline__ void issue(int j, u32x4 r, uint32_t dst, int wave, uint32_t past) {
        dn_load_lds(r, dst + (j * NW + wave) * 1024, KC ? voff[j] | past : voff[j]);
    }
    __device__ __forceinline__ uint32_t past(int kleft) const { return KC && kpiece >= kleft ? DN_OOB : 0u; }
};

// Two blocks' results (lane group lg: four columns from 4 lg on of each) ->
// eight consecutive columns from dn_joined(lg) on of the pair, so that a bf16
// store is 16 bytes and a row's four lanes write 64 in one piece.  (Stores of
// 16 bytes in every 32 took 8 us of a 256 x 256 tile; the path takes one
// 64-byte piece of a line at a time.)
__device__ __forceinline__ int dn_joined(int lg) { return 16 * (lg & 1) + 8 * (lg >> 1); }
__device__ __forceinline__ void dn_join(float4v a, float4v b, float (&v)[8]) {
    const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // lane groups (0 1 2 3) of a and b -> a0 b0 a2 b2 and a1 b1 a3 b3
        const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, av[k]), __builtin_bit_cast(uint32_t, bv[k]),
                                                        false, false);
        const uint32_t lo = r[0], hi = r[1];  // (copied out: a bit cast of a component reads the first)
        v[k] = __builtin_bit_cast(float, lo);
        v[4 + k] = __builtin_bit_cast(float, hi);
    }
}

// Workgroup -> tile: workgroups go round robin over the 8 XCDs, so each XCD
// gets a contiguous run of the tile order; the order walks groups of 8 tile
// rows column by column, so the tiles an XCD works on at a time share rows of
// both operands in its L2.
__device__ __forceinline__ void dn_tile(const DenseParams &P, int b, int &tm, int &tn) {
    const int total = P.tiles_m * P.tiles_n;
    const int q = total >> 3, r = total & 7, x = b & 7;
    const int t = x * q + min(x, r) + (b >> 3);
    constexpr int G = 8;
    const int per = G * P.tiles_n;
    const int grp = t / per, in = t - grp * per;
    const int rows = min(G, P.tiles_m - grp * G);
    tn = in / rows;
    tm = grp * G + in - tn * rows;
}

struct DnTrue {
    static constexpr bool value = true;
};
struct DnFalse {
    static constexpr bool value = false;
};

// Where an operand's next loads read: the current product's matrix at the
// step's k.  The range (bytes from the pointer) shrinks with it and is zero
// after the last step, so loads past the end fetch nothing.
template <bool KC, bool B>
struct DnCursor {
    const uint16_t *p, *p2;  // p2: the up projection
    int64_t step;            // elements from one step to the next
    int kleft;               // k left in this product
    int bytes;               // k-rows: the range
    int ld, seg, left;       // left: steps not yet loaded

    // first: the tile's first row or column; n: its rows
    __device__ __forceinline__ void open(const DenseParams &P, int i, int k0, int64_t first, int n) {
        const DenseSeg &g = P.seg[i];
        const int64_t l = B ? g.ldb : g.lda;
        const int64_t at = KC ? first * l + k0 : k0 * l + first;
        seg = i;
        ld = (int)l;
        kleft = g.K - k0;
        p = (B ? g.b : g.a) + at;
        p2 = B ? g.b2 + at : nullptr;
        step = KC ? DN_BK : DN_BK * l;
        bytes = (n * ld - k0) * 2;
    }
    __device__ __forceinline__ void advance(const DenseParams &P, int64_t first, int n) {
        p += step;
        p2 += step;
        bytes -= DN_BK * 2;
        kleft -= DN_BK;
        --left;
        if (kleft <= 0 && left > 0) open(P, seg + 1, 0, first, n);
    }
    // transposed: the rows left of this step, from the tile's first column on
    __device__ __forceinline__ int range(int64_t first) const {
        return left <= 0 ? 0 : KC ? bytes : (min(DN_BK, kleft) * ld - (int)first) * 2;
    }
};

// Main loop.  A step's 64 k are two halves of 32.  Fragments are double
// buffered in registers: while the MFMAs of one half run, the other half's
// fragments are read, so no MFMA waits for LDS.  LDS holds D slices of A
// and D + 1 of B (a slice: one operand, one step).  The first half of step s
// loads B of s+D into its spare slice, the second half A of s+D into the one
// that A of s has just been read from.  One barrier, in the middle of a step,
// says both that every wave has read step s and that step s+1 has landed.
// Loads go out through the whole step: the path into LDS moves 64 bytes a
// cycle, half the step's MFMA time for a 256 x 256 tile, and loads bunched in
// one half of it hold up the MFMAs behind them (measured, 8192 x 4096 x 4096:
// all within a quarter step 222 us, half a step 196 us).
//
// KG > 1: the workgroup's waves are KG groups, each with its own slices and
// its own part of the tile's steps; their sums are added in LDS, in order, at
// the end.  Small tiles spend their time waiting for loads; the groups keep
// KG times as many in flight and take 1 / KG of the steps.
template <int BM, int BN, int KG, int D>
constexpr int DN_LDS = KG * (D * BM + (D + 1) * BN) * 128;

#ifdef __HIP_DEVICE_COMPILE__  // (the host pass needs the kernels' stubs alone: it drops those that use the buffer builtins)
template <int BM, int BN, int WM, int WN, int KG, int D, int FORM, int EPI, int ACT>
__device__ __forceinline__ void dense_body(const DenseParams &P, int tile, int split, uint8_t *smem) {
    constexpr int NW = WM * WN;  // waves per group
    constexpr bool AKC = FORM != DN_TN, BKC = FORM == DN_NT;
    constexpr bool GATED = EPI == DN_EPI_GATED;
    constexpr int MS = BM / WM / 16, NS = BN / WN / 16;  // 16 x 16 blocks per wave
    static_assert(NS % 2 == 0, "pairs of blocks");
    constexpr int PAIR = GATED ? 16 : 0;  // blocks of 16 gate rows and the same up rows in turn
    typedef DnStream<BM, AKC, NW> SA;
    typedef DnStream<BN, BKC, NW> SB;
    constexpr int RING = D * SA::BYTES + (D + 1) * SB::BYTES;
    static_assert(RING * KG == DN_LDS<BM, BN, KG, D>, "slices");
    static_assert(KG == 1 || BM * BN * 4 <= RING, "the groups' sums fit the slices");
    lds_u8 *const lds_all = (lds_u8 *)smem;

    const int lane = threadIdx.x & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int grp = KG > 1 ? wave_all / NW : 0;
    const int wave = KG > 1 ? wave_all % NW : wave_all;
    const int wm = wave / WN, wn = wave % WN;
    lds_u8 *const lds = lds_all + grp * RING;
    int tm, tn;
    dn_tile(P, tile, tm, tn);
    const int64_t m0 = (int64_t)tm * BM;
    constexpr int BNF = GATED ? BN / 2 : BN;  // output columns per tile
    const int64_t n0 = (int64_t)tn * BNF;
    const int rows = (int)min((int64_t)BM, P.M - m0), cols = (int)min((int64_t)BNF, P.N - n0);
    // this group's steps (a group past the end multiplies zeros)
    const int s_wg = split * P.steps_per_split, e_wg = min(P.steps, s_wg + P.steps_per_split);
    const int nstep = KG > 1 ? (e_wg - s_wg + KG - 1) / KG : e_wg - s_wg;
    const int s0 = s_wg + grp * nstep;

    SA sa;
    SB sb;
    DnCursor<AKC, false> ca;
    DnCursor<BKC, true> cb;
    {
        int seg = 0, k0 = s0 * DN_BK;
        while (seg + 1 < P.nseg && k0 >= P.seg[seg].K) {  // (steps of a product: its K rounded up)
            k0 -= (P.seg[seg].K + DN_BK - 1) / DN_BK * DN_BK;
            ++seg;
        }
        ca.open(P, seg, k0, m0, rows);
        cb.open(P, seg, k0, n0, cols);
        ca.left = cb.left = min(nstep, e_wg - s0);
    }
    sa.setup(wave, lane, P.seg[0].lda, rows, 0);
    sb.setup(wave, lane, P.seg[0].ldb, cols, PAIR);
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

    // an operand's next loads: *_begin(slice), *_one(0 .. NL - 1), then the cursor's advance
    u32x4 ra, rb, ru;
    uint32_t pa, pb, da, db;
    auto a_begin = [&](int slice) {
        da = lds0 + slice * SA::BYTES;
        pa = sa.past(ca.kleft);
        ra = dn_rsrc(ca.p, ca.range(m0));
    };
    auto a_one = [&](int j) { sa.issue(j, ra, da, wave, pa); };
    auto b_begin = [&](int slice) {
        db = lds0 + D * SA::BYTES + slice * SB::BYTES;
        pb = sb.past(cb.kleft);
        rb = dn_rsrc(cb.p, cb.range(n0));
        if constexpr (GATED) ru = dn_rsrc(cb.p2, cb.range(n0));
    };
    auto b_one = [&](int j) {
        // (8 rows per load and wave: all of one matrix)
        const bool up = GATED && (((j * NW + wave) * 8 / (PAIR ? PAIR : 1)) & 1);
        sb.issue(j, up ? ru : rb, db, wave, pb);
    };

    float4v acc[MS][NS];
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
        for (int j = 0; j < NS; ++j) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};

    // fragment addresses within a stage
    const int li = lane & 15, lg = lane >> 4;
    const int a_row = wm * (BM / WM), b_row = wn * (BN / WN);
    const uint32_t a_kc = (uint32_t)((a_row + li) * 128 + ((lg ^ (li & 7)) << 4));
    const uint32_t b_kc = (uint32_t)((b_row + li) * 128 + ((lg ^ (li & 7)) << 4));
    const int tk = 8 * lg + (li >> 2);  // the k row this lane addresses (and tk + 4, + 32: the same g)
    const int ga = dn_swap<BM>(tk), gb = dn_swap<BN>(tk);
    const uint32_t a_tr = (uint32_t)(tk * BM * 2 + (li & 3) * 8), b_tr = (uint32_t)(tk * BN * 2 + (li & 3) * 8);

    auto frag_kc = [&](lds_u8 *base, uint32_t at, int row, int kk) {
        return *(lds_bf16x8 *)(base + ((at ^ (kk << 6)) + row * 128));
    };
    auto frag_tr = [&](lds_u8 *base, uint32_t at, int blk, int ld2, int kk) {
        const uint32_t o = at + (blk << 5) + kk * 32 * ld2;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(base + o));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(base + o + 4 * ld2));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, s16x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w});
    };
    bf16x8 fa[2][MS], fb[2][NS];
    // fragment q of a half: the weight side's first, then the activations'
    auto read_one = [&](int set, lds_u8 *ba, lds_u8 *bb, int kk, int q) {
        if (q < NS)
            fb[set][q] = BKC ? frag_kc(bb, b_kc, 16 * q, kk) : frag_tr(bb, b_tr, (b_row / 16 + q) ^ gb, BN * 2, kk);
        else
            fa[set][q - NS] = AKC ? frag_kc(ba, a_kc, 16 * (q - NS), kk) : frag_tr(ba, a_tr, (a_row / 16 + q - NS) ^ ga, BM * 2, kk);
    };
    constexpr int NF = NS + MS;
    // one half: MS groups of NS MFMAs on `set`, between them the reads of the
    // other half into the other set (done before the last group, so that the
    // next half starts at once) and one operand's next loads; the order is
    // fixed (the compiler's own gathers the reads in front of a full wait)
    auto half = [&](auto load_a, int set, lds_u8 *ba, lds_u8 *bb, int kk) {
        constexpr bool LA = decltype(load_a)::value;
        constexpr int NL = LA ? SA::NL : SB::NL;
        constexpr int RG = MS > 1 ? MS - 1 : 1;
#pragma unroll
        for (int i = 0; i < MS; ++i) {
#pragma unroll
            for (int j = 0; j < NL; ++j)
                if (j * MS / NL == i) {
                    if (LA)
                        a_one(j);
                    else
                        b_one(j);
                }
#pragma unroll
            for (int j = 0; j < NS; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < NF; ++q)
                if (q * RG / NF == i) read_one(set ^ 1, ba, bb, kk, q);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

#pragma unroll
    for (int t = 0; t < D; ++t) {
        b_begin(t);
#pragma unroll
        for (int j = 0; j < SB::NL; ++j) b_one(j);
        cb.advance(P, n0, cols);
        a_begin(t);
#pragma unroll
        for (int j = 0; j < SA::NL; ++j) a_one(j);
        ca.advance(P, m0, rows);
    }
    constexpr int NLD = SA::NL + SB::NL;  // loads of a step
    wait_vm<(D - 1) * NLD>();
    lds_barrier();
    lds_u8 *const lds_b = lds + D * SA::BYTES;
#pragma unroll
    for (int q = 0; q < NF; ++q) read_one(0, lds, lds_b, 0, q);
    // slices of step s: A's sl_a = s % D, B's sl_b = s % (D + 1)
    for (int s = 0, sl_a = 0, sl_b = 0; s < nstep; ++s) {
        b_begin(sl_b == 0 ? D : sl_b - 1);
        half(DnFalse(), 0, lds + sl_a * SA::BYTES, lds_b + sl_b * SB::BYTES, 1);
        cb.advance(P, n0, cols);
        a_begin(sl_a);
        wait_vm<(D - 2) * NLD + SB::NL>();  // all but the loads after step s + 1's
        lds_barrier();
        sl_a = sl_a == D - 1 ? 0 : sl_a + 1;
        sl_b = sl_b == D ? 0 : sl_b + 1;
        half(DnTrue(), 1, lds + sl_a * SA::BYTES, lds_b + sl_b * SB::BYTES, 0);
        ca.advance(P, m0, rows);
    }
    wait_vm<0>();  // (the last loads: their LDS is released when the workgroup ends)

    // Results in units: (row block i, pair of column blocks).  With groups,
    // unit u belongs to group u % KG, which adds the groups' sums from LDS.
    // A unit's two column blocks are j, j + 1; gated: the gate blocks j, j + 2
    // (with the up blocks after them), or one gate block where a wave has one.
    constexpr int JP = GATED && NS == 2 ? 1 : 2, UJ = NS / (GATED ? 2 * JP : JP), UB = NS / UJ;  // UB: blocks of a unit
    typedef float4v LdsSums[KG][NW][MS * NS][64];
    if constexpr (KG > 1) {
        __syncthreads();
        LdsSums &sums = *(LdsSums *)smem;
#pragma unroll
        for (int i = 0; i < MS; ++i)
#pragma unroll
            for (int j = 0; j < NS; ++j) sums[grp][wave][i * NS + j][lane] = acc[i][j];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MS; ++i)
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                if ((i * UJ + j / UB) % KG != grp) continue;
                float4v v = sums[0][wave][i * NS + j][lane];
#pragma unroll
                for (int g = 1; g < KG; ++g) v += sums[g][wave][i * NS + j][lane];
                acc[i][j] = v;
            }
    }
    // Split: each workgroup leaves its tile's sums, lane by lane; the last one
    // of the tile adds them in the splits' order.
    if (P.splits > 1) {
        float4v *const parts = (float4v *)P.part + (int64_t)tile * P.splits * (BM * BN / 4) + wave * (MS * NS * 64) + lane;
#pragma unroll
        for (int i = 0; i < MS; ++i)
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                if (KG > 1 && (i * UJ + j / UB) % KG != grp) continue;
                dn_store_dev(parts + (int64_t)split * (BM * BN / 4) + (i * NS + j) * 64, acc[i][j]);
            }
        if (!dn_last(P.counters + (int64_t)tile * DEC_CSTRIDE, (uint32_t)P.splits, (uint32_t *)(smem + DN_LDS<BM, BN, KG, D> - 16)))
            return;
#pragma unroll
        for (int i = 0; i < MS; ++i)
#pragma unroll
            for (int uj = 0; uj < UJ; ++uj) {
                if (KG > 1 && (i * UJ + uj) % KG != grp) continue;
                float4v v[UB];
#pragma unroll
                for (int j = 0; j < UB; ++j) v[j] = float4v{0.f, 0.f, 0.f, 0.f};
                constexpr int Q = 4;  // splits' sums in flight
                for (int q = 0; q < P.splits; q += Q) {
                    float4v w[Q][UB];
#pragma unroll
                    for (int a = 0; a < Q; ++a)
#pragma unroll
                        for (int j = 0; j < UB; ++j)
                            w[a][j] = dn_load_dev(parts + (int64_t)min(q + a, P.splits - 1) * (BM * BN / 4) + (i * NS + uj * UB + j) * 64);
#pragma unroll
                    for (int a = 0; a < Q; ++a)
                        if (q + a < P.splits) {
#pragma unroll
                            for (int j = 0; j < UB; ++j) v[j] += w[a][j];
                        }
                }
#pragma unroll
                for (int j = 0; j < UB; ++j) acc[i][uj * UB + j] = v[j];
            }
    }
    auto row = [&](int i) { return a_row + 16 * i + li; };  // of the tile
    const int N = P.N;
    if constexpr (GATED) {
        constexpr int V = JP == 2 ? 8 : 4;
        const DenseEpi &e = P.e;
        const int64_t plane = (int64_t)P.M * N;
        const DnRows gu(e.gu, m0, rows, 2 * (int64_t)N, 2);
        const DnRows h0(e.h, m0, rows, N, 2), h1(e.h_terms == 3 ? e.h + plane : nullptr, m0, rows, N, 2),
            h2(e.h_terms == 3 ? e.h + 2 * plane : nullptr, m0, rows, N, 2), hf(e.h_terms == 0 ? e.h : nullptr, m0, rows, N, 4);
#pragma unroll
        for (int i = 0; i < MS; ++i) {
#pragma unroll
            for (int uj = 0; uj < UJ; ++uj) {
                if (KG > 1 && (i * UJ + uj) % KG != grp) continue;
                const int j0 = uj * 2 * JP;
                float g[V], u[V];
                if constexpr (JP == 2) {
                    dn_join(acc[i][j0], acc[i][j0 + 2], g);
                    dn_join(acc[i][j0 + 1], acc[i][j0 + 3], u);
                } else {
                    const float4v a = acc[i][j0], b = acc[i][j0 + 1];
                    g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w;
                    u[0] = b.x, u[1] = b.y, u[2] = b.z, u[3] = b.w;
                }
                int n = (int)n0 + (b_row >> 1) + 16 * JP * uj + (JP == 2 ? dn_joined(lg) : 4 * lg);
                n = n < N ? n : DN_NO_COLUMN;
                if (e.gu) {
                    gu.template store_bf<V>(g, 2 * row(i) * N + n);
                    gu.template store_bf<V>(u, 2 * row(i) * N + N + n);
                }
                dn_act<V>(ACT, g);
#pragma unroll
                for (int k = 0; k < V; ++k) g[k] *= u[k];
                const int at = row(i) * N + n;
                // (h's roundings: see dn_epi_gated)
                if (e.h_terms == 1) {
                    h0.template store_bf<V>(g, at);
                } else if (e.h_terms == 3) {
                    uint32_t t[V][3];
#pragma unroll
                    for (int k = 0; k < V; ++k) dn_split3(g[k], t[k]);
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        u32x4 w = {dn_high2(t[0][q], t[1][q]), dn_high2(t[2][q], t[3][q]), 0u, 0u};
                        if constexpr (V == 8) {
                            w.z = dn_high2(t[4][q], t[5][q]);
                            w.w = dn_high2(t[6][q], t[7][q]);
                        }
                        const DnRows &h = q == 0 ? h0 : q == 1 ? h1 : h2;
                        if (V == 8)
                            h.store16(w, DnRows::bytes(at, 2));
                        else
                            h.store8(w, DnRows::bytes(at, 2));
                    }
                } else {
                    uint32_t w[V];
#pragma unroll
                    for (int k = 0; k < V; ++k) w[k] = __builtin_bit_cast(uint32_t, g[k]);
                    hf.template store_words<V>(w, at);
                }
            }
        }
    } else {
        // V = 8: a unit's joined blocks (bf16 results); V = 4: fp32 results,
        // where four columns are 16 bytes and a row's four lanes 64.  IN: what
        // is read at a result's place: 0 nothing, 1 bf16 values (a residual),
        // 2 fp32 values, 3 gate and up.
        auto finish = [&](auto width, auto reads) {
            constexpr int V = decltype(width)::value, IN = decltype(reads)::value, SUB = 8 / V;
            const DenseEpi &e = P.e;
            // row blocks whose input is in flight ahead of their use
            constexpr int AHEAD = IN == 0 ? 1 : IN == 2 && V == 8 ? 2 : 3;  // (what the registers hold)
            constexpr int PRE = MS < AHEAD ? MS : AHEAD;
            constexpr int LD = EPI == DN_EPI_DGATED ? 2 : 1;
            u32x4 in[PRE][UJ][SUB][2];
            int col[UJ][SUB];
            float bias[UJ][SUB][V];
            const DnRows from(EPI == DN_EPI_DGATED ? e.gu_in : e.res, m0, rows, LD * (int64_t)N, IN == 2 ? 4 : 2);
            const DnRows brow(EPI == DN_EPI_LINEAR ? e.bias : nullptr, 0, 1, N, 2);
#pragma unroll
            for (int uj = 0; uj < UJ; ++uj)
#pragma unroll
                for (int k = 0; k < SUB; ++k) {
                    const int n = (int)n0 + b_row + 32 * uj + (V == 8 ? dn_joined(lg) : 16 * k + 4 * lg);
                    col[uj][k] = n < N ? n : DN_NO_COLUMN;
                    if constexpr (EPI == DN_EPI_LINEAR) dn_unpack<V>(brow.template load_bf<V>(col[uj][k]), bias[uj][k]);
                }
            auto fetch = [&](int i) {
                if constexpr (IN > 0) {
#pragma unroll
                    for (int uj = 0; uj < UJ; ++uj) {
                        if (KG > 1 && (i * UJ + uj) % KG != grp) continue;
#pragma unroll
                        for (int k = 0; k < SUB; ++k) {
                            const int at = LD * row(i) * N + col[uj][k];
                            u32x4(&q)[2] = in[i % PRE][uj][k];
                            if constexpr (IN == 2) {
                                q[0] = from.load16(DnRows::bytes(at, 4));
                                if constexpr (V == 8) q[1] = from.load16(DnRows::bytes(at + 4, 4));
                            } else {
                                q[0] = from.template load_bf<V>(at);
                                if constexpr (IN == 3) q[1] = from.template load_bf<V>(at + N);
                            }
                        }
                    }
                }
            };
            const DnRows y(e.y, m0, rows, N, V == 4 ? 4 : 2), z(e.z, m0, rows, N, 2);
            const DnRows dgu(EPI == DN_EPI_DGATED ? e.dgu : nullptr, m0, rows, 2 * (int64_t)N, 2), h(e.h, m0, rows, N, 2);
#pragma unroll
            for (int i = 0; i < PRE; ++i) fetch(i);
#pragma unroll
            for (int i = 0; i < MS; ++i) {
#pragma unroll
                for (int uj = 0; uj < UJ; ++uj) {
                    if (KG > 1 && (i * UJ + uj) % KG != grp) continue;
                    const float4v v0 = acc[i][2 * uj], v1 = acc[i][2 * uj + 1];
                    float joined[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                    if constexpr (V == 8) dn_join(v0, v1, joined);
#pragma unroll
                    for (int k = 0; k < SUB; ++k) {
                        float v[V];
#pragma unroll
                        for (int c = 0; c < V; ++c) v[c] = joined[V * k + c];
                        const u32x4(&q)[2] = in[i % PRE][uj][k];
                        if constexpr (EPI == DN_EPI_DGATED) {
                            // v = dh: h = act(g) u, dg = dh u act'(g), du = dh act(g),
                            // each rounded once to bf16, the type their products take
                            float g[V], u[V], hv[V], du[V];
                            dn_unpack<V>(q[0], g);
                            dn_unpack<V>(q[1], u);
#pragma unroll
                            for (int c = 0; c < V; ++c) {
                                float d;
                                const float a = dn_act1<true>(ACT, g[c], d);
                                hv[c] = a * u[c];
                                du[c] = v[c] * a;
                                v[c] = v[c] * u[c] * d;
                            }
                            h.template store_bf<V>(hv, row(i) * N + col[uj][k]);
                            dgu.template store_bf<V>(v, 2 * row(i) * N + col[uj][k]);
                            dgu.template store_bf<V>(du, 2 * row(i) * N + N + col[uj][k]);
                        } else {
                            // z = v + bias, y = act(z) + residual
                            const int at = row(i) * N + col[uj][k];
#pragma unroll
                            for (int c = 0; c < V; ++c) v[c] += bias[uj][k][c];
                            if (e.z) z.template store_bf<V>(v, at);
                            if (ACT != DN_ACT_NONE) dn_act<V>(ACT, v);
                            if constexpr (IN == 1) {
                                float r[V];
                                dn_unpack<V>(q[0], r);
#pragma unroll
                                for (int c = 0; c < V; ++c) v[c] += r[c];
                            }
                            if constexpr (IN == 2) {
                                const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
                                for (int c = 0; c < V; ++c) v[c] += __builtin_bit_cast(float, w[c]);
                            }
                            if constexpr (V == 4) {
                                uint32_t w[V];
#pragma unroll
                                for (int c = 0; c < V; ++c) w[c] = __builtin_bit_cast(uint32_t, v[c]);
                                y.template store_words<V>(w, at);
                            } else {
                                y.template store_bf<V>(v, at);
                            }
                        }
                    }
                }
                if (i + PRE < MS) fetch(i + PRE);
            }
        };
        if constexpr (EPI == DN_EPI_DGATED) {
            finish(DnInt<8>(), DnInt<3>());
        } else {
            const int in = !P.e.res ? 0 : P.e.res_f32 ? 2 : 1;
            if (P.e.y_f32) {
                if (in == 0)
                    finish(DnInt<4>(), DnInt<0>());
                else if (in == 1)
                    finish(DnInt<4>(), DnInt<1>());
                else
                    finish(DnInt<4>(), DnInt<2>());
            } else {
                if (in == 0)
                    finish(DnInt<8>(), DnInt<0>());
                else if (in == 1)
                    finish(DnInt<8>(), DnInt<1>());
                else
                    finish(DnInt<8>(), DnInt<2>());
            }
        }
    }
}
#endif

template <int BM, int BN, int WM, int WN, int KG, int D, int FORM, int EPI, int ACT>
__global__ __launch_bounds__(WM *WN *KG * 64, WM *WN *KG / 4) void k_dense(DenseParams P) {
#ifdef __HIP_DEVICE_COMPILE__
    __shared__ __align__(1024) uint8_t smem[DN_LDS<BM, BN, KG, D>];
    dense_body<BM, BN, WM, WN, KG, D, FORM, EPI, ACT>(P, blockIdx.x, blockIdx.y, smem);
#endif
}

// Bias gradient: the row chunks' sums (no chunk: zero).  DN_SUM_COLS columns a
// workgroup; each of its chunk lanes adds every THREADS / DN_SUM_COLS-th
// chunk, then they are joined in order.
constexpr int DN_SUM_COLS = 32;
template <int THREADS>
__device__ __forceinline__ void dn_colsum(const ColsumParams &P, int block, float *sums) {
    constexpr int LANES = THREADS / DN_SUM_COLS, LD = DN_SUM_COLS + 1;
    const int cl = threadIdx.x % DN_SUM_COLS, l = threadIdx.x / DN_SUM_COLS;
    const int c = block * DN_SUM_COLS + cl;
    float v = 0.f;
    if (c < P.N) {
#pragma unroll 8
        for (int i = l; i < P.nchunks; i += LANES) v += P.part[(int64_t)i * P.N + c];
    }
    sums[l * LD + cl] = v;
    __syncthreads();
    if (l > 0 || c >= P.N) return;
#pragma unroll
    for (int i = 1; i < LANES; ++i) v += sums[i * LD + cl];
    if (P.out_f32) {
        float *o = (float *)P.out + c;
        *o = P.accumulate ? *o + v : v;
    } else {
        uint16_t *o = (uint16_t *)P.out + c;
        if (P.accumulate) v += dn_bf(*o);
        *o = (uint16_t)(dn_pack(v, 0.f) & 0xFFFFu);
    }
}

// A backward pass's last products, which do not depend on each other, in one
// launch: the input gradient (A B) and the weight gradients (A^T B), those
// with the longest tiles first, then the bias gradient's sums.  Apart they
// would each end in a round of tiles that leaves CUs idle, and wait for the
// launch before them.
template <int BM, int BN, int WM, int WN, int KG, int D>
__global__ __launch_bounds__(WM *WN *KG * 64, WM *WN *KG / 4) void k_dense_grads(DenseGradsParams A) {
#ifdef __HIP_DEVICE_COMPILE__
    __shared__ __align__(1024) uint8_t smem[DN_LDS<BM, BN, KG, D>];
    int b = blockIdx.x, i = 0;
    while (i < A.n && b >= A.tiles[i]) b -= A.tiles[i++];
    if (i == A.n)
        dn_colsum<WM * WN * KG * 64>(A.sum, b, (float *)smem);
    else if (i == A.dx_at)
        dense_body<BM, BN, WM, WN, KG, D, DN_NN, DN_EPI_LINEAR, DN_ACT_NONE>(A.p[i], b, 0, smem);
    else
        dense_body<BM, BN, WM, WN, KG, D, DN_TN, DN_EPI_LINEAR, DN_ACT_NONE>(A.p[i], b, 0, smem);
#endif
}

// launch(tile shape...) for a tile
#define DN_TILE_SWITCH(tile, LAUNCH)                             \
    switch (tile) {                                              \
        case DN_TILE_256x256: LAUNCH(512, 256, 256, 2, 4, 1, 2); break; \
        case DN_TILE_256x128: LAUNCH(512, 256, 128, 4, 2, 1, 2); break; \
        case DN_TILE_128x128: LAUNCH(512, 128, 128, 2, 2, 2, 2); break; \
        case DN_TILE_128x64: LAUNCH(512, 128, 64, 2, 2, 2, 3); break;   \
        case DN_TILE_64x64: LAUNCH(1024, 64, 64, 2, 2, 4, 2); break;    \
        default: return hipErrorInvalidValue;                    \
    }

// One product of the given form and epilogue.
template <int FORM, int EPI, int ACT>
hipError_t dense_tile_t(const DenseParams &P, int tile, hipStream_t st) {
    const dim3 grid((unsigned)(P.tiles_m * P.tiles_n), (unsigned)P.splits);
#define DN_LAUNCH(THREADS, ...) hipLaunchKernelGGL((k_dense<__VA_ARGS__, FORM, EPI, ACT>), grid, dim3(THREADS), 0, st, P)
    DN_TILE_SWITCH(tile, DN_LAUNCH)
#undef DN_LAUNCH
    return hipGetLastError();
}
template <int FORM, int EPI>
hipError_t dense_launch_t(const DenseParams &P, int tile, hipStream_t st) {
    constexpr bool A = FORM == DN_NT || EPI != DN_EPI_LINEAR;  // with an activation
    switch (A ? P.e.act : DN_ACT_NONE) {
        case DN_ACT_SILU: return dense_tile_t<FORM, EPI, A ? DN_ACT_SILU : 0>(P, tile, st);
        case DN_ACT_GELU: return dense_tile_t<FORM, EPI, A ? DN_ACT_GELU : 0>(P, tile, st);
        case DN_ACT_GELU_TANH: return dense_tile_t<FORM, EPI, A ? DN_ACT_GELU_TANH : 0>(P, tile, st);
        case DN_ACT_RELU: return dense_tile_t<FORM, EPI, A ? DN_ACT_RELU : 0>(P, tile, st);
        default: return dense_tile_t<FORM, EPI, DN_ACT_NONE>(P, tile, st);
    }
}

}  // namespace moe
