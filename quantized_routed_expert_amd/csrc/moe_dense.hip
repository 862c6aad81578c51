// moe_dense.hip -- the C ABI of the dense operators (linear and the gated
// feed-forward block, forward and backward; include/moe.h): host-side
// validation, workspace layout, tile and split choice, launches.  They stand
// next to the routed layer: the dense parts of the same model in bf16 (a
// shared expert kept in 16 bits, dense layers, projections).
#include <hip/hip_runtime.h>
#include <string.h>

#include "../../include/moe.h"
#include "moe_internal.h"

namespace moe {
hipError_t dense_split3_launch(const float *x, uint16_t *out, int64_t n, hipStream_t st);
hipError_t dense_dz_launch(const DzParams &P, hipStream_t st);
hipError_t dense_colsum_launch(const ColsumParams &P, hipStream_t st);
hipError_t dense_linear_launch(const DenseParams &P, int tile, hipStream_t st);
hipError_t dense_gated_launch(const DenseParams &P, int tile, hipStream_t st);
hipError_t dense_dgated_launch(const DenseParams &P, int tile, hipStream_t st);
hipError_t dense_dx_launch(const DenseParams &P, int tile, hipStream_t st);
hipError_t dense_dw_launch(const DenseParams &P, int tile, hipStream_t st);
hipError_t dense_grads_launch(const DenseGradsParams &A, int tile, hipStream_t st);
hipError_t dense_rows_linear_launch(const DenseRowsParams &P, hipStream_t st);
hipError_t dense_rows_gated_launch(const DenseRowsParams &P, hipStream_t st);
}  // namespace moe

using namespace moe;

static_assert(DN_ACT_NONE == MOE_ACT_NONE && DN_ACT_SILU == MOE_ACT_SILU && DN_ACT_GELU == MOE_ACT_GELU &&
                  DN_ACT_GELU_TANH == MOE_ACT_GELU_TANH && DN_ACT_RELU == MOE_ACT_RELU,
              "activation codes");

namespace {

constexpr int DN_MAX_WIDTH = 1 << 20;
constexpr int DN_MAX_ROWS = 1 << 24;
constexpr int DN_SPLIT_TILES = 512;  // tiles of a split product over all its splits
constexpr int DN_DZ_CHUNKS = 64;  // row chunks of the bias gradient

int64_t max64(int64_t a, int64_t b) { return a > b ? a : b; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int check_width(int32_t a, int32_t b) {
    if (a <= 0 || b <= 0) return MOE_ERR_INVALID_ARG;
    if (a % 8 || b % 8 || a > DN_MAX_WIDTH || b > DN_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
int check_rows(int32_t T) {
    if (T < 0) return MOE_ERR_INVALID_ARG;
    return T > DN_MAX_ROWS ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
bool valid_dtype(int d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16; }
bool valid_act(int a) { return a >= MOE_ACT_NONE && a <= MOE_ACT_RELU; }
bool misaligned(const void *p) { return ((uintptr_t)p & 15) != 0; }

// ---- tile and split choice ----
struct Plan {
    int tile, tiles_m, tiles_n, splits, per;
    double us;  // estimated time
};
// The least estimated time over the tiles and split counts.  Rounds of one
// tile per CU; a tile takes a fixed time and one per step (of its longest
// group), the results one per MB, a split the hand-over and the parts'
// traffic.  Fitted to the launches of 63 products (16 x 2048 x 768 to
// 8192 x 4096 x 11008, each tile, splits of 1, 2 and 4) that are within 1.9
// times the best of their product: 8% off in the mean, and the choice costs
// 0.1% over the best.  E.g. 2048 x 2048 outputs over 512 k take 10 us in
// 128 x 128 tiles and 20 in 64 x 64; 2048 x 512 outputs over 2048 k 17 and 10;
// 2048 x 1024 outputs over 2048 k 18, 19 and in 128 x 64 tiles 14.6.
struct TileCost {
    int bm, bn, groups;
    double fixed, step;  // us
};
constexpr TileCost TILES[DN_TILES] = {
    {256, 256, 1, 4.6, 1.21}, {256, 128, 1, 2.9, 0.72}, {128, 128, 2, 3.9, 0.76}, {128, 64, 2, 3.0, 0.53}, {64, 64, 4, 2.7, 0.70}};
constexpr double US_LAUNCH = 1.4, US_JOIN = 2.6, US_PER_MB = 0.18, US_PER_PART_MB = 0.6;
constexpr int CUS = 256;  // (workspace sizes do not depend on the device at hand)

double tile_us(const TileCost &c, int64_t steps) { return c.fixed + c.step * (double)ceil_div(steps, c.groups); }
double out_us(int64_t M, int64_t N) { return (double)M * (double)N * 2e-6 * US_PER_MB; }

// Time until the last of k sections of tiles (n[i] tiles of us[i] each, started
// in order) is done, each CU taking the next tile when it is free.
double tiles_us(const double *us, const int64_t *n, int k) {
    struct {
        double at;
        int64_t cus;
    } q[16] = {{0.0, CUS}};  // CUs by the time they are free at
    int nq = 1;
    for (int i = 0; i < k; ++i) {
        int64_t left = n[i];
        if (left > 4 * CUS) {  // whole rounds at once
            const int64_t rounds = left / CUS - 2;
            for (int j = 0; j < nq; ++j) q[j].at += (double)rounds * us[i];
            left -= rounds * CUS;
        }
        while (left > 0) {
            int a = 0, b = -1;
            for (int j = 1; j < nq; ++j)
                if (q[j].at < q[a].at) a = j;
            const int64_t take = q[a].cus < left ? q[a].cus : left;
            const double done = q[a].at + us[i];
            left -= take;
            q[a].cus -= take;
            for (int j = 0; j < nq; ++j)
                if (j != a && (q[j].at == done || (nq == 16 && b < 0))) b = j;
            if (b >= 0) {
                q[b].cus += take;
                q[b].at = q[b].at > done ? q[b].at : done;
                if (q[a].cus == 0) q[a] = q[--nq];
            } else if (q[a].cus == 0) {
                q[a].at = done;
                q[a].cus = take;
            } else {
                q[nq].at = done;
                q[nq++].cus = take;
            }
        }
    }
    double last = 0.0;
    for (int j = 0; j < nq; ++j) last = q[j].at > last ? q[j].at : last;
    return last;
}

// C of M x N columns of the weight side (gated: 2F) over `steps` 64-k steps
Plan make_plan(int64_t M, int64_t N, int64_t steps) {
    Plan best = {-1, 0, 0, 1, 1, 1e30};
    steps = max64(steps, 1);
    for (int t = 0; t < DN_TILES; ++t) {
        const TileCost &c = TILES[t];
        const int64_t tm = ceil_div(M, c.bm), tn = ceil_div(N, c.bn), tiles = max64(tm * tn, 1);  // (M = 0: nothing is launched)
        for (int64_t s = 1; s <= 16; s *= 2) {
            if (s > 1 && (tiles * s * c.bm * c.bn > (int64_t)DN_SPLIT_TILES * 128 * 128 || tiles > WS_COUNTERS ||
                          steps < 2 * s * c.groups))
                break;
            const int64_t per = ceil_div(steps, s);
            double us = US_LAUNCH + (double)ceil_div(tiles * s, CUS) * tile_us(c, per) + out_us(M, N);
            if (s > 1) us += US_JOIN + (double)(s * tiles * c.bm * c.bn) * 4e-6 * US_PER_PART_MB;
            if (us < best.us) best = Plan{t, (int)tm, (int)tn, (int)ceil_div(steps, per), (int)per, us};
        }
    }
    return best;
}

// The few-row kernel against tiles: a workgroup reads its weight rows and its
// activation rows (from L2), together 35 KB a microsecond; all weights at most
// 5.1 TB/s.  (T, K, N = 16, 2048, 2048: 5.2 us and 8.4 with tiles; 16, 2048,
// 11264: 13.8 and 11.2; 64, 2048, 2048: 7.9 and 8.8; 37, 1000, 520: 3.3 and
// 6.4, with fp32 activations 4.5 and 16.9; 256, 512, 512: 3.7 and 5.7.)
double rows_us(int64_t T, int64_t K, int64_t rows, bool x_f32) {
    const DenseRowsShape s = dense_rows_shape(T, rows);
    const int64_t wr = s.halves ? 8 : 16, wgs = s.wgs * s.blocks;
    const int64_t xr = T == 1 ? 1 : s.mt * wr;  // (one row: every lane's load is the same)
    const double bytes = (double)K * (double)(2 * wr + (x_f32 ? 5 : 2) * xr);
    const double rounds = wgs > CUS ? (double)wgs / CUS : 1.0;
    const double us = rounds * bytes / 35e3, hbm = (double)K * (double)rows * 2.0 / 5.1e6;
    return 2.3 + (us > hbm ? us : hbm);
}
bool few_rows(int64_t T, int64_t K, int64_t rows, bool x_f32, const Plan &tiles) {
    if (T > DN_ROWS_MAX) return false;
    return rows_us(T, K, rows, x_f32) < tiles.us + (x_f32 ? 2.7 : 0.0);  // (tiles: fp32 is split by a launch of its own)
}

int64_t ksteps(int64_t K) { return ceil_div(K, DN_BK); }

struct Carve {  // workspace regions after the head
    int64_t off = (int64_t)align_up(COUNTER_WORDS * 4, 256);
    int64_t take(int64_t bytes) {
        const int64_t a = off;
        off += (int64_t)align_up((size_t)bytes, 256);
        return a;
    }
};
uint8_t *at(void *ws, int64_t off) { return (uint8_t *)ws + off; }

void set_plan(DenseParams &P, const Plan &p, int M, int N, int steps, void *ws, int64_t part) {
    P.M = M;
    P.N = N;
    P.steps = steps;
    P.tiles_m = p.tiles_m;
    P.tiles_n = p.tiles_n;
    P.splits = p.splits;
    P.steps_per_split = p.per;
    P.part = (float *)at(ws, part);
    P.counters = (uint32_t *)ws;
}
// The parts of a split product: at most DN_SPLIT_TILES tiles of 128 x 128
// over all splits, whatever the sizes; a fixed region, so that a workspace
// sized for T rows also serves fewer.
constexpr int64_t DN_PART_BYTES = (int64_t)DN_SPLIT_TILES * 128 * 128 * 4;

// ---- workspace layouts ----
struct LinearWs {
    int64_t x3, part, total;         // forward
    int64_t dz, chunks, bpart, btotal;  // backward
    Plan fwd, dx, dw;
};
LinearWs linear_ws(int64_t T, int64_t K, int64_t N, bool x_f32) {
    LinearWs w;
    w.fwd = make_plan(T, N, ksteps(K) * (x_f32 ? 3 : 1));
    w.dx = make_plan(T, K, ksteps(N));
    w.dw = make_plan(N, K, ksteps(T));
    Carve c;
    w.x3 = c.take(x_f32 ? T * K * 6 : 0);
    w.part = c.take(DN_PART_BYTES);
    w.total = c.off;
    Carve b;
    w.dz = b.take(T * N * 2);
    w.chunks = b.take((int64_t)DN_DZ_CHUNKS * N * 4);
    w.bpart = b.take(DN_PART_BYTES);
    w.btotal = b.off;
    return w;
}
struct GatedWs {
    int64_t x3, h, part, total;
    int64_t dgu, bh, bpart, btotal;
    Plan gu, down, dh, dx, dw, dd;
};
GatedWs gated_ws(int64_t T, int64_t H, int64_t F, bool x_f32, bool y_f32) {
    GatedWs w;
    w.gu = make_plan(T, 2 * F, ksteps(H) * (x_f32 ? 3 : 1));
    w.down = make_plan(T, H, ksteps(F) * (y_f32 ? 3 : 1));
    w.dh = make_plan(T, F, ksteps(H));
    w.dx = make_plan(T, H, 2 * ksteps(F));
    w.dw = make_plan(F, H, ksteps(T));
    w.dd = make_plan(H, F, ksteps(T));
    Carve c;
    w.x3 = c.take(x_f32 ? T * H * 6 : 0);
    w.h = c.take(T * F * 2 * (y_f32 ? 3 : 1));
    w.part = c.take(DN_PART_BYTES);
    w.total = c.off;
    Carve b;
    w.dgu = b.take(T * F * 4);
    w.bh = b.take(T * F * 2);
    w.bpart = b.take(DN_PART_BYTES);
    w.btotal = b.off;
    return w;
}

inline hipStream_t S(int64_t s) { return (hipStream_t)(intptr_t)s; }
int launch_err(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

// A backward pass's last products (p[0] dx where with_dx, the rest weight
// gradients), each with the plan of a launch of its own, and the bias
// gradient's sums (sum.out): one launch of all where its estimate is lower.
int launch_grads(DenseParams *p, const Plan *plans, int n, bool with_dx, const ColsumParams &sum, hipStream_t st) {
    int order[DN_MAX_GRADS];
    double apart = 0.0;
    for (int i = 0; i < n; ++i) {  // longest tiles first
        int j = i;
        for (; j > 0 && p[i].steps > p[order[j - 1]].steps; --j) order[j] = order[j - 1];
        order[j] = i;
        apart += plans[i].us;
    }
    int best = -1;
    double best_us = 1e30;
    for (int t = 0; t < DN_TILES; ++t) {
        const TileCost &c = TILES[t];
        double us[DN_MAX_GRADS], out = 0.0;
        int64_t tiles[DN_MAX_GRADS];
        for (int i = 0; i < n; ++i) {
            const DenseParams &q = p[order[i]];
            // (tiles of 64 columns read most per product: with all CUs at work the
            // caches hold them up; 777 x 1032 x 2048: 23 us, in 128 x 128 tiles 19.5)
            us[i] = tile_us(c, q.steps) * (c.bn == 64 ? 1.25 : 1.0);
            tiles[i] = ceil_div(q.M, c.bm) * ceil_div(q.N, c.bn);
            out += out_us(q.M, q.N);
        }
        const double all_us = US_LAUNCH + out + tiles_us(us, tiles, n);
        if (all_us < best_us) {
            best_us = all_us;
            best = t;
        }
    }
    // (together, large products share the caches less: 2048 rows x 2048 x 4096
    // and smaller gain 5 to 35%, 8192 x 4096 x 11008 loses 3%)
    if (n < 2 || apart <= 1.06 * best_us) {
        if (sum.out && dense_colsum_launch(sum, st) != hipSuccess) return MOE_ERR_LAUNCH;
        for (int i = 0; i < n; ++i) {
            const hipError_t e = i == 0 && with_dx ? dense_dx_launch(p[i], plans[i].tile, st) : dense_dw_launch(p[i], plans[i].tile, st);
            if (e != hipSuccess) return MOE_ERR_LAUNCH;
        }
        return MOE_OK;
    }
    DenseGradsParams A;
    memset(&A, 0, sizeof(A));
    A.n = n;
    A.dx_at = -1;
    A.sum = sum;
    const TileCost &c = TILES[best];
    for (int i = 0; i < n; ++i) {
        DenseParams &q = A.p[i];
        q = p[order[i]];
        q.tiles_m = (int)ceil_div(q.M, c.bm);
        q.tiles_n = (int)ceil_div(q.N, c.bn);
        q.splits = 1;
        q.steps_per_split = q.steps > 0 ? q.steps : 1;
        A.tiles[i] = q.tiles_m * q.tiles_n;
        if (with_dx && order[i] == 0) A.dx_at = i;
    }
    return launch_err(dense_grads_launch(A, best, st));
}

// A weight gradient A^T B over T rows, into y or onto it
DenseParams grad_params(const DenseSeg &g, const Plan &plan, int M, int N, int T, void *y, int32_t dtype, int32_t accumulate,
                        void *ws, int64_t part) {
    DenseParams P;
    memset(&P, 0, sizeof(P));
    P.nseg = 1;
    P.seg[0] = g;
    set_plan(P, plan, M, N, (int)ksteps(T), ws, part);
    P.e.y = y;
    P.e.y_f32 = P.e.res_f32 = dtype == MOE_DTYPE_F32;
    P.e.res = accumulate ? y : nullptr;
    return P;
}

// x's products with rows of K: one (bf16) or three (fp32, its exact bf16
// terms, written to x3 first)
int x_segments(DenseParams &P, const void *x, bool x_f32, int64_t T, int64_t K, uint16_t *x3, hipStream_t st) {
    if (x_f32 && dense_split3_launch((const float *)x, x3, T * K, st) != hipSuccess) return MOE_ERR_LAUNCH;
    P.nseg = x_f32 ? 3 : 1;
    for (int i = 0; i < P.nseg; ++i) {
        P.seg[i].a = x_f32 ? x3 + (int64_t)i * T * K : (const uint16_t *)x;
        P.seg[i].lda = K;
        P.seg[i].K = (int)K;
    }
    return MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_linear_workspace_bytes(int32_t T, int32_t in, int32_t out) {
    int rc = check_rows(T);
    if (rc) return rc;
    if ((rc = check_width(in, out))) return rc;
    const LinearWs a = linear_ws(T, in, out, false), b = linear_ws(T, in, out, true);
    return max64(max64(a.total, b.total), a.btotal);
}

int moe_linear(const void *x, int32_t x_dtype, int32_t T, int32_t in, const void *w, int32_t out, const void *bias,
               int32_t act, const void *residual, int32_t r_dtype, void *z, void *y, int32_t y_dtype, void *ws,
               int64_t ws_bytes, int64_t stream) {
    if (T != 0 && (!x || !w || !y || !ws)) return MOE_ERR_INVALID_ARG;
    if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype) || !valid_act(act)) return MOE_ERR_INVALID_ARG;
    if (residual && !valid_dtype(r_dtype)) return MOE_ERR_INVALID_ARG;
    if (misaligned(x) || misaligned(w) || misaligned(bias) || misaligned(residual) || misaligned(z) || misaligned(y) ||
        misaligned(ws))
        return MOE_ERR_INVALID_ARG;
    int rc = check_rows(T);
    if (rc) return rc;
    if ((rc = check_width(in, out))) return rc;
    if (T == 0) return MOE_OK;
    const bool xf = x_dtype == MOE_DTYPE_F32;
    const LinearWs L = linear_ws(T, in, out, xf);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    int cus;
    if ((rc = device_cus(cus))) return rc;
    DenseEpi e;
    memset(&e, 0, sizeof(e));
    e.bias = (const uint16_t *)bias;
    e.res = residual;
    e.res_f32 = r_dtype == MOE_DTYPE_F32;
    e.y = y;
    e.y_f32 = y_dtype == MOE_DTYPE_F32;
    e.z = (uint16_t *)z;
    e.act = act;
    if (few_rows(T, in, out, xf, L.fwd)) {
        const DenseRowsParams R{x, (const uint16_t *)w, nullptr, e, T, out, in, xf};
        return launch_err(dense_rows_linear_launch(R, S(stream)));
    }
    DenseParams P;
    memset(&P, 0, sizeof(P));
    if ((rc = x_segments(P, x, xf, T, in, (uint16_t *)at(ws, L.x3), S(stream)))) return rc;
    for (int i = 0; i < P.nseg; ++i) {
        P.seg[i].b = (const uint16_t *)w;
        P.seg[i].ldb = in;
    }
    set_plan(P, L.fwd, T, out, (int)(ksteps(in) * P.nseg), ws, L.part);
    P.e = e;
    return launch_err(dense_linear_launch(P, L.fwd.tile, S(stream)));
}

int moe_linear_backward(const void *dy, int32_t T, int32_t in, int32_t out, const void *x, const void *w, const void *z,
                        int32_t act, void *dx, void *dw, void *dbias, int32_t dw_dtype, int32_t accumulate, void *ws,
                        int64_t ws_bytes, int64_t stream) {
    if (!dx && !dw && !dbias) return MOE_ERR_INVALID_ARG;
    if (T != 0 && (!dy || (dx && !w) || (dw && !x))) return MOE_ERR_INVALID_ARG;
    if (!valid_act(act) || !valid_dtype(dw_dtype) || !ws) return MOE_ERR_INVALID_ARG;
    if (T != 0 && act != MOE_ACT_NONE && !z) return MOE_ERR_INVALID_ARG;
    if (misaligned(dy) || misaligned(x) || misaligned(w) || misaligned(z) || misaligned(dx) || misaligned(dw) ||
        misaligned(dbias) || misaligned(ws))
        return MOE_ERR_INVALID_ARG;
    int rc = check_rows(T);
    if (rc) return rc;
    if ((rc = check_width(in, out))) return rc;
    const LinearWs L = linear_ws(T, in, out, false);
    if (ws_bytes < L.btotal) return MOE_ERR_WORKSPACE;
    int cus;
    if ((rc = device_cus(cus))) return rc;
    const hipStream_t st = S(stream);
    const bool with_act = act != MOE_ACT_NONE;
    const uint16_t *dz = with_act ? (const uint16_t *)at(ws, L.dz) : (const uint16_t *)dy;
    int nchunks = 0;
    if (T != 0 && (with_act || dbias)) {
        DzParams D;
        memset(&D, 0, sizeof(D));
        D.dy = (const uint16_t *)dy;
        D.z = with_act ? (const uint16_t *)z : nullptr;
        D.dz = with_act && (dx || dw) ? (uint16_t *)at(ws, L.dz) : nullptr;
        D.part = dbias ? (float *)at(ws, L.chunks) : nullptr;
        D.T = T;
        D.N = out;
        D.act = act;
        // chunks of at least 32 rows, at most DN_DZ_CHUNKS of them
        D.rows_per_chunk = max64(ceil_div(T, DN_DZ_CHUNKS), 32);
        nchunks = D.nchunks = (int)ceil_div(T, D.rows_per_chunk);
        if (dense_dz_launch(D, st) != hipSuccess) return MOE_ERR_LAUNCH;
    }
    const ColsumParams sum{(const float *)at(ws, L.chunks), dbias, out, nchunks, dw_dtype == MOE_DTYPE_F32, accumulate != 0};
    DenseParams P[2];
    Plan plans[2];
    int n = 0;
    const bool with_dx = dx && T != 0;
    if (with_dx) {
        DenseParams &X = P[n];
        memset(&X, 0, sizeof(X));
        X.nseg = 1;
        X.seg[0] = DenseSeg{dz, (const uint16_t *)w, nullptr, out, in, out};
        set_plan(X, L.dx, T, in, (int)ksteps(out), ws, L.bpart);
        X.e.y = dx;
        plans[n++] = L.dx;
    }
    if (dw) {
        P[n] = grad_params(DenseSeg{dz, (const uint16_t *)x, nullptr, out, in, T}, L.dw, out, in, T, dw, dw_dtype, accumulate, ws,
                           L.bpart);
        plans[n++] = L.dw;
    }
    return launch_grads(P, plans, n, with_dx, sum, st);
}

int64_t moe_gated_ffn_workspace_bytes(int32_t T, int32_t hidden, int32_t ffn) {
    int rc = check_rows(T);
    if (rc) return rc;
    if ((rc = check_width(hidden, ffn))) return rc;
    int64_t n = gated_ws(T, hidden, ffn, false, false).btotal;
    for (int i = 0; i < 4; ++i) n = max64(n, gated_ws(T, hidden, ffn, i & 1, i >> 1).total);
    return n;
}

int moe_gated_ffn(const void *x, int32_t x_dtype, int32_t T, const moe_dense_ffn *w, const void *residual, int32_t r_dtype,
                  void *gu, void *y, int32_t y_dtype, void *ws, int64_t ws_bytes, int64_t stream) {
    if (!w) return MOE_ERR_INVALID_ARG;
    if (T != 0 && (!x || !y || !ws || !w->gate || !w->up || !w->down)) return MOE_ERR_INVALID_ARG;
    if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype) || !valid_act(w->act)) return MOE_ERR_INVALID_ARG;
    if (residual && !valid_dtype(r_dtype)) return MOE_ERR_INVALID_ARG;
    if (misaligned(x) || misaligned(w->gate) || misaligned(w->up) || misaligned(w->down) || misaligned(residual) ||
        misaligned(gu) || misaligned(y) || misaligned(ws))
        return MOE_ERR_INVALID_ARG;
    int rc = check_rows(T);
    if (rc) return rc;
    const int H = w->hidden, F = w->ffn;
    if ((rc = check_width(H, F))) return rc;
    if (T == 0) return MOE_OK;
    const bool xf = x_dtype == MOE_DTYPE_F32, yf = y_dtype == MOE_DTYPE_F32;
    const GatedWs L = gated_ws(T, H, F, xf, yf);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    int cus;
    if ((rc = device_cus(cus))) return rc;
    const hipStream_t st = S(stream);
    uint16_t *h = (uint16_t *)at(ws, L.h);
    DenseEpi eg, ed;  // gate and up; down
    memset(&eg, 0, sizeof(eg));
    memset(&ed, 0, sizeof(ed));
    eg.act = w->act;
    eg.h = h;
    eg.h_terms = yf ? 3 : 1;
    eg.gu = (uint16_t *)gu;
    ed.res = residual;
    ed.res_f32 = r_dtype == MOE_DTYPE_F32;
    ed.y = y;
    ed.y_f32 = yf;
    // h between the two: fp32 (split where it is read) for the few-row down
    // product, otherwise its bf16 terms
    const bool down_rows = few_rows(T, F, H, yf, L.down);
    if (yf && down_rows) eg.h_terms = 0;
    if (few_rows(T, H, 2 * (int64_t)F, xf, L.gu)) {
        const DenseRowsParams G{x, (const uint16_t *)w->gate, (const uint16_t *)w->up, eg, T, F, H, xf};
        if (dense_rows_gated_launch(G, st) != hipSuccess) return MOE_ERR_LAUNCH;
    } else {
        DenseParams P;
        memset(&P, 0, sizeof(P));
        if ((rc = x_segments(P, x, xf, T, H, (uint16_t *)at(ws, L.x3), st))) return rc;
        for (int i = 0; i < P.nseg; ++i) {
            P.seg[i].b = (const uint16_t *)w->gate;
            P.seg[i].b2 = (const uint16_t *)w->up;
            P.seg[i].ldb = H;
        }
        set_plan(P, L.gu, T, F, (int)(ksteps(H) * P.nseg), ws, L.part);
        P.e = eg;
        if (dense_gated_launch(P, L.gu.tile, st) != hipSuccess) return MOE_ERR_LAUNCH;
    }
    if (down_rows) {
        const DenseRowsParams D{h, (const uint16_t *)w->down, nullptr, ed, T, H, F, yf};
        return launch_err(dense_rows_linear_launch(D, st));
    }
    DenseParams D;
    memset(&D, 0, sizeof(D));
    D.nseg = yf ? 3 : 1;
    for (int i = 0; i < D.nseg; ++i)
        D.seg[i] = DenseSeg{h + (int64_t)i * T * F, (const uint16_t *)w->down, nullptr, F, F, F};
    set_plan(D, L.down, T, H, (int)(ksteps(F) * D.nseg), ws, L.part);
    D.e = ed;
    return launch_err(dense_linear_launch(D, L.down.tile, st));
}

int moe_gated_ffn_backward(const void *dy, const void *x, int32_t T, const moe_dense_ffn *w, const void *gu, void *dx,
                           void *dgate, void *dup, void *ddown, int32_t dw_dtype, int32_t accumulate, void *ws,
                           int64_t ws_bytes, int64_t stream) {
    if (!w || !ws) return MOE_ERR_INVALID_ARG;
    if (!dx && !dgate && !dup && !ddown) return MOE_ERR_INVALID_ARG;
    if (T != 0 && (!dy || !gu || !w->down || ((dgate || dup) && !x) || (dx && (!w->gate || !w->up))))
        return MOE_ERR_INVALID_ARG;
    if (!valid_dtype(dw_dtype) || !valid_act(w->act)) return MOE_ERR_INVALID_ARG;
    if (misaligned(dy) || misaligned(x) || misaligned(w->gate) || misaligned(w->up) || misaligned(w->down) ||
        misaligned(gu) || misaligned(dx) || misaligned(dgate) || misaligned(dup) || misaligned(ddown) || misaligned(ws))
        return MOE_ERR_INVALID_ARG;
    int rc = check_rows(T);
    if (rc) return rc;
    const int H = w->hidden, F = w->ffn;
    if ((rc = check_width(H, F))) return rc;
    const GatedWs L = gated_ws(T, H, F, false, false);
    if (ws_bytes < L.btotal) return MOE_ERR_WORKSPACE;
    int cus;
    if ((rc = device_cus(cus))) return rc;
    const hipStream_t st = S(stream);
    uint16_t *dgu = (uint16_t *)at(ws, L.dgu), *h = (uint16_t *)at(ws, L.bh);
    if (T != 0) {  // dh = dy Wd, then dg, du and h
        DenseParams P;
        memset(&P, 0, sizeof(P));
        P.nseg = 1;
        P.seg[0] = DenseSeg{(const uint16_t *)dy, (const uint16_t *)w->down, nullptr, H, F, H};
        set_plan(P, L.dh, T, F, (int)ksteps(H), ws, L.bpart);
        P.e.act = w->act;
        P.e.gu_in = (const uint16_t *)gu;
        P.e.dgu = dgu;
        P.e.h = ddown ? h : nullptr;
        if (dense_dgated_launch(P, L.dh.tile, st) != hipSuccess) return MOE_ERR_LAUNCH;
    }
    DenseParams P[DN_MAX_GRADS];
    Plan plans[DN_MAX_GRADS];
    int n = 0;
    const bool with_dx = dx && T != 0;
    if (with_dx) {  // dx = dg Wg + du Wu
        DenseParams &X = P[n];
        memset(&X, 0, sizeof(X));
        X.nseg = 2;
        X.seg[0] = DenseSeg{dgu, (const uint16_t *)w->gate, nullptr, 2 * (int64_t)F, H, F};
        X.seg[1] = DenseSeg{dgu + F, (const uint16_t *)w->up, nullptr, 2 * (int64_t)F, H, F};
        set_plan(X, L.dx, T, H, (int)(2 * ksteps(F)), ws, L.bpart);
        X.e.y = dx;
        plans[n++] = L.dx;
    }
    auto grad = [&](const uint16_t *a, int64_t lda, const void *b, int M, int N, const Plan &plan, void *y) {
        if (!y) return;
        P[n] = grad_params(DenseSeg{a, (const uint16_t *)b, nullptr, lda, N, T}, plan, M, N, T, y, dw_dtype, accumulate, ws, L.bpart);
        plans[n++] = plan;
    };
    grad(dgu, 2 * (int64_t)F, x, F, H, L.dw, dgate);
    grad(dgu + F, 2 * (int64_t)F, x, F, H, L.dw, dup);
    grad((const uint16_t *)dy, H, h, H, F, L.dd, ddown);
    ColsumParams none;
    memset(&none, 0, sizeof(none));
    return launch_grads(P, plans, n, with_dx, none, st);
}

}  // extern "C"
