// moe_grad.hip -- the dense backward passes' plain products: the input
// gradient (C = A B) and the weight gradients (C = A^T B), each alone or all in
// one launch.
#include "moe_dense.h"

namespace moe {

hipError_t dense_dx_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_NN, DN_EPI_LINEAR>(P, tile, st);
}
hipError_t dense_dw_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_TN, DN_EPI_LINEAR>(P, tile, st);
}
hipError_t dense_grads_launch(const DenseGradsParams &A, int tile, hipStream_t st) {
    int64_t tiles = 0;
    for (int i = 0; i < A.n; ++i) tiles += A.tiles[i];
    if (A.sum.out) tiles += (A.sum.N + DN_SUM_COLS - 1) / DN_SUM_COLS;
    const dim3 grid((unsigned)tiles);
#define DN_LAUNCH(THREADS, ...) hipLaunchKernelGGL((k_dense_grads<__VA_ARGS__>), grid, dim3(THREADS), 0, st, A)
    DN_TILE_SWITCH(tile, DN_LAUNCH)
#undef DN_LAUNCH
    return hipGetLastError();
}

}  // namespace moe
