// moe_gated.hip -- the gated feed-forward block's own products: gate and up in
// one kernel (C = A B^T over rows of both, activation and product in the
// epilogue), and the backward pass's dh = dy Wd with the gradients through the
// activation and the product in its epilogue.
//
// Measured (MI355X, 8192 rows, 4096 x 11008, SiLU): gate and up 1.2 ms
// (1.23 PFLOP/s; 540 MB of h, gate and up written, 5 us of every tile's 90),
// dh 0.79 ms (0.93 PFLOP/s; 900 MB of gate and up read, their gradients and h
// written: 640 KB per tile after its 64 steps, which no step overlaps).
#include "moe_dense.h"

namespace moe {

hipError_t dense_gated_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_NT, DN_EPI_GATED>(P, tile, st);
}
hipError_t dense_dgated_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_NN, DN_EPI_DGATED>(P, tile, st);
}

}  // namespace moe
