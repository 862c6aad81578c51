// moe_gated.hip -- the gated feed-forward block's own products: gate and up in
// one kernel (C = A B^T over rows of both, activation and product in the
// epilogue), and the backward pass's dh = dy Wd with the gradients through the
// activation and the product in its epilogue.
#include "moe_dense.h"

namespace moe {

hipError_t dense_gated_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_NT, DN_EPI_GATED>(P, tile, st);
}
hipError_t dense_dgated_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_NN, DN_EPI_DGATED>(P, tile, st);
}

}  // namespace moe
