// moe_grad.hip -- the dense backward passes' plain products: the input
// gradient (C = A B) and the weight gradients (C = A^T B).
#include "moe_dense.h"

namespace moe {

hipError_t dense_dx_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_NN, DN_EPI_LINEAR>(P, tile, st);
}
hipError_t dense_dw_launch(const DenseParams &P, int tile, hipStream_t st) {
    return dense_launch_t<DN_TN, DN_EPI_GRAD>(P, tile, st);
}

}  // namespace moe
