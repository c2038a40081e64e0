// Sums of two products: the gradient of the input of gated projections.
#include "dense_tile.h"

namespace gemm_rs {
namespace ffn {

template hipError_t launch_dense<kParts>(DenseArgs &, bool, bool, int64_t, hipStream_t);

}  // namespace ffn
}  // namespace gemm_rs
