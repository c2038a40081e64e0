// Pairs of products with the same rows: gated projections.
#include "dense_tile.h"

namespace gemm_rs {
namespace ffn {

template hipError_t launch_dense<kPair>(DenseArgs &, bool, bool, int64_t, hipStream_t);

}  // namespace ffn
}  // namespace gemm_rs
