// One product of more than a few rows.
#include "dense_tile.h"

namespace gemm_rs {
namespace ffn {

template hipError_t launch_dense<kOne>(DenseArgs &, bool, bool, int64_t, hipStream_t);

}  // namespace ffn
}  // namespace gemm_rs
