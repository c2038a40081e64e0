// Matrix-pipe pieces shared by the 8-bit product and the products grouped by
// expert.
#pragma once

#include "ffn_internal.h"

namespace gemm_rs {
namespace ffn {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));

// One 32 x 32 block: 16 bytes per lane of each operand (row lane % 32, the
// lane/32-th 16 bytes of the step), 16 deep in bfloat16, 32 deep in int8.
// The operands are swapped, so the block comes out transposed: a lane holds
// output row lane % 32, registers 4q..4q+3 its columns 8q + 4*(lane/32) + 0..3.
__device__ __forceinline__ f32x16_t mma(i32x4_t a, i32x4_t b, f32x16_t acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, b),
                                                   __builtin_bit_cast(bf16x8_t, a), acc, 0, 0, 0);
}
__device__ __forceinline__ i32x16_t mma(i32x4_t a, i32x4_t b, i32x16_t acc) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, acc, 0, 0, 0);
}

}  // namespace ffn
}  // namespace gemm_rs
