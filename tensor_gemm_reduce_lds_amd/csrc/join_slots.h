// Where the waves of a workgroup leave their parts of a join's values in shared
// memory.  Plain C++: the kernels and a host check use the same function.
#pragma once

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define JOIN_SLOTS_FN __host__ __device__ __forceinline__
#else
#define JOIN_SLOTS_FN inline
#endif

namespace gemm_rs {
namespace ffn {

// Slots of a kernel whose joins have at most MOST values each.  Consecutive
// joins take turns between two halves, and a half's place depends on MOST only,
// not on how many values a join has: two consecutive joins never share a slot,
// also where they differ in number.
template <int MOST>
struct JoinSlots {
    static constexpr int kWaves = 16;     // most waves of a workgroup
    static constexpr int kFloats = 2 * MOST * kWaves;
    float v[kFloats];

    // Wave `wave`'s part of value n of a join that has turn `turn`.
    static constexpr JOIN_SLOTS_FN int at(int turn, int n, int wave) {
        return ((turn & 1) * MOST + n) * kWaves + wave;
    }
};

}  // namespace ffn
}  // namespace gemm_rs

#undef JOIN_SLOTS_FN
