// Shared by the FFN sub-layer's operators (block norm, 8-bit product,
// products grouped by expert): element access, row reductions, host checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "ffn_rules.h"
#include "gemm_rs.h"
#include "join_slots.h"

namespace gemm_rs {
namespace ffn {

// The result of a HIP call.  An error is returned and not left behind as the
// thread's last one, which a later call, also of another library, would report
// as its own.
inline hipError_t own(hipError_t e) {
    if (e != hipSuccess) (void)hipGetLastError();
    return e;
}

// work is only enqueued while the plan's device is current
inline bool on_device(int device) {
    int cur = -1;
    return own(hipGetDevice(&cur)) == hipSuccess && cur == device;
}

inline bool aligned(const void *p, size_t bytes) { return ((uintptr_t)p % bytes) == 0; }

inline bool known_type(int32_t t) { return t == GEMM_RS_BF16 || t == GEMM_RS_F32; }
inline size_t type_bytes(int32_t t) { return t == GEMM_RS_F32 ? 4 : 2; }

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// round to nearest even (NaN stays NaN)
__device__ __forceinline__ uint32_t to_bf16(float x) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return to_bf16(a) | (to_bf16(b) << 16);
}

// 8 elements as they lie in memory, kept raw until used, so that a row read
// ahead costs the registers of its storage type only.
template <bool F32> struct Raw;
template <> struct Raw<true> { u32x4_t a, b; };
template <> struct Raw<false> { u32x4_t a; };

// Row `row` of a matrix of `elem`-byte elements: a wave-uniform address, which
// a 32-bit column number per lane is added to.
__device__ __forceinline__ const void *row_of(const void *p, int64_t row, int64_t ld, int elem) {
    return (const char *)p + row * ld * elem;
}
__device__ __forceinline__ void *row_of(void *p, int64_t row, int64_t ld, int elem) {
    return (char *)p + row * ld * elem;
}

// Columns c..c+7 of a row of `cols` (c < cols).  WIDE: the row starts on 16
// bytes and cols is a multiple of 8.  Otherwise rows start on any element: the
// same 16-byte accesses, which the hardware takes at any address; a row's last
// few columns come as the last 8 of the row (or one by one in a row of fewer),
// which settle8 then shifts into place, zeros behind them.  It is a step of its
// own so that all loads can go out before the first is waited for.
typedef u32x4_t u32x4_at4_t __attribute__((aligned(4)));
typedef u32x4_t u32x4_at2_t __attribute__((aligned(2)));
typedef u32x2_t u32x2_at1_t __attribute__((aligned(1)));

template <bool F32, bool WIDE>
__device__ __forceinline__ void fetch8(Raw<F32> &r, const void *row, uint32_t c, uint32_t cols) {
    if (WIDE || cols >= 8) {
        const uint32_t at = WIDE || c + 8 <= cols ? c : cols - 8;
        if constexpr (F32) {
            typedef std::conditional_t<WIDE, u32x4_t, u32x4_at4_t> words;
            const words *q = (const words *)((const float *)row + at);
            r.a = q[0];
            r.b = q[1];
        } else {
            typedef std::conditional_t<WIDE, u32x4_t, u32x4_at2_t> words;
            r.a = *(const words *)((const uint16_t *)row + at);
        }
    } else {
        r = Raw<F32>{};
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (c + e < cols) {
                if constexpr (F32) {
                    const uint32_t w = ((const uint32_t *)row)[c + e];
                    if (e < 4) r.a[e] = w;
                    else r.b[e - 4] = w;
                } else {
                    r.a[e >> 1] |= (uint32_t)((const uint16_t *)row)[c + e] << (16 * (e & 1));
                }
            }
    }
}
template <bool F32, bool WIDE>
__device__ __forceinline__ void settle8(Raw<F32> &r, uint32_t c, uint32_t cols) {
    if (WIDE || c + 8 <= cols || c >= cols || cols < 8) return;
    const uint32_t by = c + 8 - cols;      // 1..7 elements
    constexpr int N = F32 ? 8 : 4;
    uint32_t w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (F32) w[i] = i < 4 ? r.a[i] : r.b[i - 4];
        else w[i] = r.a[i];
    }
#pragma unroll
    for (int step = 4; step >= 1; step >>= 1) {
        if (!(by & step)) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (F32) w[i] = i + step < N ? w[i + step] : 0u;
            else if (step > 1) w[i] = i + step / 2 < N ? w[i + step / 2] : 0u;
            else w[i] = (w[i] >> 16) | (i + 1 < N ? w[i + 1] << 16 : 0u);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (F32) {
            if (i < 4) r.a[i] = w[i];
            else r.b[i - 4] = w[i];
        } else {
            r.a[i] = w[i];
        }
    }
}
template <bool F32, bool WIDE>
__device__ __forceinline__ void load8(Raw<F32> &r, const void *row, uint32_t c, uint32_t cols) {
    fetch8<F32, WIDE>(r, row, c, cols);
    settle8<F32, WIDE>(r, c, cols);
}

template <bool F32>
__device__ __forceinline__ float raw_at(const Raw<F32> &r, int e) {
    if constexpr (F32) return __uint_as_float(e < 4 ? r.a[e] : r.b[e - 4]);
    else return (e & 1) ? bf16_hi(r.a[e >> 1]) : bf16_lo(r.a[e >> 1]);
}

// Columns c..c+3 of a row of `cols` floats (c < cols), aligned as above; STREAM:
// past the caches.
template <bool WIDE, bool STREAM = false>
__device__ __forceinline__ void store4(float *row, uint32_t c, uint32_t cols, const float *v) {
    if (WIDE || c + 4 <= cols) {
        typedef std::conditional_t<WIDE, u32x4_t, u32x4_at4_t> words;
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[e]);
        if constexpr (STREAM) __builtin_nontemporal_store(w, (words *)(row + c));
        else *(words *)(row + c) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (c + e < cols) row[c + e] = v[e];
    }
}
// Columns c..c+7, of either type.
template <bool F32, bool WIDE, bool STREAM = false>
__device__ __forceinline__ void store8(void *row, uint32_t c, uint32_t cols, const float *v) {
    if constexpr (F32) {
        store4<WIDE, STREAM>((float *)row, c, cols, v);
        if (WIDE || c + 4 < cols) store4<WIDE, STREAM>((float *)row, c + 4, cols, v + 4);
    } else if (WIDE || c + 8 <= cols) {
        typedef std::conditional_t<WIDE, u32x4_t, u32x4_at2_t> words;
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
        if constexpr (STREAM) __builtin_nontemporal_store(w, (words *)((uint16_t *)row + c));
        else *(words *)((uint16_t *)row + c) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (c + e < cols) ((uint16_t *)row)[c + e] = (uint16_t)to_bf16(v[e]);
    }
}

// A workgroup barrier for LDS hand-offs: waits for this wave's LDS
// operations but not for its global loads and stores.
__device__ __forceinline__ void lds_only_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct Sum {
    static __device__ __forceinline__ float join(float a, float b) { return a + b; }
    static __device__ __forceinline__ float none() { return 0.0f; }
};
// Largest bit pattern of a magnitude: as unsigned integers NaN > inf >
// every finite value, so neither is lost (a float maximum drops NaN).
struct MaxBits {
    static __device__ __forceinline__ float join(float a, float b) {
        const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
        return __uint_as_float(x > y ? x : y);
    }
    static __device__ __forceinline__ float none() { return 0.0f; }
};

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

// One wave's join of a value, in every lane: four steps inside rows of 16
// lanes (quad permutes and mirrors), then the four rows.
template <class OP>
__device__ __forceinline__ float wave_join(float v) {
    v = OP::join(v, dpp<0xb1>(v));    // lanes 1,0,3,2
    v = OP::join(v, dpp<0x4e>(v));    // lanes 2,3,0,1
    v = OP::join(v, dpp<0x141>(v));   // mirror of each 8
    v = OP::join(v, dpp<0x140>(v));   // mirror of each 16
    const int i = __float_as_int(v);
    const float a = __int_as_float(__builtin_amdgcn_readlane(i, 0));
    const float b = __int_as_float(__builtin_amdgcn_readlane(i, 16));
    const float c = __int_as_float(__builtin_amdgcn_readlane(i, 32));
    const float d = __int_as_float(__builtin_amdgcn_readlane(i, 48));
    return OP::join(OP::join(a, b), OP::join(c, d));
}

// Join of NV values over a workgroup, in every thread; the order is fixed.
// `turn` alternates between the halves of `slots`, which all joins of a kernel
// share, so one barrier per call is enough.  A wave that has not finished the
// reads of call n holds the others before the barrier of call n+1; until then
// they write call n+1's half only, which no slot of call n lies in (whatever
// the two NV are), and call n's half again in call n+2, behind that barrier.
template <class OP, int THREADS, int NV, int MOST>
__device__ __forceinline__ void block_join(float (&v)[NV], JoinSlots<MOST> &slots, int &turn) {
    constexpr int NW = THREADS / 64;
    static_assert(NV <= MOST && NW <= JoinSlots<MOST>::kWaves, "a half holds a join");
#pragma unroll
    for (int n = 0; n < NV; ++n) v[n] = wave_join<OP>(v[n]);
    if constexpr (NW > 1) {
        const int now = turn;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < NV; ++n) slots.v[slots.at(now, n, threadIdx.x >> 6)] = v[n];
        lds_only_barrier();
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float t = slots.v[slots.at(now, n, 0)];
#pragma unroll
            for (int w = 1; w < NW; ++w) t = OP::join(t, slots.v[slots.at(now, n, w)]);
            v[n] = t;
        }
    }
}

// A row's scale and the factor that quantises it, from the bits of its
// largest magnitude: q = rint(x * pre * inv), inv = 127 * (1 / max), scale =
// max / 127.  `pre` is 1, or 2^64 for rows so small that inv would overflow.
struct QuantRow {
    float scale, pre, inv;
    bool finite;
};
__device__ __forceinline__ QuantRow quant_row(float amax) {
    QuantRow r;
    r.finite = __float_as_uint(amax) < 0x7f800000u;
    r.pre = amax < 0x1p-100f ? 0x1p64f : 1.0f;
    r.scale = r.finite ? amax / 127.0f : __uint_as_float(0x7fc00000u);
    r.inv = (r.finite && amax > 0.0f) ? 127.0f * (1.0f / (amax * r.pre)) : 0.0f;
    return r;
}
__device__ __forceinline__ int quant_one(const QuantRow &r, float x) {
    if (!r.finite) return 0;
    // |x * inv| <= 127 up to rounding, which rint takes back to 127
    return (int)rintf(x * r.pre * r.inv);
}
// Columns c..c+7 of a row of `cols` bytes, from at(e).
template <bool WIDE, class F>
__device__ __forceinline__ void quant8(const QuantRow &q, int8_t *row, uint32_t c, uint32_t cols, F at) {
    if (WIDE || c + 8 <= cols) {
        typedef std::conditional_t<WIDE, u32x2_t, u32x2_at1_t> words;
        u32x2_t w = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2] |= (uint32_t)(quant_one(q, at(e)) & 0xff) << (8 * (e & 3));
        *(words *)(row + c) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (c + e < cols) row[c + e] = (int8_t)quant_one(q, at(e));
    }
}

// Threads of a launch along one axis.  Workgroups past them are dropped without an
// error from the runtime, so `launch` refuses such grids.
constexpr int64_t kMostThreads = UINT32_MAX;

// Rows of a product with N columns whose workgroups fit one launch, for kernels of at
// most 256 threads to 64 x 64 outputs, with a last tile of up to 256 rows.  (At least
// a tile: a row of 2^28 columns is refused by `launch`.)
inline int64_t rows_of_launch(int64_t N) {
    const int64_t rows = (kMostThreads / 256 / ((N + 63) / 64) * 64 - 256) / 256 * 256;
    return rows < 256 ? 256 : rows;
}

// Launches a kernel.  The result is this launch's: the thread's last error may
// be an older one of the caller's, who may not have asked for it, and stays his.
template <class... P, class... A>
inline hipError_t launch(void (*kernel)(P...), dim3 grid, int threads, int lds_bytes, hipStream_t s, const A &...args) {
    static_assert(sizeof...(P) == sizeof...(A), "an argument for each parameter");
    if ((int64_t)grid.x * threads > kMostThreads) return hipErrorInvalidConfiguration;
    return [&](P... held) {      // the arguments in the parameters' types
        void *at[] = {(void *)&held...};
        return own(hipLaunchKernel((const void *)kernel, grid, dim3((unsigned)threads), at, (size_t)lds_bytes, s));
    }(args...);
}

// The same with dynamic LDS, whose limit is a per-device attribute of the
// kernel: set on the first launch there (threads that race set it twice).
template <auto KERNEL, class ARGS>
inline hipError_t launch_lds(int64_t blocks, int threads, int lds_bytes, hipStream_t s, const ARGS &a) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> set[kMaxDevices];
    int dev = 0;
    const hipError_t got = own(hipGetDevice(&dev));
    if (got != hipSuccess) return got;
    if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_acquire)) {
        const hipError_t e = own(hipFuncSetAttribute((const void *)KERNEL,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds_bytes));
        if (e != hipSuccess) return e;
        set[dev].store(true, std::memory_order_release);
    }
    if (blocks > kMostThreads / threads) return hipErrorInvalidConfiguration;
    return launch(KERNEL, dim3((unsigned)blocks), threads, lds_bytes, s, a);
}

}  // namespace ffn
}  // namespace gemm_rs
