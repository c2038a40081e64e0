// Norms before and after a block with gate and residual scale (block_norm.h).
//
// Bound by memory (by latency for few rows).  Forward: one workgroup per row
// at a time, the whole row in registers: one read of x and y, one write of x'
// and u.  Two joins over the workgroup (the mean square of y, then of x', which
// needs the first), a third for the largest |u| when u is quantised.
// 8000 x 8192, f32 stream: 147 us, 5.4 TB/s; 8192 x 8192 bf16: 98 us, 5.5 TB/s (on
// the same card a copy runs at 4.9 TB/s, two reads and a write at 5.9, writes
// alone at 6.9).
//
// Backward: a workgroup walks a run of consecutive rows (loading one row while
// it works on the one before, where that helps) and keeps the sums for dw_post,
// dw_pre and dgate of its columns in registers; two joins per row (mean squares
// of x' and y and the product a.x' together, then b.y).  The partial sums go to
// the workspace once per workgroup and a second kernel adds them in a fixed
// order (6 to 7 us).
// 8192 x 8192 bf16: 168 us with the joining kernel, 4.8 TB/s; 1000 x 4096, f32
// stream: 25 us (few rows per workgroup, and the partial sums are a third of the
// traffic).
//
// Times in this file are of whole calls in a stream, several sets of inputs in
// turn that together exceed the caches, unless they say otherwise.
#include <math.h>
#include <stdlib.h>

#include "block_norm.h"
#include "ffn_internal.h"

using namespace gemm_rs::ffn;

namespace {

constexpr int64_t kMaxCols = 16384;

struct NormArgs {
    int64_t rows, cols, rows_per_gate;
    int64_t ld_x, ld_y, ld_x_out, ld_u, ld_dx_out, ld_du, ld_dx, ld_dy;
    float res_scale, weight_offset, eps_post, eps_pre;
    int32_t has_y, post, pre, gated, param_f32;
    const void *x, *y, *w_post, *gate, *w_pre;
    void *x_out, *u;
    float *u_scale;
    int64_t q_cols;       // columns of int8 rows that are written: zeros past cols
    const void *dx_out, *du;
    void *dx, *dy;
    float *dgate;
    // backward: rows_per_wg consecutive rows per workgroup; its partial sums
    // at part[wg][0 dw_post, 1 dw_pre, 2 gate head, 3 gate tail][cols]
    int64_t rows_per_wg;
    float *part;
};

// This thread's columns of up to three rows of parameters (null: left as they
// are), in[i] + add[i] to out[i]; all loads before the first use of one.
template <bool WIDE, int EPT, int THREADS, int N, bool F32>
__device__ __forceinline__ void load_params_of(uint32_t cols, const void *const (&in)[N], const float (&add)[N],
                                               float (*const (&out)[N])[EPT]) {
    Raw<F32> r[N][EPT / 8];
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (in[i])
#pragma unroll
            for (int k = 0; k < EPT / 8; ++k) {
                const uint32_t c = (uint32_t)(k * THREADS + threadIdx.x) * 8;
                r[i][k] = Raw<F32>{};
                if (c < cols) fetch8<F32, WIDE>(r[i][k], in[i], c, cols);
            }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (in[i]) {
#pragma unroll
            for (int k = 0; k < EPT / 8; ++k)
                settle8<F32, WIDE>(r[i][k], (uint32_t)(k * THREADS + threadIdx.x) * 8, cols);
#pragma unroll
            for (int j = 0; j < EPT; ++j) (*out[i])[j] = raw_at(r[i][j / 8], j % 8) + add[i];
        }
}
template <bool WIDE, int EPT, int THREADS, int N>
__device__ __forceinline__ void load_params(const NormArgs &a, const void *const (&in)[N], const float (&add)[N],
                                            float (*const (&out)[N])[EPT]) {
    if (a.param_f32) load_params_of<WIDE, EPT, THREADS, N, true>((uint32_t)a.cols, in, add, out);
    else load_params_of<WIDE, EPT, THREADS, N, false>((uint32_t)a.cols, in, add, out);
}

// The gate row of a row, and a row of the gate.
__device__ __forceinline__ int64_t gate_of(const NormArgs &a, int64_t row) {
    return (uint32_t)row / (uint32_t)a.rows_per_gate;
}
__device__ __forceinline__ const void *gate_at(const NormArgs &a, int64_t gate_row) {
    return row_of(a.gate, gate_row, a.cols, a.param_f32 ? 4 : 2);
}

// THREADS threads hold a row of up to THREADS * EPT columns: thread t has
// the 8 columns from (k * THREADS + t) * 8 for k < EPT / 8.
template <bool WIDE, int EPT, int THREADS, bool SF, bool YF, bool QUANT>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(NormArgs a) {
    constexpr int VPT = EPT / 8;
    __shared__ JoinSlots<1> slots;
    int turn = 0;
    const int tid = threadIdx.x;
    const float inv_cols = 1.0f / (float)a.cols;
    const uint32_t cols = (uint32_t)a.cols;

    float w_post[EPT], w_pre[EPT], gate[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) w_post[i] = w_pre[i] = gate[i] = 1.0f;
    load_params<WIDE, EPT, THREADS, 2>(a, {a.w_post, a.w_pre}, {a.weight_offset, a.weight_offset}, {&w_post, &w_pre});
    int64_t gate_end = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        Raw<SF> xr[VPT];
        Raw<YF> yr[VPT];
        float x[EPT], y[EPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
            xr[k] = Raw<SF>{};
            yr[k] = Raw<YF>{};
            if (c < cols) {
                fetch8<SF, WIDE>(xr[k], row_of(a.x, row, a.ld_x, SF ? 4 : 2), c, cols);
                if (a.has_y) fetch8<YF, WIDE>(yr[k], row_of(a.y, row, a.ld_y, YF ? 4 : 2), c, cols);
            }
        }
        if (a.gated && row >= gate_end) {
            const int64_t g = gate_of(a, row);
            gate_end = (g + 1) * a.rows_per_gate;
            load_params<WIDE, EPT, THREADS, 1>(a, {gate_at(a, g)}, {0.0f}, {&gate});
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
            settle8<SF, WIDE>(xr[k], c, cols);
            settle8<YF, WIDE>(yr[k], c, cols);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[k * 8 + e] = raw_at(xr[k], e);
                y[k * 8 + e] = raw_at(yr[k], e);
            }
        }
        if (a.has_y) {
            float r2 = 1.0f;
            if (a.post) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < EPT; ++i) s[0] += y[i] * y[i];
                block_join<Sum, THREADS, 1>(s, slots, turn);
                r2 = 1.0f / sqrtf(s[0] * inv_cols + a.eps_post);
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = k * 8 + e;
                    x[i] = a.res_scale * x[i] + gate[i] * (y[i] * r2 * w_post[i]);
                }
                if (c < cols) store8<SF, WIDE>(row_of(a.x_out, row, a.ld_x_out, SF ? 4 : 2), c, cols, x + k * 8);
            }
        }
        if (!a.pre) continue;
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s[0] += x[k * 8 + e] * x[k * 8 + e];   // columns past the row hold zeros
        block_join<Sum, THREADS, 1>(s, slots, turn);
        const float r1 = 1.0f / sqrtf(s[0] * inv_cols + a.eps_pre);
#pragma unroll
        for (int i = 0; i < EPT; ++i) x[i] = x[i] * r1 * w_pre[i];
        if constexpr (QUANT) {
            float m[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < EPT; ++i) m[0] = MaxBits::join(m[0], fabsf(x[i]));
            block_join<MaxBits, THREADS, 1>(m, slots, turn);
            const QuantRow q = quant_row(m[0]);
            if (tid == 0) a.u_scale[row] = q.scale;
            const uint32_t q_cols = (uint32_t)a.q_cols;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
                if (c >= q_cols) continue;
                quant8<WIDE>(q, (int8_t *)row_of(a.u, row, a.ld_u, 1), c, q_cols,
                             [&](int e) { return x[k * 8 + e]; });
            }
        } else {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
                if (c < cols) store8<YF, WIDE>(row_of(a.u, row, a.ld_u, YF ? 4 : 2), c, cols, x + k * 8);
            }
        }
    }
}

// EPT floats of a thread, in registers, or in LDS where a workgroup's rows take
// all registers (16-byte pieces, neighbouring threads' next to each other).
template <int EPT, int THREADS, bool LDS>
struct Own {
    float v[EPT];
    static constexpr int BYTES = 0;
    __device__ __forceinline__ void place(char *) {}
    __device__ __forceinline__ float get(int i) const { return v[i]; }
    __device__ __forceinline__ void set(int i, float x) { v[i] = x; }
};
template <int EPT, int THREADS>
struct Own<EPT, THREADS, true> {
    f32x4_t *at;
    static constexpr int BYTES = EPT * THREADS * 4;
    __device__ __forceinline__ void place(char *p) { at = (f32x4_t *)p + threadIdx.x; }
    __device__ __forceinline__ float get(int i) const { return at[i / 4 * THREADS][i % 4]; }
    __device__ __forceinline__ void set(int i, float x) { at[i / 4 * THREADS][i % 4] = x; }
};
// Rows of more than 8192 columns keep w_pre and the sums for dw_post in LDS
// (8192 x 16384 bf16: 429 us, with all in registers and spills 1224).
template <int EPT, int THREADS>
constexpr bool kOwnInLds = EPT * THREADS > 8192;

// A row's inputs of the backward, as they lie in memory.
template <int VPT, bool SF, bool YF>
struct BackwardRow {
    Raw<SF> x[VPT], d[VPT];
    Raw<YF> y[VPT], u[VPT];
};

template <bool WIDE, int EPT, int THREADS, bool SF, bool YF, bool AHEAD>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(NormArgs a) {
    constexpr int VPT = EPT / 8;
    using Row = BackwardRow<VPT, SF, YF>;
    __shared__ JoinSlots<3> slots;
    int turn = 0;
    const int tid = threadIdx.x;
    const float inv_cols = 1.0f / (float)a.cols;
    const uint32_t cols = (uint32_t)a.cols;
    const int64_t first = (int64_t)blockIdx.x * a.rows_per_wg;
    int64_t last = first + a.rows_per_wg;
    if (last > a.rows) last = a.rows;

    // gw: gate * w_post.  Summed over rows: D * yh since the last change of
    // gate row (dgate is that times w_post, and gate times that goes into
    // dw_post), and du * xh.
    constexpr bool LDS = kOwnInLds<EPT, THREADS>;
    extern __shared__ __attribute__((aligned(16))) char own[];
    Own<EPT, THREADS, LDS> w_pre, s_post;
    w_pre.place(own);
    s_post.place(own + w_pre.BYTES);
    float gw[EPT], s_dy[EPT], s_pre[EPT];
    auto take = [&](Row &r, int64_t row) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
            r.x[k] = r.d[k] = Raw<SF>{};
            r.y[k] = r.u[k] = Raw<YF>{};
            if (c < cols && row < last) {
                if (a.pre) {
                    fetch8<SF, WIDE>(r.x[k], row_of(a.x_out, row, a.ld_x_out, SF ? 4 : 2), c, cols);
                    fetch8<YF, WIDE>(r.u[k], row_of(a.du, row, a.ld_du, YF ? 4 : 2), c, cols);
                }
                if (a.has_y) fetch8<YF, WIDE>(r.y[k], row_of(a.y, row, a.ld_y, YF ? 4 : 2), c, cols);
                if (a.dx_out) fetch8<SF, WIDE>(r.d[k], row_of(a.dx_out, row, a.ld_dx_out, SF ? 4 : 2), c, cols);
            }
        }
    };
    // A row of the gate and w_post + offset (1 where there is none).
    auto load_gate = [&](int64_t row, float (&g)[EPT], float (&w)[EPT]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) g[i] = w[i] = 1.0f;
        load_params<WIDE, EPT, THREADS, 2>(a, {a.gated ? gate_at(a, row) : nullptr, a.w_post}, {0.0f, a.weight_offset},
                                           {&g, &w});
    };
    int64_t gate_row = 0, gate_end = 0;
    auto begin_gate = [&](int64_t row) __attribute__((always_inline)) {
        if (a.gated) {
            gate_row = gate_of(a, row);
            gate_end = (gate_row + 1) * a.rows_per_gate;
        }
        float g[EPT], w[EPT];
        load_gate(gate_row, g, w);
#pragma unroll
        for (int i = 0; i < EPT; ++i) gw[i] = g[i] * w[i];
    };
    // Ends a gate row's rows: its part of dw_post, and its dgate, whole if all
    // its rows are this workgroup's, else a part: the head slot for the gate
    // row of the first row, the tail slot for a later one.
    auto end_gate = [&]() __attribute__((always_inline)) {
        const int64_t lo = gate_row * a.rows_per_gate;
        int64_t hi = lo + a.rows_per_gate;
        if (hi > a.rows) hi = a.rows;
        const bool whole = lo >= first && hi <= last;
        float *to = whole ? a.dgate + gate_row * a.cols
                          : a.part + ((int64_t)blockIdx.x * 4 + (gate_row == gate_of(a, first) ? 2 : 3)) * a.cols;
        float g[EPT], w[EPT];
        load_gate(gate_row, g, w);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
            if (c >= cols) continue;
            float d[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float &s = s_dy[k * 8 + e];
                s_post.set(k * 8 + e, s_post.get(k * 8 + e) + g[k * 8 + e] * s);
                d[e] = w[k * 8 + e] * s;
                s = 0.0f;
            }
            store8<true, WIDE>(to, c, cols, d);
        }
    };
    // the first row's loads before the parameters': with few rows their latency
    // is most of the time
    Row next;
    if constexpr (AHEAD) take(next, first);
    {
        float w[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            s_dy[i] = s_pre[i] = 0.0f;
            s_post.set(i, 0.0f);
            w[i] = 1.0f;
        }
        load_params<WIDE, EPT, THREADS, 1>(a, {a.w_pre}, {a.weight_offset}, {&w});
#pragma unroll
        for (int i = 0; i < EPT; ++i) w_pre.set(i, w[i]);
        begin_gate(first);
    }
    for (int64_t row = first; row < last; ++row) {
        Row r;
        if constexpr (AHEAD) {
            r = next;
            take(next, row + 1);
        } else {
            take(r, row);
        }
        if (a.gated && row >= gate_end) {
            end_gate();
            begin_gate(row);
        }
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
            settle8<SF, WIDE>(r.x[k], c, cols);
            settle8<SF, WIDE>(r.d[k], c, cols);
            settle8<YF, WIDE>(r.y[k], c, cols);
            settle8<YF, WIDE>(r.u[k], c, cols);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = k * 8 + e;
                const float x = raw_at(r.x[k], e), y = raw_at(r.y[k], e);
                s[0] += x * x;
                s[1] += raw_at(r.u[k], e) * w_pre.get(i) * x;
                s[2] += y * y;
            }
        }
        block_join<Sum, THREADS, 3>(s, slots, turn);
        const float r1 = 1.0f / sqrtf(s[0] * inv_cols + a.eps_pre);
        const float m1 = s[1] * inv_cols * r1;          // mean(a * xh)
        const float r2 = a.post ? 1.0f / sqrtf(s[2] * inv_cols + a.eps_post) : 1.0f;
        float b[EPT];
        float t[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
            float dx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = k * 8 + e;
                const float xh = raw_at(r.x[k], e) * r1, du = raw_at(r.u[k], e);
                float d = raw_at(r.d[k], e);
                if (a.pre) d += r1 * (du * w_pre.get(i) - xh * m1);
                s_pre[i] += du * xh;
                dx[e] = a.has_y ? a.res_scale * d : d;
                const float yh = raw_at(r.y[k], e) * r2;
                s_dy[i] += d * yh;
                b[i] = d * gw[i];
                t[0] += b[i] * yh;
            }
            if (c < cols) store8<SF, WIDE>(row_of(a.dx, row, a.ld_dx, SF ? 4 : 2), c, cols, dx);
        }
        if (!a.has_y) continue;
        float m2 = 0.0f;
        if (a.post) {
            block_join<Sum, THREADS, 1>(t, slots, turn);
            m2 = t[0] * inv_cols;                        // mean(b * yh)
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
            float dy[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                dy[e] = r2 * (b[k * 8 + e] - raw_at(r.y[k], e) * r2 * m2);
            if (c < cols) store8<YF, WIDE>(row_of(a.dy, row, a.ld_dy, YF ? 4 : 2), c, cols, dy);
        }
    }
    if (a.gated) {
        end_gate();
    } else {
#pragma unroll
        for (int i = 0; i < EPT; ++i) s_post.set(i, s_dy[i]);
    }
    float *part = a.part + (int64_t)blockIdx.x * 4 * a.cols;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const uint32_t c = (uint32_t)(k * THREADS + tid) * 8;
        if (c >= cols) continue;
        float sp[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) sp[e] = s_post.get(k * 8 + e);
        if (a.post) store8<true, WIDE>(part, c, cols, sp);
        if (a.pre) store8<true, WIDE>(part + a.cols, c, cols, s_pre + k * 8);
    }
}

// Adds the workgroups' partial sums.  blockIdx.y: 0 dw_post, 1 dw_pre, then the
// gate rows whose rows are not all one workgroup's: by gate row (by_group), or
// by the workgroup w whose end is the first to lie inside the gate row, where
// that makes fewer workgroups.  32 columns per workgroup; 32 threads per column
// take every 32nd partial, then add up in a fixed order.
__global__ __launch_bounds__(1024) void norm_join_kernel(NormArgs a, int64_t wgs, int by_group,
                                                         float *dw_post, float *dw_pre) {
    __shared__ float sums[32][32];
    const int col = threadIdx.x & 31, lane = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + col, cols = a.cols;
    const int y = blockIdx.y;
    float *to = nullptr;
    int64_t lo = 0, hi = wgs, g = -1;
    if (y == 0) to = dw_post;
    else if (y == 1) to = dw_pre;
    else {
        g = by_group ? y - 2 : (int64_t)(y - 1) * a.rows_per_wg / a.rows_per_gate;
        const int64_t start = g * a.rows_per_gate;
        int64_t stop = start + a.rows_per_gate;
        if (stop > a.rows) stop = a.rows;
        lo = start / a.rows_per_wg;
        hi = (stop + a.rows_per_wg - 1) / a.rows_per_wg;
        if (hi - lo < 2 || (!by_group && lo != y - 2)) return;   // whole, or another's
        to = a.dgate + g * a.cols;
    }
    if (!to) return;
    float s = 0.0f;
    if (c < cols) {
        const float *const part = a.part + c;
        // a gate row's first workgroup has it in its tail slot, unless the
        // gate row begins with the workgroup's first row
        const int64_t head_from = g >= 0 ? (g * a.rows_per_gate + a.rows_per_wg - 1) / a.rows_per_wg : 0;
#pragma unroll 8
        for (int64_t w = lo + lane; w < hi; w += 32)
            s += part[(w * 4 + (y < 2 ? y : w >= head_from ? 2 : 3)) * cols];
    }
    sums[lane][col] = s;
    __syncthreads();
    if (lane == 0 && c < cols) {
#pragma unroll
        for (int l = 1; l < 32; ++l) s += sums[l][col];
        to[c] = s;
    }
}

__global__ void norm_zero_kernel(float *a, float *b, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) {
        if (a) a[i] = 0.0f;
        if (b) b[i] = 0.0f;
    }
}

template <bool WIDE, int EPT, int THREADS>
hipError_t launch_forward(const NormArgs &a, bool sf, bool yf, bool quant, int64_t grid, hipStream_t s) {
    auto go = [&](auto *kernel) { return launch(kernel, dim3((unsigned)grid), THREADS, 0, s, a); };
    if (quant) {
        if (sf && yf) return go(norm_forward_kernel<WIDE, EPT, THREADS, true, true, true>);
        if (sf) return go(norm_forward_kernel<WIDE, EPT, THREADS, true, false, true>);
        if (yf) return go(norm_forward_kernel<WIDE, EPT, THREADS, false, true, true>);
        return go(norm_forward_kernel<WIDE, EPT, THREADS, false, false, true>);
    }
    if (sf && yf) return go(norm_forward_kernel<WIDE, EPT, THREADS, true, true, false>);
    if (sf) return go(norm_forward_kernel<WIDE, EPT, THREADS, true, false, false>);
    if (yf) return go(norm_forward_kernel<WIDE, EPT, THREADS, false, true, false>);
    return go(norm_forward_kernel<WIDE, EPT, THREADS, false, false, false>);
}

template <bool WIDE, int EPT, int THREADS>
hipError_t launch_backward(const NormArgs &a, bool sf, bool yf, int64_t grid, hipStream_t s) {
    // The next row is loaded ahead where rows are aligned and registers are left
    // for it (8192 rows in bf16, ahead / not: 8192 columns 168 / 173 us, 4096
    // columns 88 / 108, 2048 columns 51 / 49).  Unaligned rows need more registers
    // as it is, which a workgroup's only row pays for and many rows would gain by
    // (kernels in a graph, 8 x 8191 in float 11.8 / 10.8, 255 x 8191 25.3 / 24.4;
    // 1500 x 8191 61.8 / 65.5; calls, 8192 x 8191 in bf16 187 / 214, 4095 columns
    // 108 / 130).
    constexpr bool AHEAD = WIDE && !kOwnInLds<EPT, THREADS>;
    constexpr int lds = 2 * Own<EPT, THREADS, kOwnInLds<EPT, THREADS>>::BYTES;
    if (sf && yf) return launch_lds<norm_backward_kernel<WIDE, EPT, THREADS, true, true, AHEAD>>(grid, THREADS, lds, s, a);
    if (sf) return launch_lds<norm_backward_kernel<WIDE, EPT, THREADS, true, false, AHEAD>>(grid, THREADS, lds, s, a);
    if (yf) return launch_lds<norm_backward_kernel<WIDE, EPT, THREADS, false, true, AHEAD>>(grid, THREADS, lds, s, a);
    return launch_lds<norm_backward_kernel<WIDE, EPT, THREADS, false, false, AHEAD>>(grid, THREADS, lds, s, a);
}

// Threads of a workgroup and columns of a row per thread.
template <int EPT_, int THREADS_>
struct Shape {
    static constexpr int EPT = EPT_, THREADS = THREADS_;
};

// Calls f with the kernel shape of a row length.  Up to 8192 columns: many rows
// take 512 threads, which leaves each CU rows to overlap (bf16, 512 / 1024
// threads: 8192 x 8192 98 / 100 us, 8192 x 8191 116 / 143, 300 x 8191 in a graph
// 8.6 / 10.5); up to one row per CU take 1024, whose shorter chain per thread
// serves rows that are not aligned (in a graph, 64 x 8191 5.6 / 5.3, 64 x 8192
// 4.1 / 4.3).
template <class F>
void forward_shape(int64_t rows, int64_t cols, F f) {
    if (cols <= 512) f(Shape<8, 64>{});
    else if (cols <= 1024) f(Shape<8, 128>{});
    else if (cols <= 2048) f(Shape<8, 256>{});
    else if (cols <= 4096) f(Shape<8, 512>{});
    else if (cols <= 8192 && rows < kCus) f(Shape<8, 1024>{});
    else if (cols <= 8192) f(Shape<16, 512>{});
    else f(Shape<16, 1024>{});
}
template <class F>
void backward_shape(int64_t cols, F f) {
    if (cols <= 512) f(Shape<8, 64>{});
    else if (cols <= 1024) f(Shape<8, 128>{});
    else if (cols <= 2048) f(Shape<8, 256>{});
    else if (cols <= 4096) f(Shape<8, 512>{});
    else if (cols <= 8192) f(Shape<16, 512>{});
    else f(Shape<32, 512>{});
}

// Most workgroups of a backward launch: enough to fill the CUs' wave slots
// that the kernel's registers allow, and no more, because each writes 4 rows
// of partial sums.
int64_t backward_wgs(int64_t rows, int64_t cols) {
    int64_t cap = 0;
    backward_shape(cols, [&](auto sh) {
        cap = (int64_t)kCus * 512 / decltype(sh)::THREADS;
    });
    if (cap > 2048) cap = 2048;
    return rows < cap ? rows : cap;
}

}  // namespace

struct block_norm_plan_s {
    block_norm_desc_t d;
    int device;
    float *part;
    int64_t part_bytes;
};

namespace {

bool flag(int32_t v) { return v == 0 || v == 1; }

int validate(const block_norm_desc_t &d) {
    if (d.rows < 1 || d.cols < 1 || d.rows_per_gate < 0 || d.pad != 0) return GEMM_RS_ERR_INVALID_ARG;
    if (!known_type(d.dtype) || !known_type(d.stream_dtype) || !known_type(d.param_dtype))
        return GEMM_RS_ERR_INVALID_ARG;
    if (!flag(d.has_y) || !flag(d.post) || !flag(d.pre) || !flag(d.quant) || !flag(d.backward))
        return GEMM_RS_ERR_INVALID_ARG;
    if (!d.has_y && (d.post || d.rows_per_gate || !d.pre)) return GEMM_RS_ERR_INVALID_ARG;
    if (d.quant && (!d.pre || d.backward)) return GEMM_RS_ERR_INVALID_ARG;
    if (!isfinite(d.res_scale) || !isfinite(d.weight_offset) || !isfinite(d.eps_post) ||
        !isfinite(d.eps_pre) || d.eps_post < 0 || d.eps_pre < 0)
        return GEMM_RS_ERR_INVALID_ARG;
    const int64_t lds[] = {d.ld_x, d.ld_y, d.ld_x_out, d.ld_u, d.ld_dx_out, d.ld_du, d.ld_dx, d.ld_dy};
    for (int64_t ld : lds)
        if (ld != 0 && ld < d.cols) return GEMM_RS_ERR_INVALID_ARG;
    for (int64_t ld : lds)
        if (ld > INT32_MAX) return GEMM_RS_ERR_UNSUPPORTED;
    if (d.cols > kMaxCols || d.rows > INT32_MAX || d.rows_per_gate > INT32_MAX)
        return GEMM_RS_ERR_UNSUPPORTED;
    return GEMM_RS_OK;
}

NormArgs args_of(const block_norm_desc_t &d, int64_t rows) {
    NormArgs a = {};
    a.rows = rows;
    a.cols = d.cols;
    a.rows_per_gate = d.rows_per_gate ? d.rows_per_gate : 1;
    auto ld = [&](int64_t v) { return v ? v : d.cols; };
    a.ld_x = ld(d.ld_x);
    a.ld_y = ld(d.ld_y);
    a.ld_x_out = ld(d.ld_x_out);
    a.ld_u = ld(d.ld_u);
    a.ld_dx_out = ld(d.ld_dx_out);
    a.ld_du = ld(d.ld_du);
    a.ld_dx = ld(d.ld_dx);
    a.ld_dy = ld(d.ld_dy);
    a.res_scale = d.res_scale;
    a.weight_offset = d.weight_offset;
    a.eps_post = d.eps_post;
    a.eps_pre = d.eps_pre;
    a.has_y = d.has_y;
    a.post = d.post;
    a.pre = d.pre;
    a.gated = d.rows_per_gate > 0;
    a.param_f32 = d.param_dtype == GEMM_RS_F32;
    return a;
}

// A pointer is there exactly if it is wanted, at a multiple of its element.
bool fits(const void *p, bool wanted, size_t elem) {
    return wanted ? (p && aligned(p, elem)) : !p;
}
// The same of an array of rows, which a call without rows may leave out: an
// array without elements need not have an address.
bool fits_rows(const void *p, bool wanted, size_t elem, int64_t rows) {
    return fits(p, wanted && (p || rows > 0), elem);
}

// Whether rows at p, ld elements apart, can be accessed 8 elements (8
// bytes of int8) at a time.
bool wide(const void *p, int64_t ld, size_t elem) {
    return !p || (ld % 8 == 0 && aligned(p, elem == 1 ? 8 : 16));
}

}  // namespace

extern "C" {

int block_norm_plan(const block_norm_desc_t *desc, block_norm_plan_t *out) {
    if (!desc || !out) return GEMM_RS_ERR_INVALID_ARG;
    *out = nullptr;
    const int rc = validate(*desc);
    if (rc != GEMM_RS_OK) return rc;
    block_norm_plan_s *p = (block_norm_plan_s *)calloc(1, sizeof(block_norm_plan_s));
    if (!p) return GEMM_RS_ERR_HIP;
    p->d = *desc;
    if (own(hipGetDevice(&p->device)) != hipSuccess) {
        free(p);
        return GEMM_RS_ERR_HIP;
    }
    if (desc->backward) {
        p->part_bytes = backward_wgs(desc->rows, desc->cols) * 4 * desc->cols * (int64_t)sizeof(float);
        if (own(hipMalloc((void **)&p->part, p->part_bytes)) != hipSuccess) {
            free(p);
            return GEMM_RS_ERR_HIP;
        }
    }
    *out = p;
    return GEMM_RS_OK;
}

int block_norm_run(block_norm_plan_t p, const void *x, const void *y, const void *w_post,
                   const void *gate, const void *w_pre, void *x_out, void *u, void *u_scale,
                   int64_t rows, void *stream) {
    if (!p || !on_device(p->device)) return GEMM_RS_ERR_INVALID_ARG;
    const block_norm_desc_t &d = p->d;
    if (rows < 0 || rows > d.rows) return GEMM_RS_ERR_INVALID_ARG;
    const size_t se = type_bytes(d.stream_dtype), ye = type_bytes(d.dtype), pe = type_bytes(d.param_dtype);
    const size_t ue = d.quant ? 1 : ye;
    if (!fits_rows(x, true, se, rows) || !fits_rows(y, d.has_y, ye, rows) || !fits(w_post, d.post, pe) ||
        !fits_rows(gate, d.rows_per_gate > 0, pe, rows) || !fits(w_pre, d.pre, pe) ||
        !fits_rows(x_out, d.has_y, se, rows) || !fits_rows(u, d.pre, ue, rows) ||
        !fits_rows(u_scale, d.quant, 4, rows))
        return GEMM_RS_ERR_INVALID_ARG;
    if (rows == 0) return GEMM_RS_OK;
    NormArgs a = args_of(d, rows);
    if (x == x_out && a.ld_x != a.ld_x_out) return GEMM_RS_ERR_INVALID_ARG;
    a.x = x;
    a.y = y;
    a.w_post = w_post;
    a.gate = gate;
    a.w_pre = w_pre;
    a.x_out = x_out;
    a.u = u;
    a.u_scale = (float *)u_scale;
    // (a kernel shape holds whole runs of 16 columns, so these too)
    const int64_t padded = (d.cols + 15) / 16 * 16;
    a.q_cols = a.ld_u >= padded ? padded : d.cols;
    const bool wide_rows = d.cols % 8 == 0 && wide(x, a.ld_x, se) && wide(y, a.ld_y, ye) &&
                     wide(w_post, 8, pe) && wide(gate, 8, pe) && wide(w_pre, 8, pe) &&
                     wide(x_out, a.ld_x_out, se) && wide(u, a.ld_u, ue);
    hipError_t e = hipSuccess;
    forward_shape(rows, d.cols, [&](auto sh) {
        using S = decltype(sh);
        const int64_t most = (int64_t)kCus * 2048 / S::THREADS, grid = rows < most ? rows : most;
        const bool sf = d.stream_dtype == GEMM_RS_F32, yf = d.dtype == GEMM_RS_F32;
        e = wide_rows ? launch_forward<true, S::EPT, S::THREADS>(a, sf, yf, d.quant != 0, grid, (hipStream_t)stream)
                      : launch_forward<false, S::EPT, S::THREADS>(a, sf, yf, d.quant != 0, grid, (hipStream_t)stream);
    });
    return e == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int block_norm_backward(block_norm_plan_t p, const void *dx_out, const void *du, const void *x_out,
                        const void *y, const void *w_post, const void *gate, const void *w_pre,
                        void *dx, void *dy, void *dw_post, void *dgate, void *dw_pre, int64_t rows,
                        void *stream) {
    if (!p || !on_device(p->device) || !p->d.backward) return GEMM_RS_ERR_INVALID_ARG;
    const block_norm_desc_t &d = p->d;
    if (rows < 0 || rows > d.rows) return GEMM_RS_ERR_INVALID_ARG;
    const size_t se = type_bytes(d.stream_dtype), ye = type_bytes(d.dtype), pe = type_bytes(d.param_dtype);
    const bool gated = d.rows_per_gate > 0;
    if (!fits_rows(dx_out, dx_out || !d.pre, se, rows) || !fits_rows(du, d.pre, ye, rows) ||
        !fits_rows(x_out, d.pre, se, rows) || !fits_rows(y, d.has_y, ye, rows) || !fits(w_post, d.post, pe) ||
        !fits_rows(gate, gated, pe, rows) || !fits(w_pre, d.pre, pe) || !fits_rows(dx, true, se, rows) ||
        !fits_rows(dy, d.has_y, ye, rows) || !fits(dw_post, d.post, 4) || !fits_rows(dgate, gated, 4, rows) ||
        !fits(dw_pre, d.pre, 4))
        return GEMM_RS_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = hipSuccess;
    if (rows == 0) {
        if (dw_post || dw_pre)
            e = launch(norm_zero_kernel, dim3((unsigned)((d.cols + 255) / 256)), 256, 0, s, (float *)dw_post,
                       (float *)dw_pre, d.cols);
        return e == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
    }
    NormArgs a = args_of(d, rows);
    a.x_out = (void *)x_out;
    a.dx_out = dx_out;
    a.du = du;
    a.y = y;
    a.w_post = w_post;
    a.gate = gate;
    a.w_pre = w_pre;
    a.dx = dx;
    a.dy = dy;
    a.dgate = (float *)dgate;
    a.part = p->part;
    const bool wide_rows = d.cols % 8 == 0 && wide(x_out, a.ld_x_out, se) && wide(y, a.ld_y, ye) &&
                     wide(dx_out, a.ld_dx_out, se) && wide(du, a.ld_du, ye) &&
                     wide(w_post, 8, pe) && wide(gate, 8, pe) && wide(w_pre, 8, pe) &&
                     wide(dx, a.ld_dx, se) && wide(dy, a.ld_dy, ye) && wide(dgate, 8, 4);
    int64_t wgs = backward_wgs(rows, d.cols);
    a.rows_per_wg = (rows + wgs - 1) / wgs;
    wgs = (rows + a.rows_per_wg - 1) / a.rows_per_wg;
    backward_shape(d.cols, [&](auto sh) {
        using S = decltype(sh);
        const bool sf = d.stream_dtype == GEMM_RS_F32, yf = d.dtype == GEMM_RS_F32;
        e = wide_rows ? launch_backward<true, S::EPT, S::THREADS>(a, sf, yf, wgs, s)
                      : launch_backward<false, S::EPT, S::THREADS>(a, sf, yf, wgs, s);
    });
    if (e != hipSuccess) return GEMM_RS_ERR_HIP;
    // gate rows lie across workgroups' ends unless the runs are whole groups
    const bool split = gated && wgs > 1 && a.rows_per_wg % a.rows_per_gate != 0;
    if (d.post || d.pre || split) {
        const int64_t gates = (rows + a.rows_per_gate - 1) / a.rows_per_gate;
        const bool by_group = gates < wgs - 1;
        const unsigned ny = 2 + (split ? (unsigned)(by_group ? gates : wgs - 1) : 0);
        e = launch(norm_join_kernel, dim3((unsigned)((d.cols + 31) / 32), ny), 1024, 0, s, a, wgs, (int)by_group,
                   (float *)dw_post, (float *)dw_pre);
    }
    return e == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int block_norm_query(block_norm_plan_t p, block_norm_info_t *info) {
    if (!p || !info) return GEMM_RS_ERR_INVALID_ARG;
    const block_norm_desc_t &d = p->d;
    info->gate_rows = d.rows_per_gate ? (d.rows + d.rows_per_gate - 1) / d.rows_per_gate : 0;
    info->workspace_bytes = p->part_bytes;
    return GEMM_RS_OK;
}

int block_norm_destroy(block_norm_plan_t p) {
    if (!p) return GEMM_RS_OK;
    int cur = -1;
    bool switched = false;
    if (p->part && own(hipGetDevice(&cur)) == hipSuccess && cur != p->device)
        switched = own(hipSetDevice(p->device)) == hipSuccess;
    // teardown is best effort: a failure here leaves nothing to undo
    if (p->part) (void)own(hipFree(p->part));
    if (switched) (void)own(hipSetDevice(cur));
    free(p);
    return GEMM_RS_OK;
}

}  // extern "C"
