// Gradients that the gated projections and the product with epilogue share: of the
// values before the activation, of the biases, and of the weights.
#include "dense_tile.h"

namespace gemm_rs {
namespace ffn {

namespace {

// ---- gradients of the values before the activation ---------------------------------
// dz = dy * act'(z); a pair's dz0 = dy * z1 * act'(z0), dz1 = dy * act(z0).  Bound by
// memory: a lane takes 8 columns (16 bytes of each array), a wave 512 columns of a
// row, a workgroup's 4 waves every fourth row of a chunk, 2 rows of loads ahead of
// their use.
//
// dz is rounded to bfloat16, since dx and dW take it as an operand of bfloat16 matrix
// operations; its rest as a second operand would double their work.  The rounding is
// off by 1.66e-3 of dz (root mean square), as any to bfloat16, and so are its sums in
// dx and dW, beside their own rounding: 2.35e-3 against 64 bits (8192 rows, 4096 x
// 3584 in pairs; 1000 rows, 4096 x 1792; 6001 rows, 2048 x 1792), where a product of
// unrounded dz has 1.66e-3.  The biases' gradients are sums over rows of the unrounded dz: in
// registers over a wave's rows, over the waves in LDS, over the chunks in a second
// kernel, each in a fixed order.
constexpr int kGradCols = 512, kGradWaves = 4, kGradRows = 2;

template <bool PAIR, bool DY32, bool Z32, bool WIDE>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs p) {
    constexpr int ARRAYS = PAIR ? 2 : 1, U = kGradRows;
    __shared__ float joined[kGradWaves][ARRAYS * 8][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const uint32_t cols = (uint32_t)p.N, c = blockIdx.x * kGradCols + lane * 8;
    const int64_t per = (p.rows + p.chunks - 1) / p.chunks, r0 = blockIdx.y * per;
    const int64_t r1 = r0 + per < p.rows ? r0 + per : p.rows;
    const bool sums = p.db[0] || p.db[ARRAYS - 1], live = c < cols;
    float s[ARRAYS][8] = {};
    if (live)
        for (int64_t at = r0 + wave; at < r1; at += U * kGradWaves) {
            Raw<DY32> dy[U];
            Raw<Z32> z[U][ARRAYS];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = at + u * kGradWaves;
                if (row >= r1) break;
                fetch8<DY32, WIDE>(dy[u], row_of(p.dy, row, p.ldy, DY32 ? 4 : 2), c, cols);
#pragma unroll
                for (int a = 0; a < ARRAYS; ++a)
                    if (p.Z[a]) fetch8<Z32, WIDE>(z[u][a], row_of(p.Z[a], row, p.ldz, Z32 ? 4 : 2), c, cols);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = at + u * kGradWaves;
                if (row >= r1) break;
                settle8<DY32, WIDE>(dy[u], c, cols);
                float zf[8] = {}, value[8], slope[8], d[ARRAYS][8];
#pragma unroll
                for (int a = 0; a < ARRAYS; ++a) settle8<Z32, WIDE>(z[u][a], c, cols);
                if (p.Z[0])
#pragma unroll
                    for (int e = 0; e < 8; ++e) zf[e] = raw_at(z[u][0], e);
                activate_both(p.act, zf, value, slope);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float g = raw_at(dy[u], e);
                    if constexpr (PAIR) {
                        d[0][e] = g * raw_at(z[u][1], e) * slope[e];
                        d[1][e] = g * value[e];
                    } else {
                        d[0][e] = g * slope[e];
                    }
                }
#pragma unroll
                for (int a = 0; a < ARRAYS; ++a) {
                    if (p.dZ[a]) store8<false, WIDE>(row_of((void *)p.dZ[a], row, p.lddz, 2), c, cols, d[a]);
                    // (past the row's end dy was settled to zeros)
                    if (p.copy[a]) store8<false, true>(row_of((void *)p.copy[a], row, p.copy_ld, 2), c, cols, d[a]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[a][e] += d[a][e];
                }
            }
        }
    if (!sums) return;
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a)
#pragma unroll
        for (int e = 0; e < 8; ++e) joined[wave][a * 8 + e][lane] = s[a][e];
    lds_only_barrier();
    for (int i = threadIdx.x; i < ARRAYS * kGradCols; i += 256) {
        const int a = i / kGradCols, n = i % kGradCols;
        const uint32_t col = blockIdx.x * kGradCols + n;
        float *const db = a ? p.db[ARRAYS - 1] : p.db[0];
        if (col >= cols || !db) continue;
        float t = 0;
#pragma unroll
        for (int w = 0; w < kGradWaves; ++w) t += joined[w][a * 8 + n % 8][n / 8];
        if (p.chunks > 1) p.sums[((int64_t)blockIdx.y * ARRAYS + a) * p.N + col] = t;
        else db[col] = p.add ? db[col] + t : t;
    }
}

// Adds the chunks' sums: 64 columns per workgroup, the chunks dealt out to 16 waves.
__global__ __launch_bounds__(1024) void bias_join_kernel(ActGradArgs p) {
    __shared__ float joined[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, a = blockIdx.y, arrays = gridDim.y;
    float *const db = a ? p.db[1] : p.db[0];
    const int64_t col = (int64_t)blockIdx.x * 64 + lane;
    if (!db) return;
    float t = 0;
    if (col < p.N)
#pragma unroll 4
        for (int k = wave; k < p.chunks; k += 16) t += p.sums[((int64_t)k * arrays + a) * p.N + col];
    joined[wave][lane] = t;
    __syncthreads();
    if (wave > 0 || col >= p.N) return;
    for (int w = 1; w < 16; ++w) t += joined[w][lane];
    db[col] = p.add ? db[col] + t : t;
}

// A wave per row, 16 bytes per lane at any element address; every 4 * kCopyGroups-th
// row where there are more.
constexpr int64_t kCopyGroups = 1 << 22;
__global__ __launch_bounds__(256) void padded_copy_kernel(PadArgs p) {
    constexpr int U = 4;                // loads ahead
    const int lane = threadIdx.x & 63;
    for (int64_t at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);; at += 4 * kCopyGroups) {
        int64_t row = at;
        int which = 0;
        while (which < p.count && row >= p.m[which].rows) row -= p.m[which++].rows;
        if (which == p.count) return;
        const auto &m = p.m[which];
        const uint16_t *const from = m.from + row * m.ld;
        uint16_t *const to = m.to + row * m.to_ld;
        const uint32_t cols = (uint32_t)m.cols, all = (uint32_t)m.to_ld;
        for (uint32_t c0 = lane * 8; c0 < all; c0 += U * 512) {
            Raw<false> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * 512 < all) fetch8<false, false>(r[u], from, c0 + u * 512, cols);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t c = c0 + u * 512;
                if (c >= all) break;
                settle8<false, false>(r[u], c, cols);
                *(u32x4_t *)(to + c) = r[u].a;
            }
        }
    }
}

// Rows per wave times waves to a chunk at least, and about 8 workgroups per CU.
int grad_chunks(int64_t rows, int64_t N) {
    const int64_t blocks = (N + kGradCols - 1) / kGradCols;
    int64_t most = 8 * kCus / blocks, chunks = (rows + 2 * kGradWaves * kGradRows - 1) / (2 * kGradWaves * kGradRows);
    if (most < 1) most = 1;
    if (chunks > most) chunks = most;
    return chunks < 1 ? 1 : (int)chunks;
}

}  // namespace

int64_t activation_gradient_slots(int64_t rows, int64_t N, int arrays) {
    const int chunks = grad_chunks(rows, N);
    return chunks > 1 ? chunks * arrays * N * (int64_t)sizeof(float) : 0;
}

hipError_t launch_activation_gradient(ActGradArgs &a, int64_t room, hipStream_t s) {
    const int arrays = a.pair ? 2 : 1;
    const bool sums = a.db[0] || a.db[arrays - 1];
    a.chunks = grad_chunks(a.rows, a.N);
    if (sums) {                     // (a chunk's sums fit the plan's room)
        const int64_t fit = room / (arrays * a.N * (int64_t)sizeof(float));
        if (a.chunks > 1 && fit < a.chunks) a.chunks = fit < 1 ? 1 : (int)fit;
    }
    const dim3 grid((unsigned)((a.N + kGradCols - 1) / kGradCols), (unsigned)a.chunks);
    const std::true_type yes{};
    const std::false_type no{};
    auto run = [&](auto pair, auto dy32, auto z32, auto wide) {
        return launch(act_grad_kernel<decltype(pair)::value, decltype(dy32)::value, decltype(z32)::value, decltype(wide)::value>, grid, 256, 0, s, a);
    };
    auto types = [&](auto pair, auto dy32, auto z32) { return a.wide ? run(pair, dy32, z32, yes) : run(pair, dy32, z32, no); };
    auto of = [&](auto pair, auto dy32) { return a.z_f32 ? types(pair, dy32, yes) : types(pair, dy32, no); };
    const hipError_t e = a.pair ? of(yes, no) : a.dy_f32 ? of(no, yes) : of(no, no);
    if (e != hipSuccess || !sums || a.chunks == 1) return e;
    return launch(bias_join_kernel, dim3((unsigned)((a.N + 63) / 64), (unsigned)arrays), 1024, 0, s, a);
}

hipError_t launch_padded_copies(const PadArgs &a, hipStream_t s) {
    int64_t rows = 0;
    for (int i = 0; i < a.count; ++i) rows += a.m[i].rows;
    const int64_t groups = (rows + 3) / 4;
    return rows > 0 ? launch(padded_copy_kernel, dim3((unsigned)(groups < kCopyGroups ? groups : kCopyGroups)), 256, 0, s, a) : hipSuccess;
}

// ---- weight gradients ----------------------------------------------------------
hipError_t launch_weight_gradients(DenseArgs &a, bool direct, int64_t slot_bytes, hipStream_t s) {
    a.ldr = a.ldd;
    if (!direct || (a.add && a.N < 8)) return launch_dense_narrow<kOne, true, true>(a, s);
    const DenseWay way = dense_tn_choice(a.K, a.rows, a.N, a.count, a.out_f32 ? 4 : 2);
    // Stores past the caches have to cover whole lines: a tile's rows of bfloat16 do,
    // but for their ends, those of floats only where they begin on a line.
    a.stream = !a.out_f32 || (a.ldd % 32 == 0 && aligned(a.D[0], 128) && (a.count == 1 || aligned(a.D[1], 128)));
    switch (way.kernel) {
    case kDense256: return launch_dense_tile<kOne, true, true, 256, 256, 2, 4, 2, 2>(a, way.parts, slot_bytes, s);
    case kDense128x256: return launch_dense_tile<kOne, true, true, 128, 256, 2, 4, 3, 3>(a, way.parts, slot_bytes, s);
    case kDense128Deep: return launch_dense_tile<kOne, true, true, 128, 128, 2, 4, 4, 4>(a, way.parts, slot_bytes, s);
    default: return launch_dense_tile<kOne, true, true, 128, 128, 2, 2, 2, 2>(a, way.parts, slot_bytes, s);
    }
}

}  // namespace ffn
}  // namespace gemm_rs
