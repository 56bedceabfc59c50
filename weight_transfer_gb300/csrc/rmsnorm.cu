// Residual addition and root-mean-square norm with an output in 8 bits, and
// the gradient of the norm.
//
// Forward, per row of k elements, all in binary32:
//     h = x + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = (h * rstd) * w
// and y is quantized where it is made: blockwise FP8 (one binary32 scale per
// 128) or MXFP8 (one E8M0 byte per 32), by the rules of fp8q_quantize_blockwise
// and mxfp8_quantize_swizzled applied to the binary32 y.  The norm is taken of
// the unrounded sum h; only the stored sum is rounded to bf16.
//
// The work is bound by HBM: a row is read once and stays in registers between
// the sum of squares and the output, and the next row is read meanwhile (one
// row per block without that took 110.6 us where this takes 100.4: 16,384 rows
// of 4096 with residual, MXFP8 and bf16 outputs).  Back to back that case runs
// at 6.3 TB/s (95.9 us, 93% of the measured copy rate); ncu counts 22
// thread-instructions per element and 40% of the issue slots.  Few rows are
// bound by latency, and below about 20 us by the caller's launches.
#include "fp8q_device.cuh"
#include "fp8q_host.cuh"

#include <math.h>

namespace fp8q {

enum NormOut { kNormE4M3 = 0, kNormE5M2 = 1, kNormMxRows = 2, kNormMxTiled = 3 };

struct NormArgs {
    const uint16_t* x;
    const uint16_t* residual;   // or NULL
    const uint16_t* weight;
    uint16_t* sum;              // or NULL
    uint16_t* y;                // or NULL
    uint8_t* codes;
    void* scales;
    float* rstd;                // or NULL
    int64_t rows;
    int64_t padded_rows;        // rows, or the next multiple of 128 for the tiled scale layout
    int k;
    float eps;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    return v;
}

constexpr int kNormWarps = 4;   // warps of a block whose warps have a row each

// How the threads of a block share the rows: a warp per row (short rows, no
// barrier at all) or the whole block per row.  Blocks walk over the rows with
// a fixed stride; the weights stay in registers and the next row is on its way
// while this one is summed up and written.
template <bool WARP_ROWS> struct RowGroup {
    int t;                      // thread inside the group
    int size;                   // threads of the group
    int64_t first, stride;      // rows of this group
    __device__ __forceinline__ RowGroup() {
        if (WARP_ROWS) {
            const int groups = (int)blockDim.x >> 5;
            t = (int)(threadIdx.x & 31u);
            size = 32;
            first = (int64_t)blockIdx.x * groups + (threadIdx.x >> 5);
            stride = (int64_t)gridDim.x * groups;
        } else {
            t = (int)threadIdx.x;
            size = (int)blockDim.x;
            first = blockIdx.x;
            stride = gridDim.x;
        }
    }
    // Sum over the group, the same value in every thread and the same order on
    // every run.  `slot` alternates between two shared arrays, so that one
    // barrier per row is enough.
    __device__ __forceinline__ float sum(float v, float (*red)[32], int slot) const {
        v = warp_sum(v);
        if (WARP_ROWS) return v;
        const int warps = size >> 5;
        if ((t & 31) == 0) red[slot][t >> 5] = v;
        __syncthreads();
        float s = 0.0f;
        for (int i = 0; i < warps; ++i) s += red[slot][i];
        return s;
    }
};

// Position of scale column j of row r in the 128x4-tiled layout (`tiles` column tiles).
__device__ __forceinline__ int64_t tiled_scale_at(int64_t r, int j, int tiles) {
    return ((r >> 7) * tiles + (j >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (j & 3);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Thread t of a group holds the 8-element chunks t, t + size, ... (V of them).
template <int OUT, int V, bool WARP_ROWS>
__global__ void __launch_bounds__(512) rmsnorm_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    const RowGroup<WARP_ROWS> g;
    const int chunks = a.k >> 3;
    constexpr bool kMx = OUT == kNormMxRows || OUT == kNormMxTiled;
    const int scale_cols = kMx ? a.k >> 5 : a.k >> 7;
    const int tiles = (scale_cols + 3) >> 2;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    dependency_wait();
    allow_dependents();
    uint4 w[V], x[V], r[V];
    auto fetch = [&](int64_t row) {
        const int64_t base = row * a.k;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = g.t + v * g.size;
            const bool ok = row < a.rows && c < chunks;
            x[v] = ok ? ld_once(a.x + base + c * 8) : zero;
            r[v] = ok && a.residual ? ld_once(a.residual + base + c * 8) : zero;
        }
    };
    fetch(g.first);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = g.t + v * g.size;
        w[v] = c < chunks ? *reinterpret_cast<const uint4*>(a.weight + c * 8) : zero;
    }
    int slot = 0;
    for (int64_t row = g.first; row < a.padded_rows; row += g.stride, slot ^= 1) {
        if (OUT == kNormMxTiled) {
            // padding of the tiled layout is zero: whole rows past the last one, and the columns that fill up a tile
            uint8_t* s8 = static_cast<uint8_t*>(a.scales);
            const int first = row < a.rows ? scale_cols : 0;
            for (int j = first + g.t; j < tiles * 4; j += g.size) s8[tiled_scale_at(row, j, tiles)] = 0;
            if (row >= a.rows) continue;
        }
        const int64_t base = row * a.k;
        float h[V][8];
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            unpack8(x[v], h[v]);
            if (a.residual) {
                float f[8];
                unpack8(r[v], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[v][i] = __fadd_rn(h[v][i], f[i]);
                const int c = g.t + v * g.size;
                if (a.sum && c < chunks) st_stream(a.sum + base + c * 8, pack8(h[v]));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __fmaf_rn(h[v][i], h[v][i], ss);
        }
        fetch(row + g.stride);
        const float mean = g.sum(ss, red, slot) / (float)a.k;
        const float rstd = 1.0f / sqrtf(mean + a.eps);
        if (g.t == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = g.t + v * g.size;
            const bool ok = c < chunks;
            float y[8], f[8];
            unpack8(w[v], f);
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] = __fmul_rn(__fmul_rn(h[v][i], rstd), f[i]);
                m = fmaxf(m, fabsf(y[i]));
            }
            if (ok && a.y) st_stream(a.y + base + c * 8, pack8(y));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            float q[8];
            if (kMx) {
                const int E = (int)(__float_as_uint(m) >> 23);
                const int e8 = E > 8 ? E - 8 : 0;
                const float factor = __uint_as_float((uint32_t)(254 - e8) << 23);
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(y[i], factor);
                if (ok && (c & 3) == 0) {
                    uint8_t* s8 = static_cast<uint8_t*>(a.scales);
                    const int j = c >> 2;
                    if (OUT == kNormMxRows)
                        s8[row * scale_cols + j] = (uint8_t)e8;
                    else
                        s8[tiled_scale_at(row, j, tiles)] = (uint8_t)e8;
                }
                if (ok)
                    st_stream(a.codes + base + c * 8, make_uint2(cvt_fp8x4<kE4M3>(q[0], q[1], q[2], q[3]),
                                                                 cvt_fp8x4<kE4M3>(q[4], q[5], q[6], q[7])));
            } else {
                constexpr int FMT = OUT == kNormE5M2 ? kE5M2 : kE4M3;
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
                const float s = block_scale<FMT>(m);
                // y itself carries some ulps, so that the quotient is y * RN(1 / s), within 1.5 ulp of y / s
                if (s >= 0x1p-100f || s == 0.0f) {
                    const float inv = s > 0.0f ? __frcp_rn(s) : 1.0f;   // an all-zero block keeps its zeros
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(y[i], inv);
                } else {
                    block_quotients<2, 8>(y, s, q);
                }
                if (ok && (c & 15) == 0) static_cast<float*>(a.scales)[row * scale_cols + (c >> 4)] = s;
                if (ok)
                    st_stream(a.codes + base + c * 8, make_uint2(cvt_fp8x4<FMT>(q[0], q[1], q[2], q[3]),
                                                                 cvt_fp8x4<FMT>(q[4], q[5], q[6], q[7])));
            }
        }
    }
}

// ------------------------------------------------------------- gradient ----
//   g = dy * w;  xhat = h * rstd;  dx = rstd * (g - xhat * mean(g * xhat)) + dsum;  dw = sum over rows of dy * xhat
// 16,384 rows of 4096 with dsum take 88.3 us back to back (6.1 TB/s, 90% of the
// copy rate), of which the second kernel has about 5.
// Each thread keeps dw of its own columns in registers over all its rows; the
// blocks' partial sums are joined in a fixed order by a second kernel, so the
// result does not depend on timing.
struct NormGradArgs {
    const uint16_t* dy;
    const uint16_t* h;
    const uint16_t* weight;
    const float* rstd;
    const uint16_t* dsum;       // or NULL
    uint16_t* dx;
    float* partial;             // [blocks][k]
    int64_t rows;
    int k;
};

template <int V, bool WARP_ROWS>
__global__ void __launch_bounds__(512) rmsnorm_backward_kernel(const NormGradArgs a) {
    // four chunks per thread leave no registers for the next row, nor for the weights, which come from the first-level
    // cache again (4096 x 16384 with dsum: 102 us; with both in registers 117, next row in shared memory 112)
    constexpr bool kAhead = V < 4;
    __shared__ float red[2][32];
    __shared__ float joined[WARP_ROWS ? kNormWarps * V * 256 : 1];
    const RowGroup<WARP_ROWS> g;
    const int chunks = a.k >> 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    dependency_wait();
    allow_dependents();
    uint4 w[kAhead ? V : 1], dy_next[V], h_next[V], ds_next[V];
    float rstd_next = 0.0f;
    auto fetch = [&](int64_t row) {
        const int64_t base = row * a.k;
        rstd_next = row < a.rows ? a.rstd[row] : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = g.t + v * g.size;
            const bool ok = row < a.rows && c < chunks;
            dy_next[v] = ok ? ld_once(a.dy + base + c * 8) : zero;
            h_next[v] = ok ? ld_once(a.h + base + c * 8) : zero;
            ds_next[v] = ok && a.dsum ? ld_once(a.dsum + base + c * 8) : zero;
        }
    };
    if (kAhead) fetch(g.first);
    float dw[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = g.t + v * g.size;
        if (kAhead) w[kAhead ? v : 0] = c < chunks ? *reinterpret_cast<const uint4*>(a.weight + c * 8) : zero;
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    }
    const auto weights = [&](int v) {
        const int c = g.t + v * g.size;
        return kAhead ? w[kAhead ? v : 0] : c < chunks ? *reinterpret_cast<const uint4*>(a.weight + c * 8) : zero;
    };
    int slot = 0;
    for (int64_t row = g.first; row < a.rows; row += g.stride, slot ^= 1) {
        const int64_t base = row * a.k;
        if (!kAhead) fetch(row);
        // the row stays packed; xhat and g are formed again after the sum (cheaper than 16 registers per chunk)
        const float rstd = rstd_next;
        uint4 dy[V], h[V], ds[V];
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dy[v] = dy_next[v];
            h[v] = h_next[v];
            ds[v] = ds_next[v];
            float d[8], x[8], f[8];
            unpack8(dy[v], d);
            unpack8(h[v], x);
            unpack8(weights(v), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = __fmul_rn(x[i], rstd);
                dw[v][i] = __fmaf_rn(d[i], x[i], dw[v][i]);
                dot = __fmaf_rn(__fmul_rn(d[i], f[i]), x[i], dot);
            }
        }
        if (kAhead) fetch(row + g.stride);
        const float mean = g.sum(dot, red, slot) / (float)a.k;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = g.t + v * g.size;
            float d[8], x[8], f[8], add[8];
            unpack8(dy[v], d);
            unpack8(h[v], x);
            unpack8(weights(v), f);
            unpack8(ds[v], add);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] = __fmul_rn(rstd, __fmaf_rn(-__fmul_rn(x[i], rstd), mean, __fmul_rn(d[i], f[i])));
                if (a.dsum) d[i] = __fadd_rn(d[i], add[i]);
            }
            if (c < chunks) st_stream(a.dx + base + c * 8, pack8(d));
        }
    }
    float* out = a.partial + (int64_t)blockIdx.x * a.k;
    if (WARP_ROWS) {
        // the block's warps hold the same columns: joined here, in warp order
        float* mine = joined + (threadIdx.x >> 5) * (V * 256);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) mine[(g.t + v * 32) * 8 + i] = dw[v][i];
        __syncthreads();
        for (int c = (int)threadIdx.x; c < a.k; c += (int)blockDim.x) {
            float sum = joined[c];
#pragma unroll
            for (int i = 1; i < kNormWarps; ++i) sum += joined[i * (V * 256) + c];
            out[c] = sum;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = g.t + v * g.size;
            if (c < chunks) {
                float4* p = reinterpret_cast<float4*>(out + c * 8);
                p[0] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
                p[1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
            }
        }
    }
}

// dweight[c] = sum over b of partial[b][c]: 32 columns per block, warp i takes
// the partial rows i, i + 32, ... and the warps are joined in warp order.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(kJoinWarps * 32)
rmsnorm_join_kernel(const float* __restrict__ partial, int parts, int k, float* __restrict__ dweight) {
    __shared__ float red[kJoinWarps][33];
    const int lane = (int)(threadIdx.x & 31u), warp = (int)(threadIdx.x >> 5);
    const int c = (int)blockIdx.x * 32 + lane;
    dependency_wait();
    allow_dependents();
    float s = 0.0f;
#pragma unroll 4
    for (int b = warp; b < parts; b += kJoinWarps) s += partial[(int64_t)b * k + c];
    red[warp][lane] = s;
    __syncthreads();
    s = warp_sum(red[lane][warp]);          // column `warp` of the block, lane = warp that summed it
    if (lane == 0) dweight[(int64_t)blockIdx.x * 32 + warp] = s;
}

constexpr int kNormMaxK = 16384;          // 512 threads of 4 chunks: what their registers allow

// How a call's rows are shared out (see RowGroup).
struct NormShape {
    bool warp_rows;
    int v;                      // chunks per thread
    int threads;                // of a block
    int groups;                 // row groups per block
};
// Rows of up to 128 chunks (k <= 1024) go to single warps.  Longer ones take a
// block of as many threads as `v` chunks per thread need; with few rows a
// block has one chunk per thread, as latency counts and nothing else runs.
static NormShape norm_shape(int chunks, int64_t rows, int most_v) {
    for (int v = 1; v <= most_v; v *= 2)
        if (chunks <= 32 * v) return {true, v, kNormWarps * 32, kNormWarps};
    const bool few = rows <= 2 * (int64_t)sm_count() && chunks <= 512;
    const int v = few ? 1 : chunks <= 512 * most_v ? most_v : 4;
    const int per = (chunks + v - 1) / v;
    return {false, v, (per + 31) / 32 * 32, 1};
}

// Blocks that are resident on the device at once, for each block size of a kernel.
struct ShapeCache {
    KernelCache by_warps[16];
};
template <class K>
static fp8q_status_t resident_grid(ShapeCache& sc, K kernel, const NormShape& sh, int64_t rows, unsigned* grid) {
    int resident = 0;
    const fp8q_status_t st = prepare_kernel(sc.by_warps[sh.threads / 32 - 1], kernel, sh.threads, 0, 0, &resident);
    if (st != FP8Q_OK) return st;
    *grid = grid_for((size_t)((rows + sh.groups - 1) / sh.groups), resident);
    return FP8Q_OK;
}

}  // namespace fp8q

using namespace fp8q;

namespace fp8q {

template <int OUT, int V, bool WARP_ROWS>
static fp8q_status_t norm_go(const NormShape& sh, const NormArgs& a, cudaStream_t stream) {
    static ShapeCache sc;
    unsigned grid;
    const fp8q_status_t st = resident_grid(sc, rmsnorm_kernel<OUT, V, WARP_ROWS>, sh, a.padded_rows, &grid);
    if (st != FP8Q_OK) return st;
    return launch(rmsnorm_kernel<OUT, V, WARP_ROWS>, grid, (unsigned)sh.threads, 0, stream, a);
}
template <int OUT>
static fp8q_status_t norm_go(const NormShape& sh, const NormArgs& a, cudaStream_t stream) {
    if (sh.warp_rows)
        return sh.v == 1   ? norm_go<OUT, 1, true>(sh, a, stream)
               : sh.v == 2 ? norm_go<OUT, 2, true>(sh, a, stream)
                           : norm_go<OUT, 4, true>(sh, a, stream);
    return sh.v == 1 ? norm_go<OUT, 1, false>(sh, a, stream) : norm_go<OUT, 4, false>(sh, a, stream);
}

static fp8q_status_t norm_launch(int out, const NormArgs& a, size_t scale_bytes, cudaStream_t stream) {
    const size_t n = (size_t)a.rows * (size_t)a.k;
    if (!a.x || !a.weight || !a.codes || !a.scales) return FP8Q_ERR_NULL;
    if (a.sum && !a.residual) return FP8Q_ERR_NULL;
    const void* all[] = {a.x, a.residual, a.weight, a.sum, a.y, a.codes, a.scales, a.rstd};
    for (const void* p : all)
        if (!aligned16(p)) return FP8Q_ERR_ALIGN;
    // the sum may be written over x or over the residual, whole
    const bool over_x = a.sum == a.x, over_r = a.sum == a.residual;
    const Range ins[] = {{a.x, 2 * n}, {a.residual, 2 * n}, {a.weight, 2 * (size_t)a.k}};
    const Range outs[] = {{a.y, 2 * n}, {a.codes, n}, {a.scales, scale_bytes}, {a.rstd, 4 * (size_t)a.rows}};
    if (any_alias(outs, 4, ins, 3)) return FP8Q_ERR_ALIAS;
    if (a.sum) {
        const Range s = {a.sum, 2 * n};
        if ((!over_x && overlaps(s.p, s.bytes, a.x, 2 * n)) || (!over_r && overlaps(s.p, s.bytes, a.residual, 2 * n)) ||
            any_alias(&s, 1, outs, 4) || overlaps(s.p, s.bytes, a.weight, 2 * (size_t)a.k))
            return FP8Q_ERR_ALIAS;
    }
    const NormShape sh = norm_shape(a.k >> 3, a.rows, 4);
    switch (out) {
        case kNormE4M3: return norm_go<kNormE4M3>(sh, a, stream);
        case kNormE5M2: return norm_go<kNormE5M2>(sh, a, stream);
        case kNormMxRows: return norm_go<kNormMxRows>(sh, a, stream);
        default: return norm_go<kNormMxTiled>(sh, a, stream);
    }
}

static fp8q_status_t norm_sizes(int64_t rows, int64_t k, int64_t multiple, float eps) {
    if (rows < 0 || rows >= ((int64_t)1 << 31) - 128) return FP8Q_ERR_SIZE;
    if (k <= 0 || k % multiple != 0 || k > kNormMaxK) return FP8Q_ERR_K;
    if (!(eps >= 0.0f) || !isfinite(eps)) return FP8Q_ERR_SIZE;
    return FP8Q_OK;
}

}  // namespace fp8q

extern "C" fp8q_status_t fp8q_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* weight_bf16,
                                               int64_t rows, int64_t k, float eps, fp8q_format_t fmt, void* sum_bf16,
                                               void* y_bf16, uint8_t* codes, float* scales, float* rstd,
                                               fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_rmsnorm_quantize");
    if (!valid_fmt(fmt)) return FP8Q_ERR_FORMAT;
    const fp8q_status_t st = norm_sizes(rows, k, FP8Q_BLOCK, eps);
    if (st != FP8Q_OK || rows == 0) return st;
    const NormArgs a = {static_cast<const uint16_t*>(x_bf16), static_cast<const uint16_t*>(residual_bf16),
                        static_cast<const uint16_t*>(weight_bf16), static_cast<uint16_t*>(sum_bf16),
                        static_cast<uint16_t*>(y_bf16), codes, scales, rstd, rows, rows, (int)k, eps};
    return norm_launch(fmt == FP8Q_E4M3 ? kNormE4M3 : kNormE5M2, a, (size_t)rows * (size_t)(k / FP8Q_BLOCK) * 4,
                       reinterpret_cast<cudaStream_t>(stream));
}

extern "C" fp8q_status_t mxfp8_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* weight_bf16,
                                                int64_t rows, int64_t k, float eps, int swizzled, void* sum_bf16,
                                                void* y_bf16, uint8_t* codes, uint8_t* scales, float* rstd,
                                                fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("mxfp8_rmsnorm_quantize");
    if (swizzled != 0 && swizzled != 1) return FP8Q_ERR_FLAGS;
    const fp8q_status_t st = norm_sizes(rows, k, MXFP8_BLOCK, eps);
    if (st != FP8Q_OK || rows == 0) return st;
    const NormArgs a = {static_cast<const uint16_t*>(x_bf16), static_cast<const uint16_t*>(residual_bf16),
                        static_cast<const uint16_t*>(weight_bf16), static_cast<uint16_t*>(sum_bf16),
                        static_cast<uint16_t*>(y_bf16), codes, scales, rstd, rows,
                        swizzled ? (rows + 127) / 128 * 128 : rows, (int)k, eps};
    return norm_launch(swizzled ? kNormMxTiled : kNormMxRows, a,
                       swizzled ? mxfp8_swizzled_scale_bytes(1, rows, k) : (size_t)rows * (size_t)(k / MXFP8_BLOCK),
                       reinterpret_cast<cudaStream_t>(stream));
}

namespace fp8q {

using NormGradKernel = void (*)(const NormGradArgs);
static NormGradKernel norm_backward_kernel(const NormShape& sh) {
    if (sh.warp_rows) return sh.v == 1 ? rmsnorm_backward_kernel<1, true> : rmsnorm_backward_kernel<2, true>;
    return sh.v == 1 ? rmsnorm_backward_kernel<1, false> : sh.v == 2 ? rmsnorm_backward_kernel<2, false> : rmsnorm_backward_kernel<4, false>;
}

// The gradient's shape: at most 2 chunks per thread while 512 threads are
// enough (a chunk needs 40 registers there), and no more blocks than are
// resident at once, as each adds a row of partial sums.
static fp8q_status_t norm_backward_shape(int64_t rows, int64_t k, NormShape* sh, unsigned* blocks) {
    static ShapeCache caches[5];
    *sh = norm_shape((int)(k >> 3), rows, 2);
    // a row of partial sums costs 8 bytes per column, a row of the input 6 to 8: at least four rows per group beyond
    // one block per SM
    const int64_t each = (rows + sh->groups - 1) / sh->groups, sms = sm_count();
    int64_t want = (each + 3) / 4;
    if (want < sms) want = each < sms ? each : sms;
    const int which = sh->warp_rows ? sh->v - 1 : sh->v == 1 ? 2 : sh->v == 2 ? 3 : 4;      // as in norm_backward_kernel
    return resident_grid(caches[which], norm_backward_kernel(*sh), *sh, want * sh->groups, blocks);
}

}  // namespace fp8q

extern "C" size_t fp8q_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t k) {
    if (norm_sizes(rows, k, MXFP8_BLOCK, 0.0f) != FP8Q_OK) return 0;
    NormShape sh;
    unsigned blocks = 0;
    if (rows > 0 && norm_backward_shape(rows, k, &sh, &blocks) != FP8Q_OK) return 0;
    return (size_t)blocks * (size_t)k * sizeof(float);
}

extern "C" fp8q_status_t fp8q_rmsnorm_backward(const void* dy_bf16, const void* h_bf16, const void* weight_bf16,
                                               const float* rstd, const void* dsum_bf16, int64_t rows, int64_t k,
                                               void* dx_bf16, float* dweight, void* workspace, size_t workspace_bytes,
                                               fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_rmsnorm_backward");
    const fp8q_status_t st = norm_sizes(rows, k, MXFP8_BLOCK, 0.0f);
    if (st != FP8Q_OK) return st;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const size_t n = (size_t)rows * (size_t)k;
    if (!dweight || (rows > 0 && (!dy_bf16 || !h_bf16 || !weight_bf16 || !rstd || !dx_bf16 || !workspace)))
        return FP8Q_ERR_NULL;
    const size_t need = fp8q_rmsnorm_backward_workspace_bytes(rows, k);
    if (workspace_bytes < need) return FP8Q_ERR_SIZE;
    const void* all[] = {dy_bf16, h_bf16, weight_bf16, rstd, dsum_bf16, dx_bf16, dweight, workspace};
    for (const void* p : all)
        if (!aligned16(p)) return FP8Q_ERR_ALIGN;
    // dx may be written over dy or over dsum, whole
    const Range ins[] = {{h_bf16, 2 * n}, {weight_bf16, 2 * (size_t)k}, {rstd, 4 * (size_t)rows},
                         {dx_bf16 == dy_bf16 ? nullptr : dy_bf16, 2 * n},
                         {dx_bf16 == dsum_bf16 ? nullptr : dsum_bf16, 2 * n}};
    const Range dxr = {dx_bf16, 2 * n};
    if (any_alias(&dxr, 1, ins, 5)) return FP8Q_ERR_ALIAS;
    const Range whole[] = {{h_bf16, 2 * n}, {weight_bf16, 2 * (size_t)k}, {rstd, 4 * (size_t)rows}, {dy_bf16, 2 * n},
                           {dsum_bf16, 2 * n}, {dx_bf16, 2 * n}};
    const Range rest[] = {{dweight, 4 * (size_t)k}, {workspace, need}};
    if (any_alias(rest, 2, whole, 6)) return FP8Q_ERR_ALIAS;
    unsigned blocks = 0;
    if (rows > 0) {
        NormShape sh;
        const fp8q_status_t s0 = norm_backward_shape(rows, k, &sh, &blocks);
        if (s0 != FP8Q_OK) return s0;
        const NormGradArgs a = {static_cast<const uint16_t*>(dy_bf16), static_cast<const uint16_t*>(h_bf16),
                                static_cast<const uint16_t*>(weight_bf16), rstd, static_cast<const uint16_t*>(dsum_bf16),
                                static_cast<uint16_t*>(dx_bf16), static_cast<float*>(workspace), rows, (int)k};
        const fp8q_status_t s1 = launch(norm_backward_kernel(sh), blocks, (unsigned)sh.threads, 0, cs, a);
        if (s1 != FP8Q_OK) return s1;
    }
    return launch(rmsnorm_join_kernel, (unsigned)((k + 31) / 32), kJoinWarps * 32, 0, cs,
                  static_cast<const float*>(workspace), (int)blocks, (int)k, dweight);
}
