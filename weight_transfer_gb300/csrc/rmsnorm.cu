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
// the sum of squares and the output.
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

// Sum over the block's threads, the same value in every thread and the same
// order on every run.  `slot` alternates between two shared arrays so that one
// barrier per call is enough.
__device__ __forceinline__ float block_sum(float v, float (*red)[32], int slot) {
    v = warp_sum(v);
    const int warps = (int)(blockDim.x + 31u) >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31u) == 0) red[slot][threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < warps; ++i) s += red[slot][i];
    return s;
}

// Position of scale column j of row r in the 128x4-tiled layout (`tiles` column tiles).
__device__ __forceinline__ int64_t tiled_scale_at(int64_t r, int j, int tiles) {
    return ((r >> 7) * tiles + (j >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (j & 3);
}

// One row per block; thread t holds the 8-element chunks t, t + B, ... (V of them).
template <int OUT, int V>
__global__ void rmsnorm_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    const int B = (int)blockDim.x;
    const int t = (int)threadIdx.x;
    const int chunks = a.k >> 3;
    const int64_t row = blockIdx.x;
    dependency_wait();
    allow_dependents();
    constexpr bool kMx = OUT == kNormMxRows || OUT == kNormMxTiled;
    const int scale_cols = kMx ? a.k >> 5 : a.k >> 7;
    const int tiles = (scale_cols + 3) >> 2;
    if (OUT == kNormMxTiled) {
        // padding of the tiled layout is zero: whole rows past the last one, and the columns that fill up a tile
        uint8_t* s8 = static_cast<uint8_t*>(a.scales);
        const int first = row < a.rows ? scale_cols : 0;
        for (int j = first + t; j < tiles * 4; j += B) s8[tiled_scale_at(row, j, tiles)] = 0;
        if (row >= a.rows) return;
    }
    const int64_t base = row * a.k;
    float h[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = t + v * B;
        if (c < chunks) {
            unpack8(ld_once(a.x + base + c * 8), h[v]);
            if (a.residual) {
                float r[8];
                unpack8(ld_once(a.residual + base + c * 8), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[v][i] = __fadd_rn(h[v][i], r[i]);
                if (a.sum)
                    st_stream(a.sum + base + c * 8,
                              make_uint4(pack_bf16x2(h[v][0], h[v][1]), pack_bf16x2(h[v][2], h[v][3]),
                                         pack_bf16x2(h[v][4], h[v][5]), pack_bf16x2(h[v][6], h[v][7])));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __fmaf_rn(h[v][i], h[v][i], ss);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] = 0.0f;
        }
    }
    const float mean = block_sum(ss, red, 0) / (float)a.k;
    const float rstd = 1.0f / sqrtf(mean + a.eps);
    if (t == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = t + v * B;
        const bool ok = c < chunks;
        float y[8], w[8];
        unpack8(ok ? *reinterpret_cast<const uint4*>(a.weight + c * 8) : make_uint4(0, 0, 0, 0), w);
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = __fmul_rn(__fmul_rn(h[v][i], rstd), w[i]);
            m = fmaxf(m, fabsf(y[i]));
        }
        if (ok && a.y)
            st_stream(a.y + base + c * 8, make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                     pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])));
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
            block_quotients<2, 8>(y, s, q);
            if (ok && (c & 15) == 0) static_cast<float*>(a.scales)[row * scale_cols + (c >> 4)] = s;
            if (ok)
                st_stream(a.codes + base + c * 8, make_uint2(cvt_fp8x4<FMT>(q[0], q[1], q[2], q[3]),
                                                             cvt_fp8x4<FMT>(q[4], q[5], q[6], q[7])));
        }
    }
}

// ------------------------------------------------------------- gradient ----
//   g = dy * w;  xhat = h * rstd;  dx = rstd * (g - xhat * mean(g * xhat)) + dsum;  dw = sum over rows of dy * xhat
// Blocks walk over the rows with a fixed stride, each thread keeps dw of its
// own columns in registers; the blocks' partial sums are joined in block order
// by a second kernel, so the result does not depend on timing.
struct NormGradArgs {
    const uint16_t* dy;
    const uint16_t* h;
    const uint16_t* weight;
    const float* rstd;
    const uint16_t* dsum;       // or NULL
    uint16_t* dx;
    float* partial;             // [gridDim.x][k]
    int64_t rows;
    int k;
};

template <int V>
__global__ void rmsnorm_backward_kernel(const NormGradArgs a) {
    __shared__ float red[2][32];
    const int B = (int)blockDim.x;
    const int t = (int)threadIdx.x;
    const int chunks = a.k >> 3;
    dependency_wait();
    allow_dependents();
    float dw[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, slot ^= 1) {
        const int64_t base = row * a.k;
        const float rstd = a.rstd[row];
        float g[V][8], xh[V][8];
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = t + v * B;
            if (c < chunks) {
                float dy[8], w[8];
                unpack8(ld_once(a.dy + base + c * 8), dy);
                unpack8(ld_once(a.h + base + c * 8), xh[v]);
                unpack8(*reinterpret_cast<const uint4*>(a.weight + c * 8), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    xh[v][i] = __fmul_rn(xh[v][i], rstd);
                    dw[v][i] = __fmaf_rn(dy[i], xh[v][i], dw[v][i]);
                    g[v][i] = __fmul_rn(dy[i], w[i]);
                    dot = __fmaf_rn(g[v][i], xh[v][i], dot);
                }
            }
        }
        const float mean = block_sum(dot, red, slot) / (float)a.k;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = t + v * B;
            if (c < chunks) {
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = __fmul_rn(rstd, __fmaf_rn(-xh[v][i], mean, g[v][i]));
                if (a.dsum) {
                    float r[8];
                    unpack8(ld_once(a.dsum + base + c * 8), r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] = __fadd_rn(d[i], r[i]);
                }
                st_stream(a.dx + base + c * 8, make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]),
                                                          pack_bf16x2(d[4], d[5]), pack_bf16x2(d[6], d[7])));
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = t + v * B;
        if (c < chunks) {
            float4* p = reinterpret_cast<float4*>(a.partial + (int64_t)blockIdx.x * a.k + c * 8);
            p[0] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
            p[1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
        }
    }
}

// dweight[c] = sum over b of partial[b][c]: 32 columns per block, the warps
// take every 8th partial row and are joined in warp order.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(kJoinWarps * 32)
rmsnorm_join_kernel(const float* __restrict__ partial, int parts, int k, float* __restrict__ dweight) {
    __shared__ float red[kJoinWarps][32];
    const int lane = (int)(threadIdx.x & 31u), warp = (int)(threadIdx.x >> 5);
    const int c = (int)blockIdx.x * 32 + lane;
    dependency_wait();
    allow_dependents();
    float s = 0.0f;
    if (c < k)
        for (int b = warp; b < parts; b += kJoinWarps) s += partial[(int64_t)b * k + c];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < k) {
        s = red[0][lane];
#pragma unroll
        for (int i = 1; i < kJoinWarps; ++i) s += red[i][lane];
        dweight[c] = s;
    }
}

constexpr int kNormMaxK = 16384;          // 512 threads of 4 chunks: what their registers allow

// Threads and chunks per thread for a row of `chunks` 8-element chunks.
static void norm_shape(int chunks, int* threads, int* v) {
    *v = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : 4;
    const int t = (chunks + *v - 1) / *v;
    *threads = (t + 31) / 32 * 32;
}

}  // namespace fp8q

using namespace fp8q;

namespace fp8q {

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
    int threads, v;
    norm_shape(a.k >> 3, &threads, &v);
    const unsigned grid = (unsigned)a.padded_rows;
    auto go = [&](auto k1, auto k2, auto k4) {
        return launch(v == 1 ? k1 : v == 2 ? k2 : k4, grid, (unsigned)threads, 0, stream, a);
    };
    switch (out) {
        case kNormE4M3: return go(rmsnorm_kernel<kNormE4M3, 1>, rmsnorm_kernel<kNormE4M3, 2>, rmsnorm_kernel<kNormE4M3, 4>);
        case kNormE5M2: return go(rmsnorm_kernel<kNormE5M2, 1>, rmsnorm_kernel<kNormE5M2, 2>, rmsnorm_kernel<kNormE5M2, 4>);
        case kNormMxRows: return go(rmsnorm_kernel<kNormMxRows, 1>, rmsnorm_kernel<kNormMxRows, 2>, rmsnorm_kernel<kNormMxRows, 4>);
        default: return go(rmsnorm_kernel<kNormMxTiled, 1>, rmsnorm_kernel<kNormMxTiled, 2>, rmsnorm_kernel<kNormMxTiled, 4>);
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

// Blocks of the gradient kernel, and so rows of its workspace.
static int64_t norm_backward_blocks(int64_t rows) {
    const int64_t most = (int64_t)sm_count() * 4;
    return rows < most ? rows : most;
}

extern "C" size_t fp8q_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t k) {
    if (norm_sizes(rows, k, MXFP8_BLOCK, 0.0f) != FP8Q_OK) return 0;
    return (size_t)norm_backward_blocks(rows) * (size_t)k * sizeof(float);
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
    const int parts = (int)norm_backward_blocks(rows);
    if (rows > 0) {
        const NormGradArgs a = {static_cast<const uint16_t*>(dy_bf16), static_cast<const uint16_t*>(h_bf16),
                                static_cast<const uint16_t*>(weight_bf16), rstd, static_cast<const uint16_t*>(dsum_bf16),
                                static_cast<uint16_t*>(dx_bf16), static_cast<float*>(workspace), rows, (int)k};
        int threads, v;
        norm_shape((int)(k >> 3), &threads, &v);
        const fp8q_status_t s1 = launch(v == 1   ? rmsnorm_backward_kernel<1>
                                        : v == 2 ? rmsnorm_backward_kernel<2>
                                                 : rmsnorm_backward_kernel<4>,
                                        (unsigned)parts, (unsigned)threads, 0, cs, a);
        if (s1 != FP8Q_OK) return s1;
    }
    return launch(rmsnorm_join_kernel, (unsigned)((k + 31) / 32), kJoinWarps * 32, 0, cs,
                  static_cast<const float*>(workspace), parts, (int)k, dweight);
}
