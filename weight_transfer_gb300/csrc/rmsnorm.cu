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
// With several outputs the work is bound by HBM: a row is read once and stays
// in registers between the sum of squares and the output, and the next row is
// read meanwhile (one row per block without that took 110.6 us where this takes
// 100.4: 16,384 rows of 4096 with residual, MXFP8 and bf16 outputs; 96.7 back to
// back, 92% of the measured copy rate).  With codes alone it is bound by the
// latency of its arithmetic, 12 (MXFP8) to 15 (e4m3) instructions per element:
// the 15 warps an SM has registers for issue in 59 to 64% of the cycles and wait
// for earlier instructions and shuffles, hardly ever for memory.  Hence the
// packed arithmetic on pairs, scales worked out once for each block and lane,
// and a form without residual (16,384 x 4096, one call at a time, MXFP8 alone:
// 47.1 us without these, 41.0 with; e4m3 65.5 and 49.2, exact quotients
// included).  Few rows are bound by latency, and below about 20 us by the
// caller's launches.
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
    float inv_k;                // RN(1 / k)
    int lanes;                  // see RowGroup
};

constexpr int kNormWarps = 4;   // warps of a block whose warps have rows of their own

// How the threads of a block share the rows: groups of 4 to 32 lanes with a
// row each (short rows, no barrier at all), or the whole block per row.  Blocks
// walk over the rows with a fixed stride; the weights stay in registers and the
// next row is on its way while this one is summed up and written.  A thread
// holds the 8-element chunks c0 + 32 v, v < V, of its row: fixed distances, so
// that all V accesses share one address.
enum NormGroup { kByBlock = 0, kByWarp = 1, kByLanes = 2 };
template <int V, int GROUP> struct RowGroup {
    static constexpr bool WARP_ROWS = GROUP != kByBlock;
    static_assert(GROUP != kByLanes || V == 1, "parts of a warp hold one chunk per lane");
    int lanes;                  // of a group inside one warp
    int t, size;                // thread inside the group, threads of the group
    int c0;
    int64_t first, stride;      // first row of this warp (the same in all its lanes), rows of all groups together
    int64_t at;                 // this group's place behind the warp's row
    __device__ __forceinline__ explicit RowGroup(int group_lanes) {
        const int lane = (int)(threadIdx.x & 31u), warp = (int)(threadIdx.x >> 5);
        lanes = GROUP == kByLanes ? group_lanes : 32;
        if (WARP_ROWS) {
            const int per_warp = 32 / lanes, per_block = (int)(blockDim.x >> 5) * per_warp;
            t = c0 = lane & (lanes - 1);
            size = lanes;
            first = (int64_t)blockIdx.x * per_block + warp * per_warp;
            stride = (int64_t)gridDim.x * per_block;
            at = lane / lanes;
        } else {
            t = (int)threadIdx.x;
            c0 = warp * (32 * V) + lane;
            size = (int)blockDim.x;
            first = blockIdx.x;
            stride = gridDim.x;
            at = 0;
        }
    }
    // Sum over the group, the same value in every thread and the same order on
    // every run.  `slot` alternates between two shared arrays, so that one
    // barrier per row is enough.
    __device__ __forceinline__ float sum(float v, float (*red)[32], int slot) const {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1)
            if (GROUP != kByLanes || m < lanes) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
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

// Eight bf16 as four pairs of binary32, and back (rounded).
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
    float a, b;
    f2_unpack(v, a, b);
    return pack_bf16x2(a, b);
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}

// One step of a maximum over lanes that hold N values each: the lanes at
// distance MASK share the values out, half each, so that a lane is left with
// the values whose index has its own bit.
template <int MASK, int N>
__device__ __forceinline__ void share_max(float (&m)[N / 2], const float (&all)[N], int lane) {
    const bool odd = (lane & MASK) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? all[2 * i] : all[2 * i + 1], MASK);
        m[i] = fmaxf(odd ? all[2 * i + 1] : all[2 * i], got);
    }
}

template <int OUT, int V, int GROUP, bool RES>
__global__ void __launch_bounds__(512) rmsnorm_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    const RowGroup<V, GROUP> g(a.lanes);
    const int lane = (int)(threadIdx.x & 31u);
    const int chunks = a.k >> 3;
    constexpr bool kMx = OUT == kNormMxRows || OUT == kNormMxTiled;
    const int scale_cols = kMx ? a.k >> 5 : a.k >> 7;
    const int tiles = (scale_cols + 3) >> 2;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    dependency_wait();
    allow_dependents();
    uint4 w[V], x[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = r[v] = zero;     // and zero they stay behind the row's end
    auto fetch = [&](int64_t row) {
        const int64_t base = row * a.k + g.c0 * 8;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (row < a.rows && g.c0 + v * 32 < chunks) {
                x[v] = ld_once(a.x + base + v * 256);
                if (RES) r[v] = ld_once(a.residual + base + v * 256);
            }
    };
    fetch(g.first + g.at);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = g.c0 + v * 32;
        w[v] = c < chunks ? *reinterpret_cast<const uint4*>(a.weight + c * 8) : zero;
    }
    int slot = 0;
    // the lanes of a warp stay together, whichever of their rows are there
    for (int64_t row0 = g.first; row0 < a.padded_rows; row0 += g.stride, slot ^= 1) {
        const int64_t row = row0 + g.at;
        const bool live = row < a.rows;
        if (OUT == kNormMxTiled && row < a.padded_rows) {
            // padding of the tiled layout is zero: whole rows past the last one, and the columns that fill up a tile
            uint8_t* s8 = static_cast<uint8_t*>(a.scales);
            const int first = live ? scale_cols : 0;
            for (int j = first + g.t; j < tiles * 4; j += g.size) s8[tiled_scale_at(row, j, tiles)] = 0;
        }
        const int64_t base = row * a.k + g.c0 * 8;
        uint64_t h[V][4], ss = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            unpack8(x[v], h[v]);
            if (RES) {
                uint64_t f[4];
                unpack8(r[v], f);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[v][i] = f2_add(h[v][i], f[i]);
                if (a.sum && live && g.c0 + v * 32 < chunks) st_stream(a.sum + base + v * 256, pack8(h[v]));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = f2_fma(h[v][i], h[v][i], ss);
        }
        fetch(row + g.stride);
        float even, odd;
        f2_unpack(ss, even, odd);
        const float mean = __fmul_rn(g.sum(even + odd, red, slot), a.inv_k);
        const float rstd = __frsqrt_rn(mean + a.eps);
        if (g.t == 0 && a.rstd && live) a.rstd[row] = rstd;
        // h becomes y, or -y for the blockwise quotients, which then need no other negation
        const uint64_t rstd2 = kMx ? f2_pack(rstd, rstd) : f2_pack(-rstd, -rstd);
        float m[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint64_t f[4];
            unpack8(w[v], f);
            m[v] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[v][i] = f2_mul(f2_mul(h[v][i], rstd2), f[i]);
                float y0, y1;
                f2_unpack(h[v][i], y0, y1);
                m[v] = fmaxf(m[v], fmaxf(fabsf(y0), fabsf(y1)));
            }
            if (a.y && live && g.c0 + v * 32 < chunks) {
                uint4 y = pack8(h[v]);
                if (!kMx) y = make_uint4(y.x ^ 0x80008000u, y.y ^ 0x80008000u, y.z ^ 0x80008000u, y.w ^ 0x80008000u);
                st_stream(a.y + base + v * 256, y);
            }
        }
        uint8_t* codes = a.codes + base;
        const auto put = [&](int v, const float (&q)[8]) {
            constexpr int FMT = OUT == kNormE5M2 ? kE5M2 : kE4M3;
            if (live && g.c0 + v * 32 < chunks)
                st_stream(codes + v * 256, make_uint2(cvt_fp8x4<FMT>(q[0], q[1], q[2], q[3]),
                                                      cvt_fp8x4<FMT>(q[4], q[5], q[6], q[7])));
        };
        const auto put_scaled = [&](int v, float factor) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_unpack(f2_mul(h[v][i], f2_pack(factor, factor)), q[2 * i], q[2 * i + 1]);
            put(v, q);
        };
        if (kMx) {
            // the scale needs the exponent of the four lanes' largest magnitude only: two chunks' exponents per word
            uint32_t ex[(V + 1) / 2];
#pragma unroll
            for (int i = 0; i < (V + 1) / 2; ++i) {
                ex[i] = __float_as_uint(m[2 * i]) >> 23;
                if (2 * i + 1 < V) ex[i] |= __float_as_uint(m[2 * i + (V > 1)]) >> 23 << 16;
                ex[i] = __vmaxu2(ex[i], __shfl_xor_sync(0xFFFFFFFFu, ex[i], 1));
                ex[i] = __vmaxu2(ex[i], __shfl_xor_sync(0xFFFFFFFFu, ex[i], 2));
            }
            const int j = g.c0 >> 2;            // chunk v's scale is column j + 8 v
            uint8_t* s8 = static_cast<uint8_t*>(a.scales) +
                          (OUT == kNormMxRows ? row * scale_cols + j : tiled_scale_at(row, j, tiles));
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int E = (int)(v & 1 ? ex[v / 2] >> 16 : ex[v / 2] & 0xFFFFu);
                const int e8 = E > 8 ? E - 8 : 0;
                if (live && (lane & 3) == 0 && g.c0 + v * 32 < chunks) s8[v * (OUT == kNormMxRows ? 8 : 1024)] = (uint8_t)e8;
                put_scaled(v, __uint_as_float((uint32_t)(254 - e8) << 23));
            }
        } else {
            // sixteen lanes have a block of each of their V chunks; lane i works out the scale of chunk i mod V
            float top;
            if constexpr (V == 4) {
                float two[2], one[1];
                share_max<1>(two, m, lane);
                share_max<2>(one, two, lane);
                top = one[0];
            } else if constexpr (V == 2) {
                float one[1];
                share_max<1>(one, m, lane);
                top = fmaxf(one[0], __shfl_xor_sync(0xFFFFFFFFu, one[0], 2));
            } else {
                top = fmaxf(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
            constexpr int FMT = OUT == kNormE5M2 ? kE5M2 : kE4M3;
            const float s = block_scale<FMT>(top);
            const int own = lane & 15, c = g.c0 - own + own * 32;
            if (live && own < V && c < chunks) static_cast<float*>(a.scales)[row * scale_cols + (c >> 4)] = s;
            // The code of the correctly rounded quotient y / s by one step of markstein_div in packed form, h holding
            // -y.  For a binary32 y one step rounds a value within 2^-21 half-ulps of y / s, which can show in a code
            // only beside a value between two codes; all such y and s are tried in tests/test_norm_quotient.py.
            // y * RN(1 / s) alone misses ties (16,384 x 4096, e4m3 alone, back to back: 41.5 us without the step, 44.7
            // with it, 48.1 with a second one; with residual 73.5 and 73.7).  An all-zero block keeps its zeros,
            // divided by 1.
            const float by = s == 0.0f ? 1.0f : s, inv = __frcp_rn(by);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float sv = V == 1 ? by : __shfl_sync(0xFFFFFFFFu, by, (lane & 16) | v);
                const float yr = V == 1 ? inv : __shfl_sync(0xFFFFFFFFu, inv, (lane & 16) | v);
                float q[8];
                if (sv >= 0x1p-58f) {
                    const uint64_t s2 = f2_pack(sv, sv), nyr2 = f2_pack(-yr, -yr);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint64_t q2 = f2_mul(h[v][i], nyr2);
                        q2 = f2_fma(f2_fma(q2, s2, h[v][i]), nyr2, q2);
                        f2_unpack(q2, q[2 * i], q[2 * i + 1]);
                    }
                } else {                        // too small for the steps (see block_quotients), or NaN
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f2_unpack(h[v][i], y[2 * i], y[2 * i + 1]);
                        y[2 * i] = -y[2 * i];
                        y[2 * i + 1] = -y[2 * i + 1];
                    }
                    block_quotients<2, 8>(y, sv, q);
                }
                put(v, q);
            }
        }
    }
}

// ------------------------------------------------------------- gradient ----
//   g = dy * w;  xhat = h * rstd;  dx = rstd * (g - xhat * mean(g * xhat)) + dsum;  dw = sum over rows of dy * xhat
// 16,384 rows of 4096 with dsum take 84.5 us back to back (6.4 TB/s, 94% of the
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
    float inv_k;                // RN(1 / k)
    int lanes;                  // see RowGroup
};

template <int V, int GROUP, bool RES>
__global__ void __launch_bounds__(512) rmsnorm_backward_kernel(const NormGradArgs a) {
    // four chunks per thread leave no registers for the next row, nor for the weights, which come from the first-level
    // cache again (4096 x 16384 with dsum: 88 us; with the next row on its way the registers spill, 117)
    constexpr bool kAhead = V < 4;
    __shared__ float red[2][32];
    constexpr bool WARP_ROWS = GROUP != kByBlock;
    __shared__ float joined[WARP_ROWS ? kNormWarps * V * 256 : 1];
    const RowGroup<V, GROUP> g(a.lanes);
    const int chunks = a.k >> 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    dependency_wait();
    allow_dependents();
    uint4 w[kAhead ? V : 1], dy_next[V], h_next[V], ds_next[V];
    float rstd_next = 0.0f;
    auto fetch = [&](int64_t row) {
        const int64_t base = row * a.k + g.c0 * 8;
        rstd_next = row < a.rows ? a.rstd[row] : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (row < a.rows && g.c0 + v * 32 < chunks) {
                dy_next[v] = ld_once(a.dy + base + v * 256);
                h_next[v] = ld_once(a.h + base + v * 256);
                if (RES) ds_next[v] = ld_once(a.dsum + base + v * 256);
            } else if (GROUP == kByLanes || !kAhead) {      // (a lane that goes on without a row adds zeros to dw)
                dy_next[v] = h_next[v] = ds_next[v] = zero;
            }
        }
    };
    if (kAhead)
#pragma unroll
        for (int v = 0; v < V; ++v) dy_next[v] = h_next[v] = ds_next[v] = zero;
    if (kAhead) fetch(g.first + g.at);
    const auto weight = [&](int v) {
        const int c = g.c0 + v * 32;
        return c < chunks ? *reinterpret_cast<const uint4*>(a.weight + c * 8) : zero;
    };
    uint64_t dw[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (kAhead) w[kAhead ? v : 0] = weight(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[v][i] = 0;
    }
    const auto weights = [&](int v) { return kAhead ? w[kAhead ? v : 0] : weight(v); };
    int slot = 0;
    for (int64_t row0 = g.first; row0 < a.rows; row0 += g.stride, slot ^= 1) {
        const int64_t row = row0 + g.at;
        if (!kAhead) fetch(row);
        // the row stays packed; xhat and g are formed again after the sum (cheaper than 16 registers per chunk)
        const uint64_t rstd = f2_pack(rstd_next, rstd_next);
        uint4 dy[V], h[V], ds[V];
        uint64_t dot = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dy[v] = dy_next[v];
            h[v] = h_next[v];
            ds[v] = ds_next[v];
            uint64_t d[4], x[4], f[4];
            unpack8(dy[v], d);
            unpack8(h[v], x);
            unpack8(weights(v), f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = f2_mul(x[i], rstd);
                dw[v][i] = f2_fma(d[i], x[i], dw[v][i]);
                dot = f2_fma(f2_mul(d[i], f[i]), x[i], dot);
            }
        }
        if (kAhead) fetch(row + g.stride);
        float even, odd;
        f2_unpack(dot, even, odd);
        const float mean = __fmul_rn(g.sum(even + odd, red, slot), a.inv_k);
        const uint64_t less = f2_pack(-mean, -mean);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint64_t d[4], x[4], f[4], add[4];
            unpack8(dy[v], d);
            unpack8(h[v], x);
            unpack8(weights(v), f);
            unpack8(ds[v], add);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d[i] = f2_mul(rstd, f2_fma(f2_mul(x[i], rstd), less, f2_mul(d[i], f[i])));
                if (RES) d[i] = f2_add(d[i], add[i]);
            }
            if (row < a.rows && g.c0 + v * 32 < chunks) st_stream(a.dx + row * a.k + g.c0 * 8 + v * 256, pack8(d));
        }
    }
    float* out = a.partial + (int64_t)blockIdx.x * a.k;
    if (WARP_ROWS) {
        // the block's groups hold the same columns: joined here, in their order
        float* mine = joined + (int)(threadIdx.x - g.t) / g.lanes * (g.lanes * V * 8);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f2_unpack(dw[v][i], mine[(g.t + v * 32) * 8 + 2 * i], mine[(g.t + v * 32) * 8 + 2 * i + 1]);
        __syncthreads();
        for (int c = (int)threadIdx.x; c < a.k; c += (int)blockDim.x) {
            float sum = joined[c];
            for (int i = g.lanes * V * 8 + c; i < kNormWarps * V * 256; i += g.lanes * V * 8) sum += joined[i];
            out[c] = sum;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = g.c0 + v * 32;
            if (c < chunks) {
                float p[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) f2_unpack(dw[v][i], p[2 * i], p[2 * i + 1]);
                float4* o = reinterpret_cast<float4*>(out + c * 8);
                o[0] = make_float4(p[0], p[1], p[2], p[3]);
                o[1] = make_float4(p[4], p[5], p[6], p[7]);
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
    s = red[lane][warp];                    // column `warp` of the block, lane = warp that summed it
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
    if (lane == 0) dweight[(int64_t)blockIdx.x * 32 + warp] = s;
}

constexpr int kNormMaxK = 16384;          // 512 threads of 4 chunks: what their registers allow

// How a call's rows are shared out (see RowGroup).
struct NormShape {
    NormGroup group;
    int v;                      // chunks per thread
    int threads;                // of a block
    int lanes;                  // of a group inside one warp
    int groups;                 // row groups per block
};
// Rows of up to 16 chunks go to groups of as few lanes as hold them (200,000
// rows of 128, e4m3: 28.7 us; a warp each 55.4), rows of up to 128 chunks
// (k <= 1024) to single warps.  Longer ones take a block of as many threads as
// `v` chunks per thread need; with few rows a block has one chunk per thread, as
// latency counts and nothing else runs (us from a graph, one chunk and four:
// 4 x 2048 1.5 and 1.8, 304 x 2048 1.8 and 2.0, 304 x 4096 2.4 and 2.4,
// 450 x 4096 3.8 and 3.1).
static NormShape norm_shape(int chunks, int64_t rows, int most_v) {
    int lanes = 4;
    while (lanes < 32 && lanes < chunks) lanes *= 2;
    for (int v = 1; v <= most_v; v *= 2)
        if (chunks <= 32 * v) return {lanes < 32 ? kByLanes : kByWarp, v, kNormWarps * 32, lanes, kNormWarps * 32 / lanes};
    const bool few = rows <= 2 * (int64_t)sm_count() && chunks <= 512;
    const int v = few ? 1 : chunks <= 512 * most_v ? most_v : 4;
    const int per = (chunks + v - 1) / v;
    return {kByBlock, v, (per + 31) / 32 * 32, 32, 1};
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

template <int OUT, int V, int GROUP>
static fp8q_status_t norm_go(const NormShape& sh, const NormArgs& a, cudaStream_t stream) {
    static ShapeCache caches[2];
    ShapeCache& sc = caches[a.residual != nullptr];
    const auto kernel = a.residual ? rmsnorm_kernel<OUT, V, GROUP, true> : rmsnorm_kernel<OUT, V, GROUP, false>;
    unsigned grid;
    const fp8q_status_t st = resident_grid(sc, kernel, sh, a.padded_rows, &grid);
    if (st != FP8Q_OK) return st;
    return launch(kernel, grid, (unsigned)sh.threads, 0, stream, a);
}
template <int OUT>
static fp8q_status_t norm_go(const NormShape& sh, const NormArgs& a, cudaStream_t stream) {
    if (sh.group == kByLanes) return norm_go<OUT, 1, kByLanes>(sh, a, stream);
    if (sh.group == kByWarp)
        return sh.v == 1   ? norm_go<OUT, 1, kByWarp>(sh, a, stream)
               : sh.v == 2 ? norm_go<OUT, 2, kByWarp>(sh, a, stream)
                           : norm_go<OUT, 4, kByWarp>(sh, a, stream);
    return sh.v == 1 ? norm_go<OUT, 1, kByBlock>(sh, a, stream) : norm_go<OUT, 4, kByBlock>(sh, a, stream);
}

static fp8q_status_t norm_launch(int out, NormArgs a, size_t scale_bytes, cudaStream_t stream) {
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
    a.inv_k = 1.0f / (float)a.k;
    a.lanes = sh.lanes;
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
                        static_cast<uint16_t*>(y_bf16), codes, scales, rstd, rows, rows, (int)k, eps, 0.0f, 0};
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
                        swizzled ? (rows + 127) / 128 * 128 : rows, (int)k, eps, 0.0f, 0};
    return norm_launch(swizzled ? kNormMxTiled : kNormMxRows, a,
                       swizzled ? mxfp8_swizzled_scale_bytes(1, rows, k) : (size_t)rows * (size_t)(k / MXFP8_BLOCK),
                       reinterpret_cast<cudaStream_t>(stream));
}

namespace fp8q {

using NormGradKernel = void (*)(const NormGradArgs);
template <bool RES> static NormGradKernel norm_backward_kernel(int which) {
    switch (which) {
        case 0: return rmsnorm_backward_kernel<1, kByLanes, RES>;
        case 1: return rmsnorm_backward_kernel<1, kByWarp, RES>;
        case 2: return rmsnorm_backward_kernel<2, kByWarp, RES>;
        case 3: return rmsnorm_backward_kernel<1, kByBlock, RES>;
        case 4: return rmsnorm_backward_kernel<2, kByBlock, RES>;
        default: return rmsnorm_backward_kernel<4, kByBlock, RES>;
    }
}

// The gradient's shape: at most 2 chunks per thread while 512 threads are
// enough (a chunk needs 40 registers there), and no more blocks than are
// resident at once, as each adds a row of partial sums.
static fp8q_status_t norm_backward_shape(int64_t rows, int64_t k, NormShape* sh, int* which, unsigned* blocks) {
    static ShapeCache caches[6];
    *sh = norm_shape((int)(k >> 3), rows, 2);
    // a row of partial sums costs 8 bytes per column, a row of the input 6 to 8: at least four rows per group beyond
    // one block per SM
    const int64_t each = (rows + sh->groups - 1) / sh->groups, sms = sm_count();
    int64_t want = (each + 3) / 4;
    if (want < sms) want = each < sms ? each : sms;
    *which = sh->group == kByLanes ? 0 : sh->group == kByWarp ? sh->v : sh->v == 4 ? 5 : 2 + sh->v;
    // one workspace size for both forms: the blocks of the larger, with dsum
    return resident_grid(caches[*which], norm_backward_kernel<true>(*which), *sh, want * sh->groups, blocks);
}

}  // namespace fp8q

extern "C" size_t fp8q_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t k) {
    if (norm_sizes(rows, k, MXFP8_BLOCK, 0.0f) != FP8Q_OK) return 0;
    NormShape sh;
    int which;
    unsigned blocks = 0;
    if (rows > 0 && norm_backward_shape(rows, k, &sh, &which, &blocks) != FP8Q_OK) return 0;
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
        int which;
        const fp8q_status_t s0 = norm_backward_shape(rows, k, &sh, &which, &blocks);
        if (s0 != FP8Q_OK) return s0;
        const NormGradArgs a = {static_cast<const uint16_t*>(dy_bf16), static_cast<const uint16_t*>(h_bf16),
                                static_cast<const uint16_t*>(weight_bf16), rstd, static_cast<const uint16_t*>(dsum_bf16),
                                static_cast<uint16_t*>(dx_bf16), static_cast<float*>(workspace), rows, (int)k, 1.0f / (float)k, sh.lanes};
        const fp8q_status_t s1 = launch(dsum_bf16 ? norm_backward_kernel<true>(which) : norm_backward_kernel<false>(which), blocks, (unsigned)sh.threads, 0, cs, a);
        if (s1 != FP8Q_OK) return s1;
    }
    return launch(rmsnorm_join_kernel, (unsigned)((k + 31) / 32), kJoinWarps * 32, 0, cs,
                  static_cast<const float*>(workspace), (int)blocks, (int)k, dweight);
}
