// The experts' products with MXFP8 weights, on the tensor cores.
//
// Rows of activations are sorted by expert (expert e owns rows offsets[e] ..
// offsets[e + 1]); expert e's weights are a row-major [n, k] matrix, codes and
// swizzled scales as mxfp8_quantize_swizzled writes them for a batch of
// experts.  With a = sum over blocks of 32 of 2^(s - 127) * code on both sides
//     matmul   out[r, f]  = sum over k of W[e(r), f, k] * a[r, k]
//     swiglu   g, u the same products with two weight tensors,
//              h[r, f] = g / (1 + exp(-g)) * u, quantized to MXFP8 rows
// Products of 8-bit codes and their scales are exact, sums are binary32 in the
// tensor core's accumulators.
//
// The weights are the M side of the product (128 features a tile) and the
// rows its N side (16 .. 224 a tile, as many as the expert has): an expert
// with one row costs a 16-wide product, not a 128-wide one, and each feature
// is a TMEM lane, so that a block of 32 features is one warp and its largest
// magnitude one warp reduction.
//
// One CTA per SM walks over the tiles.  Warp 0 copies weights, rows and
// weight scales by TMA, warp 2 brings the rows' scales into the tensor core's
// tile order (rows of an expert start anywhere, so their scales cannot lie
// pre-tiled), warp 1 issues the products, warps 4 to 11 read the accumulators
// of one tile while the products of the next fill the other half of TMEM (two
// warps for each quarter of the lanes, every other 16 rows each).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp8q_host.cuh"
#include "tcgen05.cuh"

namespace fp8q {

constexpr int kMpReaders = 8;                   // warps that read the accumulators
constexpr int kMpThreads = 128 + 32 * kMpReaders;
constexpr int kMpStages = 4;
constexpr int kMpMaxExperts = 1024;
constexpr int kMpRowBoxes = 4;                  // row boxes of 128, 64, 32 and 16 rows
constexpr uint32_t kMpTmemColumns = 512;
constexpr uint32_t kMpAccColumns = 224;         // per accumulator half
constexpr uint32_t kMpScaleColumns = 448;       // scales: 12 columns per stage from here
constexpr unsigned kErrProductTimeout = 2u;

// WT weight tensors (1: matmul, 2: gate and up), up to kRows rows per tile.
template <int WT> struct MpShape {
    static constexpr int kRows = WT == 1 ? 224 : 112;
    static constexpr int kStageBytes = WT * 16384 + kRows * 128;
    static constexpr int kScaleBytes = WT * 512 + 1024;
    static constexpr int kBars = 2 * kMpStages + 4;
    static constexpr int kOutBytes = WT == 1 ? kMpReaders * 2048 : 0;    // two 16-row staging areas per reading warp
    static constexpr size_t kSmem = (size_t)kMpStages * (kStageBytes + kScaleBytes) + kOutBytes + kBars * 8 + 16 +
                                    2 * (kMpMaxExperts + 2) * 4 + 1024;
};

struct MpArgs {
    CUtensorMap w[2];                           // [experts][n][k] codes, 128 x 128 boxes
    CUtensorMap rows[kMpRowBoxes];              // [rows][k] codes
    const uint8_t* w_scales[2];
    const uint8_t* row_scales;                  // [rows][k / 32]
    const int* offsets;
    uint16_t* out_bf16;                         // matmul
    uint8_t* out_codes;                         // swiglu
    uint8_t* out_scales;
    int rows_total;
    int experts, n, k;
    int feature_tiles, k_steps;                 // ceil(n / 128), ceil(k / 128)
};

// The tiles of one CTA, in the order in which every warp of it walks over
// them.  Both tables are in shared memory: row_start[e] is the first row of
// expert e (row_start[experts] the first row of no expert, row_start[experts +
// 1] = rows), prefix[e] the number of row tiles before it.
struct MpTiles {
    const int* prefix;
    const int* row_start;
    int experts, feature_tiles;
    int step_rt, step_f;                        // one grid further
    int rt, ft;                                 // row tile and feature tile
    int e, end;                                 // expert (`experts`: rows of none, written as zeros), its last row tile + 1
    int per;                                    // rows of its full tiles
    int r0, rows;                               // first row and number of rows of the tile

    __device__ __forceinline__ MpTiles(const MpArgs& a, const int* prefix_, const int* row_start_)
        : prefix(prefix_), row_start(row_start_), experts(a.experts), feature_tiles(a.feature_tiles) {
        rt = (int)blockIdx.x / feature_tiles;
        ft = (int)blockIdx.x - rt * feature_tiles;
        step_rt = (int)gridDim.x / feature_tiles;
        step_f = (int)gridDim.x - step_rt * feature_tiles;
        e = -1;
        end = 0;
    }
    // Resolves the current tile; false if there is none left.
    __device__ __forceinline__ bool here() {
        if (rt >= prefix[experts + 1]) return false;
        if (rt >= end) {
            int lo = e + 1, hi = experts;       // the last expert with prefix[.] <= rt
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (prefix[mid] <= rt) lo = mid; else hi = mid - 1;
            }
            e = lo;
            end = prefix[e + 1];
            const int tiles = end - prefix[e];
            // equal tiles, in steps of 16 rows: fewer, fuller columns than full tiles and a rest
            per = ((row_start[e + 1] - row_start[e] + tiles - 1) / tiles + 15) & ~15;
        }
        r0 = row_start[e] + (rt - prefix[e]) * per;
        const int left = row_start[e + 1] - r0;
        rows = left < per ? left : per;
        return true;
    }
    __device__ __forceinline__ void next() {
        rt += step_rt;
        ft += step_f;
        if (ft >= feature_tiles) {
            ft -= feature_tiles;
            ++rt;
        }
    }
    __device__ __forceinline__ bool none() const { return e >= experts; }
};

// The four E8M0 bytes of one row for K step kb (128 columns); bytes past k are 0.
__device__ __forceinline__ uint32_t row_scale_word(const uint8_t* row, int kb, int cols) {
    uint32_t w = 0;
    for (int j = 0; j < 4; ++j)
        if (kb * 4 + j < cols) w |= (uint32_t)row[kb * 4 + j] << (8 * j);
    return w;
}

// Byte of 16-byte chunk `chunk` (8 features) of row r in a reading warp's
// 16 x 64-byte staging area; the exclusive or spreads 8 rows over all banks.
__device__ __forceinline__ int out_stage_at(int r, int chunk) { return r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4); }

// g / (1 + exp(-g)) * u.  The reciprocal is the hardware's (1 ulp, with
// subnormal results); the result is about to be rounded to 8 bits.
__device__ __forceinline__ float silu_times(float g, float u) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, expf(-g))));
    return __fmul_rn(__fmul_rn(g, r), u);
}

// One step of the 4 x 4 byte transpose of the words x and y over four lanes:
// with the lane at distance `mask`, a lane exchanges the bytes whose index
// differs from its own in bit BIT (0: odd and even bytes, 1: halves).  Each
// word gives away two bytes, so that one shuffle serves both words.
template <int BIT>
__device__ __forceinline__ void transpose_step(uint32_t& x, uint32_t& y, int mask, bool upper) {
    const uint32_t send = BIT == 0 ? __byte_perm(x, y, upper ? 0x6420u : 0x7531u) : __byte_perm(x, y, upper ? 0x5410u : 0x7632u);
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, send, mask);      // two bytes for x, two for y
    if (BIT == 0) {
        x = __byte_perm(x, got, upper ? 0x3514u : 0x5240u);
        y = __byte_perm(y, got, upper ? 0x3716u : 0x7260u);
    } else {
        x = __byte_perm(x, got, upper ? 0x3254u : 0x5410u);
        y = __byte_perm(y, got, upper ? 0x3276u : 0x7610u);
    }
}

__device__ __forceinline__ bool mp_wait(uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity)) return true;
    raise_error(kErrProductTimeout);
    return false;
}

template <int WT>
__global__ void __launch_bounds__(kMpThreads, 1) moe_product_kernel(const __grid_constant__ MpArgs a) {
    using S = MpShape<WT>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* sscale = smem + kMpStages * S::kStageBytes;
    uint8_t* sout = sscale + kMpStages * S::kScaleBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(sout + S::kOutBytes);
    uint64_t* empty = full + kMpStages;
    uint64_t* acc_full = empty + kMpStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    int* prefix = reinterpret_cast<int*>(tmem_slot + 4);
    int* row_start = prefix + kMpMaxExperts + 2;
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < kMpStages; ++s) {
            mbar_init(&full[s], 33);            // the copying thread and the scale warp's lanes
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kMpReaders);
        }
        fence_barrier_init();
    }
    if (warp == 3) tmem_alloc(tmem_slot, kMpTmemColumns);
    dependency_wait();
    allow_dependents();
    if (warp == 0) {
        // the offsets, taken into 0 .. rows and not decreasing, whatever they hold; then the tiles before each expert
        int top = 0, run = 0;
        for (int e0 = 0; e0 <= a.experts + 1; e0 += 32) {
            const int e = e0 + lane;
            int o = e == 0 ? 0 : e <= a.experts ? a.offsets[e] : a.rows_total;
            o = max(0, min(o, a.rows_total));
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int q = __shfl_up_sync(0xFFFFFFFFu, o, d);
                if (lane >= d) o = max(o, q);
            }
            o = max(o, top);
            int before = __shfl_up_sync(0xFFFFFFFFu, o, 1);
            if (lane == 0) before = top;
            top = __shfl_sync(0xFFFFFFFFu, o, 31);
            int incl = (o - before + S::kRows - 1) / S::kRows;      // row tiles of expert e - 1
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int q = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if (lane >= d) incl += q;
            }
            if (e <= a.experts + 1) {
                row_start[e] = o;
                prefix[e] = run + incl;
            }
            run += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 columns are allocated, so they begin at column 0: a constant that keeps the products' operands uniform
    constexpr uint32_t tmem = 0;
    if (tid == 0 && *tmem_slot != tmem) raise_error(kErrProductTimeout);
    if (*tmem_slot != tmem) prefix[a.experts + 1] = 0;         // no tiles
    MpTiles d(a, prefix, row_start);

    if (warp == 0) {
        if (elect_one()) {
            // copies: weights, rows and weight scales
            int it = 0;
            bool ok = true;
            for (; ok && d.here(); d.next()) {
                if (d.none()) continue;
                const int n16 = (d.rows + 15) >> 4;
                const uint32_t bytes = WT * (16384 + 512) + n16 * 2048;
                const int64_t scale_tile = ((int64_t)d.e * a.feature_tiles + d.ft) * a.k_steps;
                for (int kb = 0; kb < a.k_steps; ++kb, ++it) {
                    const int s = it % kMpStages;
                    if (!mp_wait(&empty[s], (uint32_t)((it / kMpStages) & 1) ^ 1u)) {
                        ok = false;
                        break;
                    }
                    uint8_t* st = smem + s * S::kStageBytes;
                    mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
                    for (int i = 0; i < WT; ++i) {
                        tma_3d_g2s(st + i * 16384, &a.w[i], kb * 128, d.ft * 128, d.e, &full[s]);
                        bulk_g2s(sscale + s * S::kScaleBytes + i * 512, a.w_scales[i] + (scale_tile + kb) * 512, 512, &full[s]);
                    }
                    int at = 0;
#pragma unroll
                    for (int b = 0; b < kMpRowBoxes; ++b) {
                        const int h = 128 >> b;
                        if (n16 & (h >> 4)) {
                            tma_2d_g2s(st + WT * 16384 + at * 128, &a.rows[b], kb * 128, d.r0 + at, &full[s]);
                            at += h;
                        }
                    }
                }
            }
            if (!ok) {
                // let the copies in flight land before the shared memory is given up
                for (int s = 0; s < kMpStages && s < it; ++s) {
                    const int last = (it - 1 - s);
                    mbar_wait(&full[last % kMpStages], (uint32_t)((last / kMpStages) & 1));
                }
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t st0 = operand_desc(smem_addr(smem)), sc0 = scale_desc(smem_addr(sscale));
            int it = 0, tile = 0;
            bool ok = true;
            for (; ok && d.here(); d.next()) {
                if (d.none()) continue;
                const int b = tile & 1;
                const uint32_t idesc = mx_instr_desc((d.rows + 15) & ~15);
                const uint32_t acc = tmem + (uint32_t)b * kMpAccColumns;
                if (!mp_wait(&acc_empty[b], (uint32_t)((tile >> 1) & 1) ^ 1u)) break;
                tc_fence_after();
                for (int kb = 0; kb < a.k_steps; ++kb, ++it) {
                    const int s = it % kMpStages;
                    if (!mp_wait(&full[s], (uint32_t)((it / kMpStages) & 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    fence_proxy_async_smem();   // the scale warp's stores, before the tensor core reads them
                    const uint32_t st = st0 + (uint32_t)s * (S::kStageBytes >> 4);
                    const uint32_t sc = sc0 + (uint32_t)s * (S::kScaleBytes >> 4);
                    const uint32_t tsc = tmem + kMpScaleColumns + (uint32_t)s * 12;
#pragma unroll
                    for (int i = 0; i < WT; ++i) tc_copy_scales(tsc + 4 * i, sc + (512 >> 4) * i);
                    tc_copy_scales(tsc + 4 * WT, sc + (512 >> 4) * WT);
                    if (WT == 1 && d.rows > 128) tc_copy_scales(tsc + 8, sc + (1024 >> 4));
#pragma unroll
                    for (int i = 0; i < WT; ++i)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tc_mma_mx(acc + (uint32_t)(i * S::kRows), st + i * (16384 >> 4) + q * 2,
                                      st + WT * (16384 >> 4) + q * 2, mx_instr_step(idesc, q), tsc + 4 * i, tsc + 4 * WT,
                                      kb > 0 || q > 0);
                    tc_commit(&empty[s]);
                }
                tc_commit(&acc_full[b]);
                ++tile;
            }
        }
    } else if (warp == 2) {
        // the rows' scales: lane l takes rows l, l + 32, ... of the tile, whose words for one K step are
        // 16 consecutive bytes of the tensor core's scale tile
        const int cols = a.k >> 5;
        const bool words = (cols & 3) == 0;
        int it = 0;
        bool ok = true;
        for (; ok && d.here(); d.next()) {
            if (d.none()) continue;
            const uint8_t* base = a.row_scales + (int64_t)d.r0 * cols;
            constexpr int kWords = (S::kRows + 31) / 32;
            for (int kb = 0; kb < a.k_steps; ++kb, ++it) {
                const int s = it % kMpStages;
                if (!__all_sync(0xFFFFFFFFu, mp_wait(&empty[s], (uint32_t)((it / kMpStages) & 1) ^ 1u))) {
                    ok = false;
                    break;
                }
                uint8_t* sc = sscale + s * S::kScaleBytes + WT * 512 + lane * 16;
                if (words) {
                    // asynchronous 4-byte copies: this warp never waits for memory, only for a free stage
#pragma unroll
                    for (int c = 0; c < kWords; ++c) {
                        const int r = lane + 32 * c;
                        cp_async4(sc + (c >> 2) * 512 + (c & 3) * 4, base + (r < d.rows ? (int64_t)r * cols + kb * 4 : 0),
                                  r < d.rows ? 4 : 0);
                    }
                    cp_async_arrive(&full[s]);
                } else {
#pragma unroll
                    for (int c = 0; c < kWords; ++c) {
                        const int r = lane + 32 * c;
                        *reinterpret_cast<uint32_t*>(sc + (c >> 2) * 512 + (c & 3) * 4) =
                            r < d.rows ? row_scale_word(base + (int64_t)r * cols, kb, cols) : 0u;
                    }
                    mbar_arrive(&full[s]);
                }
            }
        }
        cp_async_wait_all();                    // none of this warp's copies outlives the block, whatever stopped it
    } else if (warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        int tile = 0;
        for (; d.here(); d.next()) {
            const bool zero = d.none();
            const int b = tile & 1;
            if (!zero) {
                if (!__all_sync(0xFFFFFFFFu, mp_wait(&acc_full[b], (uint32_t)((tile >> 1) & 1)))) break;
                tc_fence_after();
            }
            const uint32_t acc = tmem + (uint32_t)b * kMpAccColumns + lanes;
            const int f0 = d.ft * 128 + quarter * 32;
            const int64_t r0 = d.r0;
            if (WT == 1) {
                int area = 0;
                uint32_t lo[8], hi[8];                              // features 0..15 and 16..31 of the warp
                const auto fetch = [&](int c) {
                    if (!zero && c < d.rows) {
                        tmem_load_16x256b_x2(acc + c, lo);
                        tmem_load_16x256b_x2(acc + (16u << 16) + c, hi);
                    }
                };
#pragma unroll
                for (int i = 0; i < 8; ++i) lo[i] = hi[i] = 0u;
                fetch(half * 16);
                for (int c0 = half * 16; c0 < d.rows; c0 += 32, area ^= 1024) {
                    uint8_t* stage = sout + (warp - 4) * 2048 + area;   // [16 rows][32 features] bf16
                    // register pair i of `lo` holds rows c0 + 8 * (i / 2) + 2 * (lane % 4) + {0, 1} of feature
                    // lane / 4 + 8 * (i % 2); stored transposed, 8 features are 16 bytes of an output row
                    tmem_load_wait(lo, hi);
                    uint32_t m[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            m[h][i] = pack_bf16x2(__uint_as_float(lo[4 * h + 2 * i]), __uint_as_float(lo[4 * h + 2 * i + 1]));
                            m[h][2 + i] = pack_bf16x2(__uint_as_float(hi[4 * h + 2 * i]), __uint_as_float(hi[4 * h + 2 * i + 1]));
                        }
                    fetch(c0 + 32);
#pragma unroll
                    for (int h = 0; h < 2; ++h) stmatrix_x4_trans(stage + out_stage_at(8 * h + (lane & 7), lane >> 3), m[h]);
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = 8 * h + (lane >> 2), chunk = lane & 3;
                        const uint4 v = *reinterpret_cast<const uint4*>(stage + out_stage_at(r, chunk));
                        const int ff = f0 + chunk * 8;
                        if (c0 + r < d.rows && ff < a.n) {
                            uint16_t* o = a.out_bf16 + (r0 + c0 + r) * a.n + ff;
                            if ((a.n & 7) == 0)
                                *reinterpret_cast<uint4*>(o) = v;
                            else
                                st_u16_tail(o, &v.x, 4, a.n - ff);
                        }
                    }
                }
                __syncwarp();                                       // both areas free for the next tile
            } else {
                // fragment order (see tmem_load_16x256b_x2): this lane holds rows c0 + 8 h + 2 q + j of features
                // p + 8 i, q = lane % 4, p = lane / 4; the 8 lanes of one q hold the 32 features of their rows
                const int q4 = lane & 3, p = lane >> 2;
                const int64_t scale_cols = a.n >> 5;
                uint32_t g[2][8], u[2][8];
                const auto fetch = [&](int c) {
                    if (!zero && c < d.rows) {
                        tmem_load_16x256b_x2(acc + c, g[0]);
                        tmem_load_16x256b_x2(acc + (16u << 16) + c, g[1]);
                        tmem_load_16x256b_x2(acc + S::kRows + c, u[0]);
                        tmem_load_16x256b_x2(acc + (16u << 16) + S::kRows + c, u[1]);
                    }
                };
#pragma unroll
                for (int i = 0; i < 8; ++i) g[0][i] = g[1][i] = u[0][i] = u[1][i] = 0u;
                fetch(half * 16);
                for (int c0 = half * 16; c0 < d.rows; c0 += 32) {
                    tmem_load_wait(g[0], g[1]);
                    tmem_load_wait(u[0], u[1]);
                    // v[r][i]: row r = 2 h + j of this lane's four, feature p + 8 i
                    float v[4][4];
                    uint32_t top[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        top[r] = 0u;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int at = 4 * (r >> 1) + 2 * (i & 1) + (r & 1);
                            v[r][i] = silu_times(__uint_as_float(g[i >> 1][at]), __uint_as_float(u[i >> 1][at]));
                            top[r] = max(top[r], __float_as_uint(fabsf(v[r][i])));
                        }
                    }
                    fetch(c0 + 32);
                    // the scale needs the exponent of the block's largest magnitude only: two rows' exponents per word
                    uint32_t ex[2] = {(top[0] >> 23) | (top[1] >> 23 << 16), (top[2] >> 23) | (top[3] >> 23 << 16)};
#pragma unroll
                    for (int m = 4; m < 32; m <<= 1) {
                        ex[0] = __vmaxu2(ex[0], __shfl_xor_sync(0xFFFFFFFFu, ex[0], m));
                        ex[1] = __vmaxu2(ex[1], __shfl_xor_sync(0xFFFFFFFFu, ex[1], m));
                    }
                    int e8[4];
                    uint32_t w[4];                                  // byte i: feature p + 8 i
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int E = (int)((ex[r >> 1] >> (16 * (r & 1))) & 0xFFFFu);
                        e8[r] = E > 8 ? E - 8 : 0;
                        const float factor = __uint_as_float((uint32_t)(254 - e8[r]) << 23);
                        w[r] = cvt_fp8x4<kE4M3>(__fmul_rn(v[r][0], factor), __fmul_rn(v[r][1], factor),
                                                __fmul_rn(v[r][2], factor), __fmul_rn(v[r][3], factor));
                    }
                    // 4 x 4 byte transposes over the lanes p, p ^ 1, p ^ 2, p ^ 3: byte b of the result is feature
                    // 8 (p % 4) + 4 (p / 4) + b, so that a word is four neighbours
                    transpose_step<0>(w[0], w[1], 4, (p & 1) != 0);
                    transpose_step<0>(w[2], w[3], 4, (p & 1) != 0);
                    transpose_step<1>(w[0], w[1], 8, (p & 2) != 0);
                    transpose_step<1>(w[2], w[3], 8, (p & 2) != 0);
                    if (f0 < a.n) {
                        const int64_t row0 = r0 + c0 + 2 * q4;
                        const int fo = f0 + 8 * (p & 3) + 4 * (p >> 2);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int c = 8 * (r >> 1) + (r & 1);
                            if (c0 + 2 * q4 + c < d.rows)
                                *reinterpret_cast<uint32_t*>(a.out_codes + (row0 + c) * a.n + fo) = w[r];
                        }
                        const int c = 8 * ((p >> 1) & 1) + (p & 1);   // lane p < 4 writes the scale of row r = p
                        const int e = p == 0 ? e8[0] : p == 1 ? e8[1] : p == 2 ? e8[2] : e8[3];
                        if (p < 4 && c0 + 2 * q4 + c < d.rows)
                            a.out_scales[(row0 + c) * scale_cols + (f0 >> 5)] = (uint8_t)e;
                    }
                }
            }
            if (!zero) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[b]);
                ++tile;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_free(*tmem_slot, kMpTmemColumns);
}

unsigned unit_errors_moe_product(bool clear) { return read_unit_errors(clear); }

}  // namespace fp8q

using namespace fp8q;

namespace fp8q {

static bool mp_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const void* base, int rank,
                   const cuuint64_t* dims, const cuuint64_t* strides, int box_rows) {
    const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
    const cuuint32_t estride[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estride,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct MpCall {
    const uint8_t* codes;
    const uint8_t* scales;
    const uint8_t* w[2];
    const uint8_t* ws[2];
    const int32_t* offsets;
    int64_t rows, n, k;
    int experts;
    void* out;
    uint8_t* out_scales;
};

template <int WT>
static fp8q_status_t mp_launch(const MpCall& c, cudaStream_t stream) {
    if (c.rows < 0 || c.rows >= (int64_t)1 << 31 || c.experts < 1 || c.experts > kMpMaxExperts || c.n < 0)
        return FP8Q_ERR_SIZE;
    if (c.k <= 0 || c.k % MXFP8_BLOCK != 0 || (WT == 2 && c.n % MXFP8_BLOCK != 0)) return FP8Q_ERR_K;
    if (c.n >= (int64_t)1 << 31 || c.k >= (int64_t)1 << 31) return FP8Q_ERR_SIZE;
    if (c.n > 0 && (uint64_t)c.k > FP8Q_MAX_ELEMENTS / (uint64_t)c.n / (uint64_t)c.experts) return FP8Q_ERR_SIZE;
    const int64_t wide = c.n > c.k ? c.n : c.k;
    if (c.rows > 0 && (uint64_t)wide > FP8Q_MAX_ELEMENTS / (uint64_t)c.rows) return FP8Q_ERR_SIZE;
    if (c.rows == 0 || c.n == 0) return FP8Q_OK;
    const void* need[] = {c.codes, c.scales, c.w[0], c.ws[0], c.offsets, c.out, WT == 2 ? c.w[1] : c.w[0],
                          WT == 2 ? c.ws[1] : c.ws[0], WT == 2 ? c.out_scales : c.out};
    for (const void* p : need)
        if (!p) return FP8Q_ERR_NULL;
    for (const void* p : need)
        if (!aligned16(p)) return FP8Q_ERR_ALIGN;
    const size_t wn = (size_t)c.experts * (size_t)c.n * (size_t)c.k;
    const size_t wsn = mxfp8_swizzled_scale_bytes(c.experts, c.n, c.k);
    const size_t on = (size_t)c.rows * (size_t)c.n;
    const Range ins[] = {{c.codes, (size_t)(c.rows * c.k)}, {c.scales, (size_t)(c.rows * (c.k / 32))}, {c.w[0], wn},
                         {c.ws[0], wsn}, {c.w[1], wn}, {c.ws[1], wsn}, {c.offsets, 4 * (size_t)(c.experts + 1)}};
    const Range outs[] = {{c.out, WT == 1 ? 2 * on : on}, {c.out_scales, on / 32}};
    if (any_alias(outs, 2, ins, 7)) return FP8Q_ERR_ALIAS;

    using S = MpShape<WT>;
    const int64_t feature_tiles = (c.n + 127) / 128;
    const int64_t row_tiles = c.rows / S::kRows + (c.rows < c.experts ? c.rows : c.experts) + 1;
    if (feature_tiles * row_tiles >= (int64_t)1 << 31) return FP8Q_ERR_SIZE;
    const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
    if (!encode) return cuda_status(cudaErrorNotSupported);
    MpArgs a;
    const cuuint64_t wd[3] = {(cuuint64_t)c.k, (cuuint64_t)c.n, (cuuint64_t)c.experts};
    const cuuint64_t wst[2] = {(cuuint64_t)c.k, (cuuint64_t)c.k * (cuuint64_t)c.n};
    const cuuint64_t rd[2] = {(cuuint64_t)c.k, (cuuint64_t)c.rows};
    const cuuint64_t rst[1] = {(cuuint64_t)c.k};
    for (int i = 0; i < WT; ++i)
        if (!mp_map(encode, &a.w[i], c.w[i], 3, wd, wst, 128)) return cuda_status(cudaErrorInvalidValue);
    if (WT == 1) a.w[1] = a.w[0];
    for (int b = 0; b < kMpRowBoxes; ++b)
        if (!mp_map(encode, &a.rows[b], c.codes, 2, rd, rst, 128 >> b)) return cuda_status(cudaErrorInvalidValue);
    a.w_scales[0] = c.ws[0];
    a.w_scales[1] = c.ws[1];
    a.row_scales = c.scales;
    a.offsets = c.offsets;
    a.out_bf16 = static_cast<uint16_t*>(WT == 1 ? c.out : nullptr);
    a.out_codes = static_cast<uint8_t*>(WT == 2 ? c.out : nullptr);
    a.out_scales = c.out_scales;
    a.rows_total = (int)c.rows;
    a.experts = c.experts;
    a.n = (int)c.n;
    a.k = (int)c.k;
    a.feature_tiles = (int)feature_tiles;
    a.k_steps = (int)((c.k + 127) / 128);
    static KernelCache kc;
    int resident = 0;
    const fp8q_status_t st = prepare_kernel(kc, moe_product_kernel<WT>, kMpThreads, S::kSmem, S::kSmem, &resident);
    if (st != FP8Q_OK) return st;
    return launch(moe_product_kernel<WT>, grid_for((size_t)(feature_tiles * row_tiles), 1), kMpThreads, S::kSmem, stream, a);
}

}  // namespace fp8q

extern "C" fp8q_status_t mxfp8_moe_matmul(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                          const uint8_t* w_codes, const uint8_t* w_scales, const int32_t* offsets,
                                          int experts, int64_t n, int64_t k, void* out_bf16, fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("mxfp8_moe_matmul");
    const MpCall c = {codes, scales, {w_codes, nullptr}, {w_scales, nullptr}, offsets, rows, n, k, experts, out_bf16, nullptr};
    return mp_launch<1>(c, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" fp8q_status_t mxfp8_moe_swiglu(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                          const uint8_t* gate_codes, const uint8_t* gate_scales,
                                          const uint8_t* up_codes, const uint8_t* up_scales, const int32_t* offsets,
                                          int experts, int64_t n, int64_t k, uint8_t* out_codes, uint8_t* out_scales,
                                          fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("mxfp8_moe_swiglu");
    const MpCall c = {codes, scales, {gate_codes, up_codes}, {gate_scales, up_scales}, offsets, rows, n, k, experts,
                      out_codes, out_scales};
    return mp_launch<2>(c, reinterpret_cast<cudaStream_t>(stream));
}
