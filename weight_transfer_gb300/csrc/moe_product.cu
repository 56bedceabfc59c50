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
// With many rows per expert two CTAs work as a pair on 256 features: each
// holds its own 128 features' weights and half of the rows.
//
// One CTA per SM walks over the tiles.  Warp 0 copies weights and rows by TMA,
// as few copies a K step as possible (its one thread's instructions bound the
// pipeline), warp 2 copies the scales and brings the rows' into the tensor
// core's tile order (rows of an expert start anywhere, so their scales cannot
// lie pre-tiled), warp 1 issues the products, warps 4 to 11 read the accumulators
// of one tile while the products of the next fill the other half of TMEM (two
// warps for each quarter of the lanes, every other 16 rows each).
//
// Measured back to back, 128 experts: 65,533 rows through 2048 x 768 weights
// 107 us (98 from a graph; HBM alone needs 78; of 528 MB half are writes),
// 65,536 rows through two 768 x 2048 weights 184 us, 2.2 PFLOP/s (164 us with
// pauses between, at a higher clock), 512 rows through the same 60 us, 6.8 TB/s of weights.  The
// prefill cases wait for a stage's round trip: five stages of 39 KB are on
// their way, the tensor pipe is busy about half the time (profiled at 32
// experts).  Tried and slower: weights multicast to two pairs (186 us against
// 176 then), 208 rows per tile with one set of accumulators (211 against 173),
// weights brought into L2 ahead (170 to 205 against 168), 16 reading warps
// (matmul 114.7 against 108.5; gate/up 164.0 against 160.1, though 16.5 against
// 18.6 for 6244 rows of k 320, whose epilogue they share).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp8q_host.cuh"
#include "tcgen05.cuh"

namespace fp8q {

constexpr int kMpMaxExperts = 1024;
constexpr int kMpListed = 128;                  // tiles of a CTA that are found ahead (see MpTiles)
constexpr int kMpRowBoxes = 6;
constexpr uint32_t kMpTmemColumns = 512;
constexpr unsigned kErrProductTimeout = 2u;

// How a call's CTAs work: singly with tiles of up to 32 rows (more and smaller
// stages: the weights' latency counts), singly, or in pairs.
enum MpKind { kMpFew, kMpSingle, kMpPair };

// WT weight tensors (1: matmul, 2: gate and up).
template <int WT, int KIND> struct MpShape {
    static constexpr bool PAIR = KIND == kMpPair;
    static constexpr int kReaders = 8;                                      // warps that read the accumulators
    static constexpr int kThreads = 128 + 32 * kReaders;
    static constexpr int kRows = KIND == kMpFew ? 32 : WT == 2 ? 112 : PAIR ? 208 : 224;    // most rows of a tile
    static constexpr int kHeld = PAIR ? kRows / 2 : kRows;                  // rows of it in this CTA's shared memory
    // Rows are copied by one box a K step, the lowest of these that holds the tile's, in units of 16 (8 for a pair's half).
    static constexpr int kUnits = kRows / 16;
    static __host__ __device__ constexpr int box(int b) {
        constexpr int big = kUnits > 8;         // 14: 14 12 10 7 4 1, 13: 13 11 9 7 4 1, 7: 7 5 4 3 2 1
        const int u = b == 0 ? kUnits : b == 1 ? kUnits - 2 : b == 2 ? kUnits - 3 - big : b == 3 ? (kUnits + big) / 2 : b == 4 ? (kUnits + 3) / 4 : 1;
        return u > 1 ? u : 1;
    }
    static constexpr int kStages = KIND == kMpFew ? (WT == 1 ? 9 : 5) : KIND == kMpSingle ? 4 : WT == 1 ? 6 : 5;
    static constexpr int kHalves = 2;                                       // tiles whose accumulators fit TMEM
    static constexpr uint32_t kAccColumns = WT * kRows;                     // of one tile
    static constexpr uint32_t kScaleBase = kHalves * kAccColumns;           // scales behind them:
    static constexpr uint32_t kScaleColumns = 4 * WT + (kRows > 128 ? 8 : 4);   // of one stage
    static_assert(kScaleBase + kStages * kScaleColumns <= kMpTmemColumns, "tensor memory");
    static constexpr int kStageBytes = WT * 16384 + kHeld * 128;
    static constexpr int kScaleBytes = WT * 512 + (kRows > 128 ? 1024 : 512);
    // Staging of the outputs: two areas of 16 bf16 rows per reading warp (matmul), or one area of 16 code rows per reading
    // warp and two of a tile's scale words (swiglu).
    static constexpr int kOutBytes = WT == 1 ? kReaders * 2048 : kReaders * 608 + 2 * kRows * 4;
    static constexpr int kBars = 2 * kStages + 4;
    static constexpr size_t kSmem = (size_t)kStages * (kStageBytes + kScaleBytes) + (kOutBytes + 15) / 16 * 16 + kBars * 8 + 16 +
                                    kMpListed * 16 + 2 * (kMpMaxExperts + 2) * 4 + 1024;
    static_assert(kStageBytes % 1024 == 0 && kSmem <= 232448, "shared memory");
    static constexpr bool boxes_fall() {
        for (int b = 1; b < kMpRowBoxes; ++b)
            if (box(b) > box(b - 1) || (box(b) == box(b - 1) && box(b) > 1)) return false;
        return box(0) == kUnits && box(kMpRowBoxes - 1) == 1;
    }
    static_assert(boxes_fall(), "the lowest box that holds a tile is the last one that does");
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

// A tile: rows r0 .. r0 + rows of expert e (`experts`: rows of no expert, which
// are written as zeros) and 128 features; rows < 0 behind the last tile.
struct MpTile {
    int e, ft, r0, rows;
};

// Tile number j of this CTA.  Both tables are in shared memory: row_start[e]
// is the first row of expert e (row_start[experts] the first row of no expert,
// row_start[experts + 1] = rows), prefix[e] the number of row tiles before it.
template <bool PAIR>
__device__ __forceinline__ MpTile mp_find(const MpArgs& a, const int* prefix, const int* row_start, int j) {
    const int units = PAIR ? (a.feature_tiles + 1) >> 1 : a.feature_tiles;      // feature tiles, or pairs of them
    const int me = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x, all = PAIR ? (int)gridDim.x >> 1 : (int)gridDim.x;
    const uint32_t t = (uint32_t)me + (uint32_t)j * (uint32_t)all;     // the host allows for fewer than 2^31 tiles
    MpTile d = {0, 0, 0, -1};
    if (t >= (uint32_t)prefix[a.experts + 1] * (uint32_t)units) return d;
    const int rt = (int)(t / (uint32_t)units), unit = (int)(t - (uint32_t)rt * (uint32_t)units);
    int lo = 0, hi = a.experts;                 // the last expert with prefix[.] <= rt
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= rt) lo = mid; else hi = mid - 1;
    }
    const int tiles = prefix[lo + 1] - prefix[lo];
    // equal tiles, in steps of 16 rows: fewer, fuller columns than full tiles and a rest
    const int per = ((row_start[lo + 1] - row_start[lo] + tiles - 1) / tiles + 15) & ~15;
    d.e = lo;
    d.ft = PAIR ? 2 * unit + (int)cluster_rank() : unit;
    d.r0 = row_start[lo] + (rt - prefix[lo]) * per;
    d.rows = min(row_start[lo + 1] - d.r0, per);
    return d;
}

// The tiles of one CTA, in the order in which every warp of it walks over
// them.  Finding one takes a search and two divisions, some 700 cycles that a
// single thread cannot hide (matmul, 65,533 rows: 22 us of 130); so the first
// kMpListed are found by all threads at once and kept in shared memory.
template <bool PAIR>
struct MpTiles {
    const MpArgs& a;
    const MpTile* listed;
    const int* prefix;
    const int* row_start;
    int j = 0;
    MpTile d;
    __device__ __forceinline__ bool here() {
        if (j < kMpListed) {
            const int4 v = *reinterpret_cast<const int4*>(listed + j);
            d = {v.x, v.y, v.z, v.w};
        } else {
            d = mp_find<PAIR>(a, prefix, row_start, j);
        }
        return d.rows >= 0;
    }
    __device__ __forceinline__ bool none() const { return d.e >= a.experts; }
};

// The scales of a tile's rows whose length is no multiple of 4 bytes: lane l
// holds rows l, l + 32, ... (C of them).  K step kb's four bytes of a row lie
// across the aligned words kb and kb + 1 behind the row's start.
template <int C>
struct MpScaleRows {
    const uint8_t* base;                        // the aligned word where the tile's first row begins
    uint32_t end;                               // bytes from there to the end of the array (as far as 32 bits reach)
    uint32_t at[C];                             // of each row's start from there; ~0 for no row

    __device__ __forceinline__ void open(const MpArgs& a, const MpTile& t, int lane) {
        const int64_t cols = a.k >> 5, first = t.r0 * cols, left = a.rows_total * cols - (first & ~(int64_t)3);
        base = a.row_scales + (first & ~(int64_t)3);
        end = left < 0xFFFFFFF0ll ? (uint32_t)left : 0xFFFFFFF0u;
#pragma unroll
        for (int c = 0; c < C; ++c)
            at[c] = lane + 32 * c < t.rows ? (uint32_t)(first & 3) + (uint32_t)(lane + 32 * c) * (uint32_t)cols : ~0u;
    }
    __device__ __forceinline__ int shift(int c) const { return 8 * (int)(at[c] & 3u); }
    // Words i .. i + N - 1 of row c; bytes past the array's end and rows that are none give 0.
    template <int N> __device__ __forceinline__ void words(int c, int i, uint32_t* w) const {
        const uint32_t o = (at[c] & ~3u) + 4u * (uint32_t)i;
        if (at[c] != ~0u && o + 4u * N <= end) {
#pragma unroll
            for (int n = 0; n < N; ++n) w[n] = *reinterpret_cast<const uint32_t*>(base + o + 4 * n);
            return;
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            w[n] = 0u;
            for (uint32_t j = 0; at[c] != ~0u && j < 4; ++j)
                if (o + 4 * n + j < end) w[n] |= (uint32_t)base[o + 4 * n + j] << (8 * j);
        }
    }
};

// Byte of 16-byte chunk `chunk` (8 features) of row r in a reading warp's
// 16 x 64-byte staging area; the exclusive or spreads 8 rows over all banks.
__device__ __forceinline__ int out_stage_at(int r, int chunk) { return r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4); }

// g / (1 + exp(-g)) * u of two values.  exp and the reciprocal are the
// hardware's (2 ulp and 1 ulp, subnormal results kept); rounding the exponent's
// product and its constant costs |g| * 2^-23.7 more, relative to exp(-g).  With
// g below -88.72 exp(-g) is infinite and the result -0.  The result is about to
// be rounded to 8 bits.
__device__ __forceinline__ uint64_t silu_times2(uint64_t g, uint64_t u) {
    constexpr float kLog2E = 1.44269504088896340736f;
    float a, b;
    f2_unpack(f2_mul(g, f2_pack(-kLog2E, -kLog2E)), a, b);
    asm("ex2.approx.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.f32 %0, %0;" : "+f"(b));
    f2_unpack(f2_add(f2_pack(a, b), f2_pack(1.0f, 1.0f)), a, b);
    asm("rcp.approx.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.f32 %0, %0;" : "+f"(b));
    return f2_mul(f2_mul(g, f2_pack(a, b)), u);
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

template <bool CLUSTER = false> __device__ __forceinline__ bool mp_wait(uint64_t* bar, uint32_t parity) {
    if (mbar_wait<CLUSTER>(bar, parity)) return true;
    raise_error(kErrProductTimeout);
    return false;
}

template <int WT, int KIND>
__global__ void __launch_bounds__((MpShape<WT, KIND>::kThreads), 1) moe_product_kernel(const __grid_constant__ MpArgs a) {
    using S = MpShape<WT, KIND>;
    constexpr bool PAIR = S::PAIR;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* sscale = smem + S::kStages * S::kStageBytes;
    uint8_t* sout = sscale + S::kStages * S::kScaleBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(sout + (S::kOutBytes + 15) / 16 * 16);
    uint64_t* empty = full + S::kStages;
    uint64_t* acc_full = empty + S::kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    MpTile* listed = reinterpret_cast<MpTile*>(tmem_slot + 4);
    int* prefix = reinterpret_cast<int*>(listed + kMpListed);
    int* row_start = prefix + kMpMaxExperts + 2;
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            // the copying thread and the scale warp's lanes (and the warp once more, where it also stores); for the first
            // of a pair the second one's full stage, too
            mbar_init(&full[s], 33 + ((a.k & 127) != 0 ? 1 : 0) + (PAIR && cluster_rank() == 0 ? 1 : 0));
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], PAIR ? 2 * S::kReaders : S::kReaders);
        }
        fence_barrier_init();
    }
    if (warp == 2 && lane < WT + kMpRowBoxes) prefetch_tmap(lane < WT ? &a.w[lane] : &a.rows[lane - WT]);
    if (warp == 3) {
        if (PAIR) tmem_alloc_pair(tmem_slot, kMpTmemColumns); else tmem_alloc(tmem_slot, kMpTmemColumns);
    }
    dependency_wait();
    allow_dependents();
    // the offsets, taken into 0 .. rows: fetched by all threads at once, as one warp would wait for each 32 of them
    for (int e = tid; e <= a.experts + 1; e += S::kThreads) {
        const int o = e == 0 ? 0 : e <= a.experts ? a.offsets[e] : a.rows_total;
        row_start[e] = max(0, min(o, a.rows_total));
    }
    __syncthreads();
    if (warp == 0) {
        // ... and made not to decrease, whatever they hold; then the tiles before each expert.  Each lane takes a run
        // of neighbours, so that two scans over the warp are enough.
        const int per = (a.experts + 2 + 31) >> 5, e0 = lane * per, e1 = min(e0 + per, a.experts + 2);
        int top = 0;
        for (int e = e0; e < e1; ++e) top = max(top, row_start[e]);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int q = __shfl_up_sync(0xFFFFFFFFu, top, d);
            if (lane >= d) top = max(top, q);
        }
        top = __shfl_up_sync(0xFFFFFFFFu, top, 1);
        if (lane == 0) top = 0;
        int run = 0;
        for (int e = e0; e < e1; ++e) {
            const int o = max(top, row_start[e]);
            run += (o - top + S::kRows - 1) / S::kRows;             // row tiles of expert e - 1
            row_start[e] = top = o;
            prefix[e] = run;
        }
        int before = run;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int q = __shfl_up_sync(0xFFFFFFFFu, before, d);
            if (lane >= d) before += q;
        }
        before -= run;
        for (int e = e0; e < e1; ++e) prefix[e] += before;
    }
    __syncthreads();
    if (tid < kMpListed) listed[tid] = mp_find<PAIR>(a, prefix, row_start, tid);
    tc_fence_before();
    if (PAIR) cluster_sync(); else __syncthreads();     // the other CTA's barriers are ready too
    tc_fence_after();
    // all 512 columns are allocated, so they begin at column 0: a constant that keeps the products' operands uniform
    constexpr uint32_t tmem = 0;
    if (tid == 0 && *tmem_slot != tmem) raise_error(kErrProductTimeout);
    const bool usable = *tmem_slot == tmem;
    const int rank = PAIR ? (int)cluster_rank() : 0;
    MpTiles<PAIR> tiles = {a, listed, prefix, row_start};

    if (warp == 0) {
        if (elect_one()) {
            // copies: weights, rows and weight scales
            int it = 0;
            bool ok = usable;
            for (; ok && tiles.here(); ++tiles.j) {
                if (tiles.none()) continue;
                const MpTile d = tiles.d;
                const int units = (d.rows + 15) >> 4;
                int box = 0;
#pragma unroll
                for (int b = 1; b < kMpRowBoxes; ++b)
                    if (S::box(b) >= units) box = b;
                constexpr int kUnit = PAIR ? 8 : 16;
                const int first = PAIR ? d.r0 + rank * units * kUnit : d.r0;
                uint32_t bytes = S::kUnits;
#pragma unroll
                for (int b = 1; b < kMpRowBoxes; ++b)
                    if (box == b) bytes = S::box(b);
                bytes = WT * 16384 + bytes * kUnit * 128;
                for (int kb = 0; kb < a.k_steps; ++kb, ++it) {
                    const int s = it % S::kStages;
                    if (!mp_wait(&empty[s], (uint32_t)((it / S::kStages) & 1) ^ 1u)) {
                        ok = false;
                        break;
                    }
                    uint8_t* st = smem + s * S::kStageBytes;
                    mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
                    for (int i = 0; i < WT; ++i) tma_3d_g2s(st + i * 16384, &a.w[i], kb * 128, d.ft * 128, d.e, &full[s]);
                    tma_2d_g2s(st + WT * 16384, &a.rows[box], kb * 128, first, &full[s]);
                }
            }
            // every stage given back: no commit of the pair's other CTA is on its way to this one any more
            for (int s = 0; PAIR && ok && s < S::kStages && s < it; ++s) {
                const int last = it - 1 - s;
                ok = mp_wait(&empty[last % S::kStages], (uint32_t)((last / S::kStages) & 1));
            }
            if (!ok) {
                // let the copies in flight land before the shared memory is given up
                for (int s = 0; s < S::kStages && s < it; ++s) {
                    const int last = (it - 1 - s);
                    mbar_wait(&full[last % S::kStages], (uint32_t)((last / S::kStages) & 1));
                }
            }
        }
    } else if (warp == 1 && PAIR && rank == 1) {
        if (elect_one()) {
            // the pair's first CTA issues the products; it learns here that this one's stage is full, and acquires
            // what this one's scale warp stored
            int it = 0;
            bool ok = usable;
            for (; ok && tiles.here(); ++tiles.j) {
                if (tiles.none()) continue;
                const MpTile d = tiles.d;
                for (int kb = 0; ok && kb < a.k_steps; ++kb, ++it) {
                    const int s = it % S::kStages;
                    ok = mp_wait(&full[s], (uint32_t)((it / S::kStages) & 1));
                    fence_proxy_async_smem();   // the scale warp's stores, before the tensor core reads them
                    if (ok) mbar_arrive_first(&full[s]);
                }
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t st0 = operand_desc(smem_addr(smem)), sc0 = scale_desc(smem_addr(sscale));
            int it = 0, tile = 0;
            bool ok = usable;
            for (; ok && tiles.here(); ++tiles.j) {
                if (tiles.none()) continue;
                const MpTile d = tiles.d;
                const int b = tile % S::kHalves;
                const uint32_t idesc = mx_instr_desc(PAIR ? 256 : 128, (d.rows + 15) & ~15);
                const uint32_t acc = tmem + (uint32_t)b * S::kAccColumns;
                if (!mp_wait<PAIR>(&acc_empty[b], (uint32_t)((tile / S::kHalves) & 1) ^ 1u)) break;
                tc_fence_after();
                for (int kb = 0; kb < a.k_steps; ++kb, ++it) {
                    const int s = it % S::kStages;
                    if (!mp_wait<PAIR>(&full[s], (uint32_t)((it / S::kStages) & 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    fence_proxy_async_smem();   // the scale warp's stores, before the tensor core reads them
                    const uint32_t st = st0 + (uint32_t)s * (S::kStageBytes >> 4);
                    const uint32_t sc = sc0 + (uint32_t)s * (S::kScaleBytes >> 4);
                    const uint32_t tsc = tmem + S::kScaleBase + (uint32_t)s * S::kScaleColumns;
#pragma unroll
                    for (int i = 0; i < WT + (S::kRows > 128 ? 2 : 1); ++i)
                        if (i <= WT || d.rows > 128) {
                            if (PAIR) tc_copy_scales_pair(tsc + 4 * i, sc + (512 >> 4) * i);
                            else tc_copy_scales(tsc + 4 * i, sc + (512 >> 4) * i);
                        }
#pragma unroll
                    for (int i = 0; i < WT; ++i)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t dst = acc + (uint32_t)(i * S::kRows);
                            const uint32_t wd = st + i * (16384 >> 4) + q * 2, rd = st + WT * (16384 >> 4) + q * 2;
                            if (PAIR) tc_mma_mx_pair(dst, wd, rd, mx_instr_step(idesc, q), tsc + 4 * i, tsc + 4 * WT, kb > 0 || q > 0);
                            else tc_mma_mx(dst, wd, rd, mx_instr_step(idesc, q), tsc + 4 * i, tsc + 4 * WT, kb > 0 || q > 0);
                        }
                    if (PAIR) tc_commit_pair(&empty[s]); else tc_commit(&empty[s]);
                }
                if (PAIR) tc_commit_pair(&acc_full[b]); else tc_commit(&acc_full[b]);
                ++tile;
            }
        }
    } else if (warp == 2) {
        // the scales: the weights' lie tiled, 16 bytes a lane; of the rows' lane l takes rows l, l + 32, ... of the
        // tile, whose words for one K step are 16 consecutive bytes of the tensor core's scale tile
        const int cols = a.k >> 5;
        constexpr int kWords = (S::kRows + 31) / 32;
        int it = 0;
        bool ok = usable;
        // waits for the stage of this step, sends for its weight scales and gives the place of the rows'
        const auto stage = [&](int64_t weights_at) -> uint8_t* {
            const int s = it % S::kStages;
            ok = __all_sync(0xFFFFFFFFu, mp_wait(&empty[s], (uint32_t)((it / S::kStages) & 1) ^ 1u));
            uint8_t* sc = sscale + s * S::kScaleBytes + lane * 16;
#pragma unroll
            for (int i = 0; i < WT; ++i)
                if (ok) cp_async16(sc + i * 512, a.w_scales[i] + weights_at);
            return sc + WT * 512;
        };
        const auto weights_of = [&](const MpTile& d) {
            const int sft = d.ft < a.feature_tiles ? d.ft : a.feature_tiles - 1;    // an odd one out has no scales
            return ((int64_t)d.e * a.feature_tiles + sft) * a.k_steps * 512 + lane * 16;
        };
        if ((cols & 3) == 0) {
            // asynchronous 4-byte copies: this warp never waits for memory, only for a free stage
            for (; ok && tiles.here(); ++tiles.j) {
                if (tiles.none()) continue;
                const MpTile d = tiles.d;
                const uint8_t* base = a.row_scales + (int64_t)d.r0 * cols;
                const int64_t wsc = weights_of(d);
                for (int kb = 0; kb < a.k_steps; ++kb, ++it) {
                    uint8_t* sc = stage(wsc + kb * 512);
                    if (!ok) break;
#pragma unroll
                    for (int c = 0; c < kWords; ++c) {
                        const int r = lane + 32 * c;
                        cp_async4(sc + (c >> 2) * 512 + (c & 3) * 4, r < d.rows ? base + ((int64_t)r * cols + kb * 4) : a.row_scales,
                                  r < d.rows ? 4 : 0);
                    }
                    cp_async_arrive(&full[it % S::kStages]);
                }
            }
        } else {
            // through registers, four K steps' words at a time, the next four (of this tile or the next) on their way
            MpScaleRows<kWords> rows;
            uint32_t now[kWords][5], then[kWords][5];
            bool opened = false;
            for (; ok && tiles.here(); ++tiles.j) {
                if (tiles.none()) continue;
                const MpTile d = tiles.d;
                const int64_t wsc = weights_of(d);
                if (!opened) {
                    rows.open(a, d, lane);
#pragma unroll
                    for (int c = 0; c < kWords; ++c) rows.template words<5>(c, 0, now[c]);
                    opened = true;
                }
                for (int kb0 = 0; ok && kb0 < a.k_steps; kb0 += 4) {
                    int shift[kWords];
#pragma unroll
                    for (int c = 0; c < kWords; ++c) shift[c] = rows.shift(c);
                    if (kb0 + 4 < a.k_steps) {
#pragma unroll
                        for (int c = 0; c < kWords; ++c) {
                            then[c][0] = now[c][4];
                            rows.template words<4>(c, kb0 + 5, then[c] + 1);
                        }
                    } else {
                        MpTiles<PAIR> behind = tiles;
                        ++behind.j;
                        if (behind.here() && !behind.none()) {
                            rows.open(a, behind.d, lane);
#pragma unroll
                            for (int c = 0; c < kWords; ++c) rows.template words<5>(c, 0, then[c]);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int kb = kb0 + q, left = cols - 4 * kb;
                        if (left <= 0) break;
                        uint8_t* sc = stage(wsc + kb * 512);
                        if (!ok) break;
                        const uint32_t mask = left < 4 ? (1u << (8 * left)) - 1u : ~0u;
                        uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
                        for (int c = 0; c < kWords; ++c) w[c] = __funnelshift_r(now[c][q], now[c][q + 1], shift[c]) & mask;
                        *reinterpret_cast<uint4*>(sc) = make_uint4(w[0], w[1], w[2], w[3]);
                        if (kWords > 4) *reinterpret_cast<uint4*>(sc + 512) = make_uint4(w[4], w[5], w[6], w[7]);
                        cp_async_arrive(&full[it % S::kStages]);        // the weights' scales
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&full[it % S::kStages]);     // the stores above, of all lanes
                        ++it;
                    }
#pragma unroll
                    for (int c = 0; c < kWords; ++c)
#pragma unroll
                        for (int i = 0; i < 5; ++i) now[c][i] = then[c][i];
                }
            }
        }
        cp_async_wait_all();                    // none of this warp's copies outlives the block, whatever stopped it
    } else if (warp >= 4) {
        const int quarter = warp & 3, share = (warp - 4) >> 2;     // lanes, and which 16 rows out of every kStep
        constexpr int kStep = 16 * (S::kReaders / 4);
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        int tile = 0, scale_area = 0;
        bool dead = false;
        for (; usable && tiles.here(); ++tiles.j) {
            const MpTile d = tiles.d;
            const bool zero = tiles.none();
            const int b = tile % S::kHalves;
            // a wait that ran out ends the output, not the walk: the reading warps meet at a barrier for every tile
            if (!zero && !dead) dead = !__all_sync(0xFFFFFFFFu, mp_wait(&acc_full[b], (uint32_t)((tile / S::kHalves) & 1)));
            if (!zero) tc_fence_after();
            const int rows_here = dead ? 0 : d.rows;
            const uint32_t acc = tmem + (uint32_t)b * S::kAccColumns + lanes;
            const int f0 = d.ft * 128 + quarter * 32;
            const int64_t r0 = d.r0;
            if (WT == 1) {
                int area = 0;
                uint32_t lo[8], hi[8];                              // features 0..15 and 16..31 of the warp
                const auto fetch = [&](int c) {
                    if (!zero && c < rows_here) {
                        tmem_load_16x256b_x2(acc + c, lo);
                        tmem_load_16x256b_x2(acc + (16u << 16) + c, hi);
                    }
                };
#pragma unroll
                for (int i = 0; i < 8; ++i) lo[i] = hi[i] = 0u;
                fetch(share * 16);
                for (int c0 = share * 16; c0 < rows_here; c0 += kStep, area ^= 1024) {
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
                    fetch(c0 + kStep);
#pragma unroll
                    for (int h = 0; h < 2; ++h) stmatrix_x4_trans(stage + out_stage_at(8 * h + (lane & 7), lane >> 3), m[h]);
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = 8 * h + (lane >> 2), chunk = lane & 3;
                        const uint4 v = *reinterpret_cast<const uint4*>(stage + out_stage_at(r, chunk));
                        const int ff = f0 + chunk * 8;
                        if (c0 + r < rows_here && ff < a.n) {
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
                uint8_t* tile_scales = sout + S::kReaders * 608 + scale_area * S::kRows * 4;
                uint32_t g[2][8], u[2][8];
                const auto fetch = [&](int c) {
                    if (!zero && c < rows_here) {
                        tmem_load_16x256b_x2(acc + c, g[0]);
                        tmem_load_16x256b_x2(acc + (16u << 16) + c, g[1]);
                        tmem_load_16x256b_x2(acc + S::kRows + c, u[0]);
                        tmem_load_16x256b_x2(acc + (16u << 16) + S::kRows + c, u[1]);
                    }
                };
#pragma unroll
                for (int i = 0; i < 8; ++i) g[0][i] = g[1][i] = u[0][i] = u[1][i] = 0u;
                fetch(share * 16);
                for (int c0 = share * 16; c0 < rows_here; c0 += kStep) {
                    tmem_load_wait(g[0], g[1]);
                    tmem_load_wait(u[0], u[1]);
                    // v[h][i]: rows c0 + 8 h + 2 q + {0, 1} (a register pair) of feature p + 8 i
                    uint64_t v[2][4];
                    uint32_t top[4];                                // of row r = 2 h + j of this lane's four
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float big[2] = {0.0f, 0.0f};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int at = 4 * h + 2 * (i & 1);
                            v[h][i] = silu_times2(
                                f2_pack(__uint_as_float(g[i >> 1][at]), __uint_as_float(g[i >> 1][at + 1])),
                                f2_pack(__uint_as_float(u[i >> 1][at]), __uint_as_float(u[i >> 1][at + 1])));
                            float x, y;
                            f2_unpack(v[h][i], x, y);
                            big[0] = fmaxf(big[0], fabsf(x));
                            big[1] = fmaxf(big[1], fabsf(y));
                        }
                        top[2 * h] = __float_as_uint(big[0]);
                        top[2 * h + 1] = __float_as_uint(big[1]);
                    }
                    fetch(c0 + kStep);
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
                    for (int h = 0; h < 2; ++h) {
                        float factor[2], f[2][4];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int E = (int)((ex[h] >> (16 * j)) & 0xFFFFu);
                            e8[2 * h + j] = E > 8 ? E - 8 : 0;
                            factor[j] = __uint_as_float((uint32_t)(254 - e8[2 * h + j]) << 23);
                        }
                        const uint64_t both = f2_pack(factor[0], factor[1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f2_unpack(f2_mul(v[h][i], both), f[0][i], f[1][i]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) w[2 * h + j] = cvt_fp8x4<kE4M3>(f[j][0], f[j][1], f[j][2], f[j][3]);
                    }
                    // 4 x 4 byte transposes over the lanes p, p ^ 1, p ^ 2, p ^ 3: byte b of the result is feature
                    // 8 (p % 4) + 4 (p / 4) + b, so that a word is four neighbours
                    transpose_step<0>(w[0], w[1], 4, (p & 1) != 0);
                    transpose_step<0>(w[2], w[3], 4, (p & 1) != 0);
                    transpose_step<1>(w[0], w[1], 8, (p & 2) != 0);
                    transpose_step<1>(w[2], w[3], 8, (p & 2) != 0);
                    // 16 rows of 32 bytes leave as one store of 16 bytes per lane, the scales below as words: with 4-byte
                    // stores of codes and single bytes of scales the stores bounded short sums (22,529 rows, n 1856,
                    // k 256: 86.0 -> 79.9 us; 65,536 rows, n 768: k 512 96.3 -> 90.1, k 2048 166.0 -> 164.0).  The row
                    // pitch (8 words, and 8 more behind every fourth row) keeps both sides free of bank conflicts
                    uint32_t* words = reinterpret_cast<uint32_t*>(sout + (warp - 4) * 608);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int c = 8 * (r >> 1) + 2 * q4 + (r & 1);
                        words[c * 8 + (c >> 2) * 8 + 2 * (p & 3) + (p >> 2)] = w[r];
                    }
                    const int sr = 8 * ((p >> 1) & 1) + 2 * q4 + (p & 1);     // lane p < 4 has the scale of row r = p
                    const int e = p == 0 ? e8[0] : p == 1 ? e8[1] : p == 2 ? e8[2] : e8[3];
                    if (p < 4 && c0 + sr < rows_here) tile_scales[(c0 + sr) * 4 + quarter] = (uint8_t)e;
                    __syncwarp();
                    const int c = lane >> 1;
                    if (f0 < a.n && c0 + c < rows_here)
                        *reinterpret_cast<uint4*>(a.out_codes + (r0 + c0 + c) * a.n + f0 + 16 * (lane & 1)) =
                            *reinterpret_cast<const uint4*>(words + c * 8 + (c >> 2) * 8 + 4 * (lane & 1));
                    __syncwarp();
                }
                // the tile's scales, four neighbouring blocks' bytes a row at once: behind a barrier of the reading warps
                // (the next tile's go to the other area, and are not read before the next barrier)
                named_barrier(1, 32 * S::kReaders);
                const int blocks = min(4, (a.n - d.ft * 128 + 31) >> 5);
                for (int r = tid - 128; r < rows_here && blocks > 0; r += 32 * S::kReaders) {
                    uint8_t* o = a.out_scales + (r0 + r) * (int64_t)(a.n >> 5) + d.ft * 4;
                    if (blocks == 4 && (a.n & 127) == 0)
                        *reinterpret_cast<uint32_t*>(o) = *reinterpret_cast<const uint32_t*>(tile_scales + r * 4);
                    else
                        for (int i = 0; i < blocks; ++i) o[i] = tile_scales[r * 4 + i];
                }
                scale_area ^= 1;
            }
            if (!zero) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && !dead) {
                    if (PAIR) mbar_arrive_first(&acc_empty[b]); else mbar_arrive(&acc_empty[b]);
                }
                ++tile;
            }
        }
    }
    tc_fence_before();
    if (PAIR) cluster_sync(); else __syncthreads();
    tc_fence_after();
    if (warp == 3) {
        if (PAIR) tmem_free_pair(*tmem_slot, kMpTmemColumns); else tmem_free(*tmem_slot, kMpTmemColumns);
    }
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

// The kind for a call (see MpKind), by the mean number of rows per expert.
// Measured with 78 experts (matmul 1760 x 768 / swiglu 768 x 2048): at 30 rows
// 30.7 / 59.4 us in small tiles, 32.8 / 61.5 in pairs, 34.8 / 61.4 singly; at
// 59 rows 36.9 / 63.4, 32.8 / 62.1 and 36.9 / 63.5.  A pair with an odd feature
// tile out computes it for nothing, which only many tiles make up for.
static MpKind mp_kind(int64_t rows, int experts, int64_t feature_tiles) {
    const int64_t each = rows / experts;
    if (each <= 48) return kMpFew;
    return feature_tiles % 2 == 0 || feature_tiles >= 8 ? kMpPair : kMpSingle;
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

template <int WT, int KIND>
static fp8q_status_t mp_start(const MpArgs& a, int64_t tiles, cudaStream_t stream);

template <int WT>
static fp8q_status_t mp_launch(const MpCall& c, cudaStream_t stream) {
    if (c.rows < 0 || c.rows >= (int64_t)1 << 30 || c.experts < 1 || c.experts > kMpMaxExperts || c.n < 0)
        return FP8Q_ERR_SIZE;
    if (c.k <= 0 || c.k % MXFP8_BLOCK != 0 || (WT == 2 && c.n % MXFP8_BLOCK != 0)) return FP8Q_ERR_K;
    if (c.n >= (int64_t)1 << 31 || c.k >= (int64_t)1 << 28) return FP8Q_ERR_SIZE;
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

    const int64_t feature_tiles = (c.n + 127) / 128;
    const MpKind kind = mp_kind(c.rows, c.experts, feature_tiles);
    const int most = kind == kMpFew ? MpShape<WT, kMpFew>::kRows : kind == kMpSingle ? MpShape<WT, kMpSingle>::kRows : MpShape<WT, kMpPair>::kRows;
    const int64_t row_tiles = c.rows / most + (c.rows < c.experts ? c.rows : c.experts) + 1;
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
    int height = 0;
    for (int b = 0; b < kMpRowBoxes; ++b) {
        const int h = kind == kMpFew      ? MpShape<WT, kMpFew>::box(b) * 16
                      : kind == kMpSingle ? MpShape<WT, kMpSingle>::box(b) * 16
                                          : MpShape<WT, kMpPair>::box(b) * 8;
        if (h == height)
            a.rows[b] = a.rows[b - 1];
        else if (!mp_map(encode, &a.rows[b], c.codes, 2, rd, rst, h))
            return cuda_status(cudaErrorInvalidValue);
        height = h;
    }
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
    const int64_t tiles = feature_tiles * row_tiles;
    switch (kind) {
        case kMpFew: return mp_start<WT, kMpFew>(a, tiles, stream);
        case kMpSingle: return mp_start<WT, kMpSingle>(a, tiles, stream);
        default: return mp_start<WT, kMpPair>(a, tiles, stream);
    }
}

template <int WT, int KIND>
static fp8q_status_t mp_start(const MpArgs& a, int64_t tiles, cudaStream_t stream) {
    static KernelCache kc;
    int resident = 0;
    constexpr size_t kSmem = MpShape<WT, KIND>::kSmem;
    const fp8q_status_t st = prepare_kernel(kc, moe_product_kernel<WT, KIND>, MpShape<WT, KIND>::kThreads, kSmem, kSmem, &resident);
    if (st != FP8Q_OK) return st;
    if (KIND != kMpPair) return launch(moe_product_kernel<WT, KIND>, grid_for((size_t)tiles, 1), MpShape<WT, KIND>::kThreads, kSmem, stream, a);
    // as many pairs as are resident at once, since each walks over its own share of the tiles
    static std::atomic<int> cached[kMaxDevices];
    const int dev = current_device();
    const bool cache = dev >= 0 && dev < kMaxDevices;
    int pairs = cache ? cached[dev].load(std::memory_order_relaxed) : 0;
    if (pairs < 1) {
        pairs = resident_clusters(moe_product_kernel<WT, KIND>, 2, MpShape<WT, KIND>::kThreads, kSmem);
        if (cache) cached[dev].store(pairs, std::memory_order_relaxed);
    }
    return launch_clusters(moe_product_kernel<WT, KIND>, 2u * (unsigned)pairs, 2, MpShape<WT, KIND>::kThreads, kSmem, stream, a);
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
