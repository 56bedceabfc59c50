// A mixture-of-experts layer on MXFP8 weights for a few tokens.
//
//     h[t, j] = silu(gate_e x_t) * (up_e x_t)  for token t's choice j, e = ids[t, j]
//     out[t]  = sum over j of weights[t, j] * (down_e h[t, j])
// x in MXFP8 rows, the weights as mxfp8_quantize_swizzled writes them.  Two
// launches: the gate and up products with the activation, and the down product
// with the sum.  Between them h is held as two f16 terms with a scale for every
// 32 of them, 22 bits of each value, whose products with e4m3 codes are exact;
// 16 bits of it in one term would show in the output, binary32 cannot enter the
// products.  The sum over the choices is rounded once.
//
// Every chosen expert's weights are read once, whatever number of tokens chose
// it, which is what bounds the layer: 39 MB for one token and 8 of 128 experts of
// 2048 x 768, 544 MB for 32 tokens.  The products themselves are tiles of 16 rows
// of weights and 8 columns (mma.sync): with one to four rows of x per expert, the
// 128 rows and 16 columns of a tcgen05 tile would leave a token's 8 experts to 48
// of the 152 SMs, and their scales would have to be laid out for each expert.
// This GPU has no e4m3 form of mma.sync: the codes are converted to f16, exactly.
// The warps' own instructions are the second bound, 218 (gate and up) and 280
// (down) for a unit of 2 KB of weights, issued in 0.56 and 0.60 of all cycles at
// 32 tokens.
//     one, two, four, eight, sixteen and 32 tokens 13.8, 18.6, 32.0, 47.2, 69.4
//     and 96.0 us (5.7 TB/s) from a graph; through sort, gather, swiglu, matmul
//     and combine 22.0, 26.8, 40.1, 56.3, 79.3 and 99.9
// Columns without rows hold further blocks of K, so that a lane scales and adds
// one sum for four: without, one token took 1.06 times and 32 tokens 1.03 times as
// long as with.
// What did not gain, each against the kernel of its time: x or h fetched a unit
// ahead (the same), x held in shared memory (the same), partial sums without a
// barrier (the same), whole K to a warp (1.12 times as long), a lane's units in
// registers instead of rings (2.5 times).  Of the down products: tiles of 32
// features, which halve the reading of h (0.99, but 1.01 for sixteen tokens);
// units cut evenly over all SMs with sums joined in memory (1.05, one token 1.6).
#include "fp8q_device.cuh"
#include "fp8q_host.cuh"

#include <algorithm>
#include <type_traits>

namespace fp8q {

constexpr int kMdMaxChoices = FP8Q_MOE_DECODE_MAX_TOKENS * FP8Q_MOE_MAX_TOPK;

struct MdArgs {
    const uint8_t *codes, *scales;                  // [tokens, k], [tokens, k / 32]
    const void* ids;
    int id64;
    const float* weights;                           // [tokens, topk]
    int tokens, topk, experts;
    int64_t n, k;
    const uint8_t *gate, *gate_scales, *up, *up_scales, *down, *down_scales;
    uint16_t* h;                                    // [tokens * topk, 2, n], h's two terms in f16
    uint8_t* hs;                                    // [tokens * topk, hgroups * 4], their scales
    int hgroups;                                    // groups of four blocks of 32
    uint16_t* out;                                  // [tokens, k]
};

// ------------------------------------------------------------ building blocks ----
// D += A * B for 16 rows, 16 columns of K and 8 columns, in f16.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
// Products of 16 rows of weights with 8 columns over a block of 32.  Each is exact;
// an instruction adds its 16 and the sum so far, cut off 25 bits below the largest
// of them and then to 24 bits, towards zero.  The order of K is free as long as A
// and B share it: lane 4 r + t holds bytes 8 t .. 8 t + 7 of the block for rows r
// and r + 8 of A and column r of B, the latter as f16.
__device__ __forceinline__ void mma_block(float (&d)[4], uint2 a0, uint2 a1, uint4 b) {
    d[0] = d[1] = d[2] = d[3] = 0.0f;
    mma_f16(d, e4m3_f16(a0.x), e4m3_f16(a1.x), e4m3_f16(a0.x >> 16), e4m3_f16(a1.x >> 16), b.x, b.y);
    mma_f16(d, e4m3_f16(a0.y), e4m3_f16(a1.y), e4m3_f16(a0.y >> 16), e4m3_f16(a1.y >> 16), b.z, b.w);
}
// Byte i of each of two words of E8M0 scales -> 2^(byte - 127), NaN for 255.
__device__ __forceinline__ void e8m0_of(uint32_t a, uint32_t b, int i, float& x, float& y) {
    uint32_t r;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"((uint16_t)__byte_perm(a, b, (uint32_t)(i | (i + 4) << 4))));
    x = bf16_lo(r);
    y = bf16_hi(r);
}
// v[i], i below P.
template <int P> __device__ __forceinline__ float pick(const float (&v)[4], int i) {
    if (P == 1) return v[0];
    const float lo = i & 1 ? v[1] : v[0];
    if (P == 2) return lo;
    const float hi = i & 1 ? v[3] : v[2];
    return i & 2 ? hi : lo;
}
// 16 bytes global -> shared, past the first-level cache.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}

// The 16 bytes of the 128 x 4 tiled layout that hold the scales of blocks 4 j ..
// 4 j + 3 of row r, as their word (r / 32) % 4.
__device__ __forceinline__ const uint8_t* scale_line(const uint8_t* s, int64_t r, int64_t j, int64_t tiles) {
    return s + ((r >> 7) * tiles + j) * 512 + (r & 31) * 16;
}

// ------------------------------------------------------- choices by expert ----
// Every block sorts the choices by expert for itself, and cuts each expert's into
// passes of no more rows than a tile of its products takes.
struct MdList {                             // arrays in shared memory, list_stride(choices) long
    int16_t* expert;                        // the passes' experts, rising
    int16_t* start;                         // where their choices start in `order`
    int16_t* order;                         // choices by expert, and in their order
    int16_t* token;                         // their tokens
    int passes;
};
__host__ __device__ __forceinline__ int list_stride(int choices) { return (choices + 8) & ~7; }

struct MdScratch {
    int key[kMdMaxChoices + 4], sorted[kMdMaxChoices + 1];
    int heads[kMdMaxChoices / 32], cuts[kMdMaxChoices / 32];        // where an expert starts, and where a pass does
    int live;
};

// A choice's key is its expert and, below that, its own number, so that keys are
// unique and its place is the number of smaller ones; dropped choices go last.
// The ids are read past the first-level cache: the down products' kernel reads
// them before its own dependency wait.
constexpr int kMdDropped = 1024 << 10;
template <int NT, int ROWS> __device__ __forceinline__ void sort_choices(const MdArgs& a, MdList& s, MdScratch& w) {
    const int tid = (int)threadIdx.x, lane = tid & 31;
    const int choices = a.tokens * a.topk, padded = (choices + 3) & ~3;
    for (int i = tid; i < padded; i += NT) {
        int64_t id = -1;
        if (i < choices)
            id = a.id64 ? (int64_t)__ldcg(static_cast<const long long*>(a.ids) + i) : (int64_t)__ldcg(static_cast<const int*>(a.ids) + i);
        w.key[i] = id >= 0 && id < a.experts ? (int)id << 10 | i : kMdDropped | i;
    }
    if (tid == 0) w.sorted[0] = -1;
    __syncthreads();
    for (int i = tid; i < choices; i += NT) {
        const int key = w.key[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < padded; j += 4) {
            const int4 k = *reinterpret_cast<const int4*>(&w.key[j]);
            place += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
        }
        w.sorted[place + 1] = key;
        s.order[place] = (int16_t)i;
        s.token[place] = (int16_t)(i / a.topk);
    }
    __syncthreads();
    // an expert starts where the sorted keys' experts change
    for (int i = tid; i < ((choices + 31) & ~31); i += NT) {
        const int key = i < choices ? w.sorted[i + 1] : kMdDropped, before = i < choices ? w.sorted[i] : kMdDropped;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, key < kMdDropped && key >> 10 != before >> 10);
        if (lane == 0) w.heads[i >> 5] = (int)m;
        if (i < choices && key >= kMdDropped && before < kMdDropped) w.live = i;
        if (i == choices - 1 && key < kMdDropped) w.live = choices;
    }
    __syncthreads();
    const int live = w.live;
    for (int i = tid; i < ((choices + 31) & ~31); i += NT) {
        int word = i >> 5, heads = w.heads[word] & (int)((2u << lane) - 1u);
        while (heads == 0 && word > 0) heads = w.heads[--word];
        const int first = word * 32 + 31 - __clz(heads);                // where this choice's expert starts
        const unsigned m = __ballot_sync(0xFFFFFFFFu, i < live && (i - first) % ROWS == 0);
        if (lane == 0) w.cuts[i >> 5] = (int)m;
    }
    __syncthreads();
    int passes = 0;
    for (int i = 0; i < (choices + 31) >> 5; ++i) passes += __popc(w.cuts[i]);
    for (int i = tid; i < choices; i += NT) {
        const int word = i >> 5;
        if (!(w.cuts[word] >> lane & 1)) continue;
        int at = __popc(w.cuts[word] & ((1u << lane) - 1u));
        for (int j = 0; j < word; ++j) at += __popc(w.cuts[j]);
        s.expert[at] = (int16_t)(w.sorted[i + 1] >> 10);
        s.start[at] = (int16_t)i;
    }
    if (tid == 0) s.start[passes] = (int16_t)live;
    s.passes = passes;
    __syncthreads();
}

// ------------------------------------------------------------------- units ----
// Both launches read their weights in units of 16 rows of 128 bytes and the
// rows' scales.  A unit comes into a ring of a warp's own by asynchronous copies
// that run DEPTH - 1 units ahead, across experts and tiles, so that no barrier
// stops them.
//   In a stage the four pieces of 32 bytes of a row lie in an order of their own,
// piece b at b ^ (row % 4), so that the rows a warp reads at once keep off each
// other's banks.
constexpr int kMdRow = 128;
constexpr int kMdScales = 16 * kMdRow;                  // where a stage's 16 scale lines lie
constexpr int kMdStage = kMdScales + 16 * 16;

// Copies 16 rows of which this lane brings bytes c .. c + 15 of four: rows
// lane / 8 and that + 4 from `upper`, + 8 and + 12 from `lower`.  Columns from
// `left` on do not exist and become zeros.
__device__ __forceinline__ void copy_unit(uint32_t stage, const uint8_t* upper, const uint8_t* lower, int64_t four, const uint8_t* line,
                                          int left) {
    const int lane = (int)(threadIdx.x & 31u), c = (lane & 7) * 16;
    const uint32_t d = stage + (lane >> 3) * kMdRow + (c ^ (lane >> 3) * 32);
    if (left >= 128) {
        copy16(d, upper);
        copy16(d + 4 * kMdRow, upper + four);
        copy16(d + 8 * kMdRow, lower);
        copy16(d + 12 * kMdRow, lower + four);
    } else {
        const bool in = c < left;
        const int64_t back = in ? 0 : -c;               // to a column that exists, of which nothing is read
        copy16_or_zero(d, upper + back, in);
        copy16_or_zero(d + 4 * kMdRow, upper + back + four, in);
        copy16_or_zero(d + 8 * kMdRow, lower + back, in);
        copy16_or_zero(d + 12 * kMdRow, lower + back + four, in);
    }
    if (lane < 16) copy16(stage + kMdScales + lane * 16, line);
}

// What this lane multiplies of a unit: its two rows' bytes of the four blocks,
// and their scales.  `word`: the scale word of the unit's rows.  Scales of blocks
// from `nblocks` on may be anything and become 0, as the codes there are.
struct Weights {
    uint2 u[4], l[4];
    uint32_t su, sl;
};
__device__ __forceinline__ uint32_t only(uint32_t scales, int nblocks) {
    return nblocks < 4 ? scales & ((1u << (8 * nblocks)) - 1u) : scales;
}
__device__ __forceinline__ void read_unit(Weights& w, uint32_t stage, uint32_t word, int nblocks) {
    const int lane = (int)(threadIdx.x & 31u), q = lane >> 2, t = lane & 3;
    const uint32_t scales = stage + kMdScales + q * 16 + word, row = stage + q * kMdRow + t * 8;
    w.su = only(lds32(scales), nblocks);
    w.sl = only(lds32(scales + 128), nblocks);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const uint32_t at = row + ((b ^ (q & 3)) << 5);
        w.u[b] = lds64(at);
        w.l[b] = lds64(at + 8 * kMdRow);
    }
}

// ------------------------------------------------------ gate and up products ----
// A block takes 32 features of one pass, and a pair of its warps eight of
// them: their gate rows are the upper and their up rows the lower half of a unit,
// so that a lane gets both sums of a feature.  The two take turns at the groups
// of 128 columns.  A tensor-core tile's columns are 8 rows of x; columns
// without a row repeat the first one's data, and their sums are not read.
//   Up to four or two rows leave room for P = 2 or 4 blocks of 32 in the columns:
// those of block b are P-th parts of a tile, of which a product with the weights
// of one block gives one part.  A lane takes its part from each product, and
// scales and adds one sum instead of P.
constexpr int kUpThreads = 256;
constexpr int kUpRows = 8;                              // of a pass
constexpr int kUpWarps = kUpThreads / 32;
constexpr int kUpDepth = 3;
constexpr int kUpRing = kUpWarps * kUpDepth * kMdStage;
constexpr int kUpWords = 4 * 33;                        // a warp's partial sums
constexpr int kUpSums = 2 * kUpWarps * kUpWords * 4;

template <int BLOCKS> __global__ void __launch_bounds__(kUpThreads, BLOCKS) moe_decode_up_kernel(const MdArgs a) {
    extern __shared__ __align__(16) unsigned char dyn[];
    float* red = reinterpret_cast<float*>(dyn + kUpRing);           // [2][warps][4][33]
    const int stride = list_stride(a.tokens * a.topk);
    int16_t* lists = reinterpret_cast<int16_t*>(dyn + kUpRing + kUpSums);
    MdList list = {lists, lists + stride, lists + 2 * stride, lists + 3 * stride, 0};
    uint32_t* xscales = reinterpret_cast<uint32_t*>(lists + 4 * stride);                    // [tokens][groups]
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kb = (int)(a.k / 32), groups = (kb + 3) / 4, blocks = (int)(a.n / 32);
    dependency_wait();
    allow_dependents();
    sort_choices<kUpThreads, kUpRows>(a, list, *reinterpret_cast<MdScratch*>(dyn));
    const uint32_t ring = smem_addr(dyn) + warp * kUpDepth * kMdStage;
    const int q = lane >> 2, t = lane & 3;
    const int offset = (warp >> 1) * 8, part = warp & 1;
    const int items = list.passes * blocks, item0 = (int)blockIdx.x, item_step = (int)gridDim.x;

    int c_item = item0, c_col = 0;                      // where the copies are
    const uint8_t *upper = nullptr, *lower = nullptr, *line = nullptr;
    const int64_t four = 4 * a.k, matrix = (a.n + 127) / 128 * groups * 512;
    auto aim = [&] {
        c_col = part * 128;
        if (c_item >= items) return;
        const int ai = c_item / blocks;
        const int64_t e = list.expert[ai], f = (int64_t)(c_item - ai * blocks) * 32 + offset;
        const int64_t at = (e * a.n + f + (lane >> 3)) * a.k + c_col + (lane & 7) * 16;
        upper = a.gate + at;
        lower = a.up + at;
        line = scale_line(lane < 8 ? a.gate_scales : a.up_scales, f + (lane & 7), part, groups) + matrix * e;
    };
    auto issue = [&](uint32_t at) {
        if (c_item < items && part < groups) {
            copy_unit(ring + at, upper, lower, four, line, (int)a.k - c_col);
            upper += 256;
            lower += 256;
            line += 1024;
            c_col += 256;
            if (c_col >= (int)a.k) {
                c_item += item_step;
                aim();
            }
        }
        copy_commit();
    };
    aim();
#pragma unroll
    for (int i = 0; i < kUpDepth - 1; ++i) issue(i * kMdStage);
    for (int i = tid; i < a.tokens * groups; i += kUpThreads) {
        const uint8_t* s = a.scales + (int64_t)(i / groups) * kb + i % groups * 4;
        uint32_t w = 0;
        for (int b = 0; b < 4; ++b)
            if (i % groups * 4 + b < kb) w |= (uint32_t)s[b] << (8 * b);
        xscales[i] = w;
    }
    __syncthreads();

    uint32_t stage = 0;
    int flip = 0;
    for (int item = item0; item < items; item += item_step) {
        const int ai = item / blocks, block = item - ai * blocks;
        const int at = list.start[ai], left = list.start[ai + 1] - at;
        uint64_t acc[2] = {0, 0};
        auto multiply = [&](auto packed) {
            constexpr int P = decltype(packed)::value, R = 8 / P;       // blocks in the columns, rows of x
            // this lane's column of B, and its sums' two columns, whose rows are 2 t and 2 t + 1 modulo R
            const int xr = q % R, r = 2 * t % R, xblock = q / R, sblock = t * P / 4;
            const uint8_t* xb = a.codes + list.token[at + (xr < left ? xr : 0)] * a.k + (part * 4 + xblock) * 32 + t * 8;
            uint32_t s0 = smem_addr(xscales + list.token[at + (r < left ? r : 0)] * groups + part);
            uint32_t s1 = smem_addr(xscales + list.token[at + (r + 1 < left ? r + 1 : 0)] * groups + part);
            for (int b0 = part * 4; b0 < kb; b0 += 8) {
                uint2 x[4 / P];
                if (b0 + 4 <= kb) {
#pragma unroll
                    for (int i = 0; i < 4 / P; ++i) x[i] = *reinterpret_cast<const uint2*>(xb + i * P * 32);
                } else {
#pragma unroll
                    for (int i = 0; i < 4 / P; ++i)
                        x[i] = b0 + i * P + xblock < kb ? *reinterpret_cast<const uint2*>(xb + i * P * 32) : make_uint2(0u, 0u);
                }
                xb += 256;
                const uint32_t w0 = lds32(s0), w1 = lds32(s1);
                s0 += 8;
                s1 += 8;
                copy_wait<kUpDepth - 2>();
                __syncwarp();
                issue(stage == 0 ? (kUpDepth - 1) * kMdStage : stage - kMdStage);
                Weights w;
                read_unit(w, ring + stage, (uint32_t)(block & 3) * 4, kb - b0);
#pragma unroll
                for (int i = 0; i < 4 / P; ++i) {
                    const uint4 f = make_uint4(e4m3_f16(x[i].x), e4m3_f16(x[i].x >> 16), e4m3_f16(x[i].y), e4m3_f16(x[i].y >> 16));
                    float d[4][4], su, sl, c0, c1;
#pragma unroll
                    for (int b = 0; b < P; ++b) {
                        float v[4];
                        mma_block(v, w.u[i * P + b], w.l[i * P + b], f);
#pragma unroll
                        for (int j = 0; j < 4; ++j) d[j][b] = v[j];
                    }
                    e8m0_of(w.su, w.sl, i * P + sblock, su, sl);
                    e8m0_of(w0, w1, i * P + sblock, c0, c1);
                    const uint64_t c = f2_pack(c0, c1), up = f2_pack(su, su), lo = f2_pack(sl, sl);
                    acc[0] = f2_fma(f2_mul(f2_pack(pick<P>(d[0], sblock), pick<P>(d[1], sblock)), up), c, acc[0]);
                    acc[1] = f2_fma(f2_mul(f2_pack(pick<P>(d[2], sblock), pick<P>(d[3], sblock)), lo), c, acc[1]);
                }
                stage = stage + kMdStage < kUpDepth * kMdStage ? stage + kMdStage : 0;
            }
#pragma unroll
            for (int o = 4 / P; o < 4; o <<= 1) {
                acc[0] = f2_add(acc[0], __shfl_xor_sync(0xFFFFFFFFu, acc[0], o));
                acc[1] = f2_add(acc[1], __shfl_xor_sync(0xFFFFFFFFu, acc[1], o));
            }
        };
        if (left <= 2) multiply(std::integral_constant<int, 4>());
        else if (left <= 4) multiply(std::integral_constant<int, 2>());
        else multiply(std::integral_constant<int, 1>());
        float v[4];
        f2_unpack(acc[0], v[0], v[1]);
        f2_unpack(acc[1], v[2], v[3]);
        float* p = red + (flip * kUpWarps + warp) * kUpWords + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j * 33] = v[j];
        __syncthreads();
        // a warp takes a row, a lane a feature: the sums, the activation, and the terms of h
        if (warp < left) {
            const float* s = red + (flip * kUpWarps + (lane >> 3) * 2) * kUpWords +
                             (warp & 1) * 33 + (lane & 7) * 4 + (warp >> 1);
            const float g = s[0] + s[kUpWords], u = s[66] + s[kUpWords + 66];
            const float h = g / (1.0f + expf(-g)) * u;
            // the block's largest value goes to [2^14, 2^15): h = (hi + lo) * 2^(byte - 127)
            uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu) >> 23;
            top = top < 16u ? 16u : top > 254u ? 254u : top;
            const float v = h * __uint_as_float((268u - top) << 23);
            const __half hi = __float2half_rn(v);
            const __half lo = __hisinf(hi) ? __half(0.0f) : __float2half_rn(v - __half2float(hi));
            const int64_t choice = list.order[at + warp];
            uint16_t* out = a.h + choice * 2 * a.n + block * 32 + lane;
            out[0] = __half_as_ushort(hi);
            out[a.n] = __half_as_ushort(lo);
            if (lane == 0) a.hs[choice * a.hgroups * 4 + block] = (uint8_t)(top - 14u);
        }
        flip ^= 1;                                  // the other half is free: its readers have met the barrier above
    }
    copy_wait<0>();
}

// -------------------------------------------- down product, sum over choices ----
// A block, or a cluster of them where there are few, takes 16 output features
// of all tokens.  The pairs of a pass and a group of 128 columns of n are cut
// evenly over its warps; the columns of a tensor-core tile are the two terms of
// four rows of h, or of fewer in P blocks of K, as above.  A warp adds its
// products, times the choices' weights, to sums of its own, which are joined over
// the warps and over the cluster's blocks in a fixed order.  The first weights are
// on their way before h is waited for.
constexpr int kDownDepth = 3;
constexpr int kDownRows = 4;                            // of a pass
__host__ __device__ constexpr int down_ring(int threads) { return threads / 32 * kDownDepth * kMdStage; }
constexpr int kDownMaxCluster = 8;

template <int NT> __global__ void __launch_bounds__(NT, 1) moe_decode_down_kernel(const MdArgs a) {
    constexpr int kWarps = NT / 32;
    extern __shared__ __align__(16) unsigned char dyn[];
    float* part = reinterpret_cast<float*>(dyn + down_ring(NT));        // [warps][tokens][17]
    float* gather = reinterpret_cast<float*>(dyn);      // [ranks][tokens][16], in the first block, where its rings were
    const int stride = list_stride(a.tokens * a.topk), sums = a.tokens * 17;
    int16_t* lists = reinterpret_cast<int16_t*>(part + kWarps * sums);
    MdList list = {lists, lists + stride, lists + 2 * stride, lists + 3 * stride, 0};
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t ranks;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
    // Ids and weights may be read at once: the blocks of the launch before this one let it start only when whatever
    // wrote them had completed.
    sort_choices<NT, kDownRows>(a, list, *reinterpret_cast<MdScratch*>(dyn));
    const int64_t f0 = (int64_t)(blockIdx.x / ranks) * 16;
    const int groups = a.hgroups, nb = (int)(a.n / 32);
    const int units = list.passes * groups, shares = (int)ranks * kWarps, share = (int)rank * kWarps + warp;
    const int lo = (int)((int64_t)units * share / shares), hi = (int)((int64_t)units * (share + 1) / shares);
    const uint32_t ring = smem_addr(dyn) + warp * kDownDepth * kMdStage;
    const int q = lane >> 2, t = lane & 3;

    int c_unit = lo, c_g = 0;                           // where the copies are
    const int64_t four = 4 * a.n, matrix = (a.k + 127) / 128 * groups * 512;
    const uint8_t *upper = nullptr, *line = nullptr;
    auto aim = [&] {
        if (c_unit >= hi) return;
        const int ai = c_unit / groups;
        c_g = c_unit - ai * groups;
        const int64_t e = list.expert[ai];
        upper = a.down + (e * a.k + f0 + (lane >> 3)) * a.n + c_g * 128 + (lane & 7) * 16;
        line = scale_line(a.down_scales, f0 + (lane & 15), c_g, groups) + matrix * e;
    };
    auto issue = [&](uint32_t at) {
        if (c_unit < hi) {
            copy_unit(ring + at, upper, upper + 2 * four, four, line, (int)a.n - c_g * 128);
            upper += 128;
            line += 512;
            ++c_unit;
            if (++c_g == groups) aim();
        }
        copy_commit();
    };
    aim();
#pragma unroll
    for (int i = 0; i < kDownDepth - 1; ++i) issue(i * kMdStage);
    float* mine = part + warp * sums;
    for (int i = lane; i < sums; i += 32) mine[i] = 0.0f;
    __syncwarp();
    dependency_wait();
    allow_dependents();

    uint32_t stage = 0;
    const uint32_t word = (uint32_t)(f0 >> 5 & 3) * 4;
    for (int u = lo; u < hi;) {
        // one pass's groups g0 .. g1 - 1; the tile's columns are both terms of R rows in P blocks, and a lane's sums both
        // terms of one row in one of the blocks
        const int ai = u / groups, g0 = u - ai * groups, g1 = g0 + (hi - u) < groups ? g0 + (hi - u) : groups;
        const int at = list.start[ai], left = list.start[ai + 1] - at;
        float upper_sum = 0.0f, lower_sum = 0.0f;
        int choice = 0;
        auto multiply = [&](auto packed) {
            constexpr int P = decltype(packed)::value, R = 4 / P;       // blocks in the columns, rows of h
            const int hr = (q >> 1) % R, r = t % R, hblock = (q >> 1) / R, sblock = t / R;
            choice = list.order[at + (r < left ? r : 0)];
            const uint16_t* hb = a.h + ((int64_t)list.order[at + (hr < left ? hr : 0)] * 2 + (q & 1)) * a.n + g0 * 128 + hblock * 32 + t * 8;
            const uint32_t* sb = reinterpret_cast<const uint32_t*>(a.hs) + (int64_t)choice * groups;
            for (int g = g0; g < g1; ++g, hb += 128) {
                uint4 x[4 / P];
                if (g * 4 + 4 <= nb) {
#pragma unroll
                    for (int i = 0; i < 4 / P; ++i) x[i] = *reinterpret_cast<const uint4*>(hb + i * P * 32);
                } else {
#pragma unroll
                    for (int i = 0; i < 4 / P; ++i)
                        x[i] = g * 4 + i * P + hblock < nb ? *reinterpret_cast<const uint4*>(hb + i * P * 32) : make_uint4(0u, 0u, 0u, 0u);
                }
                const uint32_t c = only(sb[g], nb - g * 4);
                copy_wait<kDownDepth - 2>();
                __syncwarp();
                issue(stage == 0 ? (kDownDepth - 1) * kMdStage : stage - kMdStage);
                Weights w;
                read_unit(w, ring + stage, word, nb - g * 4);
#pragma unroll
                for (int i = 0; i < 4 / P; ++i) {
                    float upper[4], lower[4], su, sl, f, none;
#pragma unroll
                    for (int b = 0; b < P; ++b) {
                        float d[4];
                        mma_block(d, w.u[i * P + b], w.l[i * P + b], x[i]);
                        upper[b] = d[0] + d[1];
                        lower[b] = d[2] + d[3];
                    }
                    e8m0_of(w.su, w.sl, i * P + sblock, su, sl);
                    e8m0_of(c, 0u, i * P + sblock, f, none);
                    upper_sum = __fmaf_rn(pick<P>(upper, sblock) * su, f, upper_sum);
                    lower_sum = __fmaf_rn(pick<P>(lower, sblock) * sl, f, lower_sum);
                }
                stage = stage + kMdStage < kDownDepth * kMdStage ? stage + kMdStage : 0;
            }
#pragma unroll
            for (int o = R; o < 4; o <<= 1) {
                upper_sum += __shfl_xor_sync(0xFFFFFFFFu, upper_sum, o);
                lower_sum += __shfl_xor_sync(0xFFFFFFFFu, lower_sum, o);
            }
        };
        if (left == 1) multiply(std::integral_constant<int, 4>());
        else if (left == 2) multiply(std::integral_constant<int, 2>());
        else multiply(std::integral_constant<int, 1>());
        // one row after the other: a token that names an expert twice has two of them
        const float p = __ldcg(a.weights + choice);
        float* o = mine + choice / a.topk * 17 + q;
        for (int turn = 0; turn < 4 && turn < left; ++turn) {
            if (t == turn) o[0] = __fmaf_rn(p, upper_sum, o[0]), o[8] = __fmaf_rn(p, lower_sum, o[8]);
            __syncwarp();
        }
        u += g1 - g0;
    }
    copy_wait<0>();
    __syncthreads();
    if (ranks > 1) cluster_sync();                      // the first block's rings are free
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_addr(gather + rank * a.tokens * 16)));
    for (int i = tid; i < a.tokens * 16; i += NT) {
        const float* p = part + (i >> 4) * 17 + (i & 15);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += p[w * sums];
        if (ranks > 1) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * i), "f"(v) : "memory");
        else a.out[(int64_t)(i >> 4) * a.k + f0 + (i & 15)] = (uint16_t)pack_bf16x2(v, 0.0f);
    }
    if (ranks == 1) return;
    cluster_sync();
    if (rank != 0) return;
    for (int i = tid; i < a.tokens * 16; i += NT) {
        float v = 0.0f;
        for (uint32_t r = 0; r < ranks; ++r) v += gather[r * a.tokens * 16 + i];
        a.out[(int64_t)(i >> 4) * a.k + f0 + (i & 15)] = (uint16_t)pack_bf16x2(v, 0.0f);
    }
}

}  // namespace fp8q

using namespace fp8q;

namespace {

// The two terms of h and a byte for every 32 of its values, rows of them filled up to words.
size_t workspace_of(int64_t tokens, int topk, int64_t n) {
    const size_t choices = (size_t)tokens * (size_t)topk;
    return choices * (size_t)n * 4 + choices * (size_t)((n + 127) / 128) * 4;
}

// Sixteen warps a block for one or two tokens, whose units last each of them a
// few steps (one token 13.8 us, with twenty 14.9, with twenty-four 14.8; two 18.6,
// 19.2 and 19.4), twenty-four beyond (32 tokens 96.0 us, with twenty 97.1, with
// sixteen 101.1; eight 47.2, 47.3 and 48.1; four 32.0, 31.6 and 31.6).
constexpr int64_t kDownFewTokens = 2;
template <int NT> fp8q_status_t launch_down(const MdArgs& a, unsigned ranks, size_t lists, cudaStream_t stream) {
    const auto bytes = [&](int tokens, size_t l) { return down_ring(NT) + (size_t)NT / 32 * 17 * tokens * sizeof(float) + l; };
    static KernelCache cache;
    int resident = 0;
    const fp8q_status_t st = prepare_kernel(cache, moe_decode_down_kernel<NT>, NT, down_ring(NT),
                                            bytes(FP8Q_MOE_DECODE_MAX_TOKENS, 8 * (kMdMaxChoices + 8)), &resident);
    if (st != FP8Q_OK) return st;
    return launch_clusters(moe_decode_down_kernel<NT>, (unsigned)(a.k / 16) * ranks, ranks, NT, bytes(a.tokens, lists), stream, a);
}

// Two blocks per SM with 116 registers a thread, or three with 80 where that takes
// all items at once and two would not (16 experts of 768 features: two tokens
// 18.5 us, with two blocks 21.1; 8 experts 15.2 and 13.8, 81 experts 56.3 and 55.5,
// sixteen and 32 tokens the same; but four and eight tokens 31.1 and 46.0 with
// three, 32.0 and 47.2 with two).
template <int BLOCKS> fp8q_status_t launch_up(const MdArgs& a, size_t items, size_t smem, size_t most, cudaStream_t stream) {
    static KernelCache cache;
    int resident = 0;
    const fp8q_status_t st = prepare_kernel(cache, moe_decode_up_kernel<BLOCKS>, kUpThreads, most, most, &resident);
    return st != FP8Q_OK ? st : launch(moe_decode_up_kernel<BLOCKS>, grid_for(items, BLOCKS), kUpThreads, smem, stream, a);
}

bool valid_row(int64_t k) { return k > 0 && k % MXFP8_BLOCK == 0 && k <= FP8Q_MOE_DECODE_MAX_ROW; }

}  // namespace

extern "C" size_t mxfp8_moe_decode_workspace_bytes(int64_t tokens, int topk, int64_t n) {
    if (tokens < 0 || tokens > FP8Q_MOE_DECODE_MAX_TOKENS || topk < 1 || topk > FP8Q_MOE_MAX_TOPK || !valid_row(n)) return 0;
    return workspace_of(tokens, topk, n);
}

extern "C" fp8q_status_t mxfp8_moe_decode(const uint8_t* codes, const uint8_t* scales, const void* ids, int id_bytes,
                                          const float* weights, int64_t tokens, int topk, const uint8_t* gate_codes,
                                          const uint8_t* gate_scales, const uint8_t* up_codes, const uint8_t* up_scales,
                                          const uint8_t* down_codes, const uint8_t* down_scales, int experts, int64_t n,
                                          int64_t k, void* out_bf16, void* workspace, size_t workspace_bytes,
                                          fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("mxfp8_moe_decode");
    if (id_bytes != 4 && id_bytes != 8) return FP8Q_ERR_FORMAT;
    if (tokens < 0 || tokens > FP8Q_MOE_DECODE_MAX_TOKENS || experts < 1 || experts > FP8Q_MOE_MAX_EXPERTS) return FP8Q_ERR_SIZE;
    if (topk < 1 || topk > FP8Q_MOE_MAX_TOPK || !valid_row(n) || !valid_row(k)) return FP8Q_ERR_K;
    if (tokens == 0) return FP8Q_OK;
    const void* in[] = {codes, scales, ids, weights, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales};
    for (const void* p : in)
        if (!p) return FP8Q_ERR_NULL;
    if (!out_bf16 || !workspace) return FP8Q_ERR_NULL;
    for (const void* p : in)
        if (!aligned16(p)) return FP8Q_ERR_ALIGN;
    if (!aligned16(out_bf16) || !aligned16(workspace)) return FP8Q_ERR_ALIGN;
    const size_t need = workspace_of(tokens, topk, n);
    if (workspace_bytes < need) return FP8Q_ERR_SIZE;
    const size_t t = (size_t)tokens, w = (size_t)experts * (size_t)n * (size_t)k;
    const Range outs[] = {{out_bf16, t * (size_t)k * 2}, {workspace, need}};
    const size_t up_sc = mxfp8_swizzled_scale_bytes(experts, n, k), down_sc = mxfp8_swizzled_scale_bytes(experts, k, n);
    const Range ins[] = {{codes, t * (size_t)k}, {scales, t * (size_t)k / 32}, {ids, t * topk * id_bytes}, {weights, t * topk * 4},
                         {gate_codes, w}, {gate_scales, up_sc}, {up_codes, w}, {up_scales, up_sc},
                         {down_codes, w}, {down_scales, down_sc}};
    if (any_alias(outs, 2, ins, 10)) return FP8Q_ERR_ALIAS;
    const int choices = (int)tokens * topk;
    MdArgs a = {codes, scales, ids, id_bytes == 8, weights, (int)tokens, topk, experts, n, k, gate_codes, gate_scales,
                up_codes, up_scales, down_codes, down_scales};
    a.hgroups = (int)((n + 127) / 128);
    a.h = static_cast<uint16_t*>(workspace);
    a.hs = reinterpret_cast<uint8_t*>(a.h + (size_t)choices * n * 2);
    a.out = static_cast<uint16_t*>(out_bf16);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    static_assert(kUpRing >= sizeof(MdScratch) && down_ring(512) >= sizeof(MdScratch), "the sort works where the rings lie");
    static_assert(down_ring(512) >= kDownMaxCluster * FP8Q_MOE_DECODE_MAX_TOKENS * 16 * sizeof(float), "and the cluster's sums too");
    constexpr size_t kMaxLists = 8 * (kMdMaxChoices + 8);
    constexpr size_t kMaxUp = kUpRing + kUpSums + kMaxLists +
                              FP8Q_MOE_DECODE_MAX_TOKENS * (FP8Q_MOE_DECODE_MAX_ROW / 128) * 4;
    const size_t lists = 8 * (size_t)list_stride(choices);
    const size_t up_smem = kUpRing + kUpSums + lists + (size_t)tokens * (size_t)((k + 127) / 128) * 4;
    const size_t passes = std::min((size_t)choices, (size_t)experts + (size_t)choices / kUpRows);      // at most
    const size_t items = passes * (size_t)(n / 32), sms = (size_t)sm_count();
    const fp8q_status_t st = items > 2 * sms && items <= 3 * sms ? launch_up<3>(a, items, up_smem, kMaxUp, s)
                                                                 : launch_up<2>(a, items, up_smem, kMaxUp, s);
    if (st != FP8Q_OK) return st;
    unsigned ranks = 1;
    while (ranks < kDownMaxCluster && (int64_t)(k / 16) * ranks * 2 <= sm_count()) ranks *= 2;
    return tokens <= kDownFewTokens ? launch_down<512>(a, ranks, lists, s) : launch_down<768>(a, ranks, lists, s);
}
