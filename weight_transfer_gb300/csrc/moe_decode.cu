// A mixture-of-experts layer on MXFP8 weights for a few tokens.
//
//     h[t, j] = silu(gate_e x_t) * (up_e x_t)  for token t's choice j, e = ids[t, j]
//     out[t]  = sum over j of weights[t, j] * (down_e h[t, j])
// x in MXFP8 rows, the weights as mxfp8_quantize_swizzled writes them; h stays
// in binary32, and the sum over the choices is rounded once.
//
// Two launches: the gate and up products with the activation, and the down
// product with the sum.
#include "fp8q_device.cuh"
#include "fp8q_host.cuh"

#include <algorithm>

namespace fp8q {

constexpr int kMdThreads = 256;
constexpr int kMdWarps = kMdThreads / 32;
constexpr int kMdMaxChoices = FP8Q_MOE_DECODE_MAX_TOKENS * FP8Q_MOE_MAX_TOPK;
constexpr int kMdTiles = 2;                 // tiles of 8 columns that one pass over an expert's weights takes
constexpr int kMdRow = 160;                 // bytes from row to row of a stage: 128, and 32 that keep rows off each other's banks

struct MdArgs {
    const uint8_t *codes, *scales;                  // [tokens, k], [tokens, k / 32]
    const void* ids;
    int id64;
    const float* weights;                           // [tokens, topk]
    int tokens, topk, experts;
    int64_t n, k;
    const uint8_t *gate, *gate_scales, *up, *up_scales, *down, *down_scales;
    uint8_t* h;                                     // [tokens * topk, 4, n], h's four terms
    uint8_t* hs;                                    // [tokens * topk, hgroups * 4], the first one's scales
    int hgroups;                                    // groups of four blocks of 32
    float* y;                                       // [tokens * topk, k], the down products
    int* done;                                      // [ceil(k / 64)], blocks of a tile of features that have stored theirs
    uint16_t* out;                                  // [tokens, k]
    int tiles;                                      // column tiles that a pass takes, at most kMdTiles
};

// ------------------------------------------------------------ building blocks ----
// D = A * B for 16 rows, 32 columns of K and 8 columns, e4m3 codes.  The order
// of K is free as long as A and B share it: lane 4 r + t holds bytes 8 t .. 8 t
// + 7 of the block of 32 for rows r and r + 8 of A and column r of B.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint2 a0, uint2 a1, uint2 b) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0.x), "r"(a1.x), "r"(a0.y), "r"(a1.y), "r"(b.x), "r"(b.y), "f"(0.0f));
}
// Four E8M0 bytes -> 2^(byte - 127) each, NaN for 255.
__device__ __forceinline__ void e8m0x4(uint32_t w, float (&f)[4]) {
    uint32_t a, b;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(a) : "h"((uint16_t)w));
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
    f[0] = bf16_lo(a); f[1] = bf16_hi(a); f[2] = bf16_lo(b); f[3] = bf16_hi(b);
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
// acc += (d * row) * column for a tile's sums over one block of 32: rows' scales a and b, columns' c.
__device__ __forceinline__ void scaled_add(uint64_t (&acc)[2], const float (&d)[4], float a, float b, uint64_t c) {
    acc[0] = f2_fma(f2_mul(f2_pack(d[0], d[1]), f2_pack(a, a)), c, acc[0]);
    acc[1] = f2_fma(f2_mul(f2_pack(d[2], d[3]), f2_pack(b, b)), c, acc[1]);
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
// Every block sorts the choices by expert for itself.
struct MdList {                             // arrays in shared memory, list_stride(choices) long
    int16_t* expert;                        // the experts that are chosen, rising
    int16_t* start;                         // where their choices start in `order`
    int16_t* order;                         // choices by expert, and in their order
    int16_t* token;                         // their tokens
    int active;
};
__host__ __device__ __forceinline__ int list_stride(int choices) { return (choices + 8) & ~7; }

struct MdScratch {
    int count[FP8Q_MOE_MAX_EXPERTS];
    int16_t key[kMdMaxChoices + 8], rank[kMdMaxChoices];
    int warp[kMdWarps];
    int active;
};

// The ids are read past the first-level cache: the down products' kernel reads
// them before its own dependency wait.
__device__ __forceinline__ void sort_choices(const MdArgs& a, MdList& s, MdScratch& w) {
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int choices = a.tokens * a.topk;
    for (int i = tid; i < a.experts; i += kMdThreads) w.count[i] = 0;
    for (int i = tid; i < ((choices + 7) & ~7); i += kMdThreads) {
        int64_t id = -1;
        if (i < choices)
            id = a.id64 ? (int64_t)__ldcg(static_cast<const long long*>(a.ids) + i) : (int64_t)__ldcg(static_cast<const int*>(a.ids) + i);
        w.key[i] = id >= 0 && id < a.experts ? (int16_t)id : (int16_t)-1;
    }
    __syncthreads();
    // a choice's rank: the earlier ones of its expert, counted eight at a time
    for (int i = tid; i < choices; i += kMdThreads) {
        const int key = w.key[i];
        if (key < 0) continue;
        atomicAdd(&w.count[key], 1);
        const uint32_t both = (uint32_t)key * 0x10001u;
        int below = 0;
        for (int j = 0; j < i; j += 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(&w.key[j]);
            const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t d = h[m] ^ both;
                below += (j + 2 * m < i && (d & 0xFFFFu) == 0) + (j + 2 * m + 1 < i && (d >> 16) == 0);
            }
        }
        w.rank[i] = (int16_t)below;
    }
    __syncthreads();
    // chosen experts and choices in front of each expert, in one scan: both stay below 2^16
    const int per = FP8Q_MOE_MAX_EXPERTS / kMdThreads;
    uint32_t mine[per], sum = 0;
#pragma unroll
    for (int j = 0; j < per; ++j) {
        const int e = tid * per + j;
        const int c = e < a.experts ? w.count[e] : 0;
        mine[j] = sum;
        sum += (c > 0 ? 0x10000u : 0u) + (uint32_t)c;
    }
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) w.warp[warp] = (int)upto;
    __syncthreads();
    uint32_t before = upto - sum;
    for (int j = 0; j < warp; ++j) before += (uint32_t)w.warp[j];
#pragma unroll
    for (int j = 0; j < per; ++j) {
        const int e = tid * per + j;
        if (e >= a.experts) break;
        const int c = w.count[e];
        const uint32_t at = before + mine[j];
        if (c > 0) {
            s.expert[at >> 16] = (int16_t)e;
            s.start[at >> 16] = (int16_t)(at & 0xFFFFu);
        }
        w.count[e] = (int)(at & 0xFFFFu);
    }
    if (tid == kMdThreads - 1) {
        w.active = (int)((before + sum) >> 16);
        s.start[w.active] = (int16_t)((before + sum) & 0xFFFFu);
    }
    __syncthreads();
    for (int i = tid; i < choices; i += kMdThreads) {
        const int key = w.key[i];
        if (key >= 0) {
            const int at = w.count[key] + w.rank[i];
            s.order[at] = (int16_t)i;
            s.token[at] = (int16_t)(i / a.topk);
        }
    }
    s.active = w.active;
    __syncthreads();
}

// out for 64 features from f0 on: the choices' products, weighted, in their order.
__device__ __forceinline__ void sum_choices(const MdArgs& a, int64_t f0) {
    for (int i = (int)threadIdx.x; i < a.tokens * 16; i += kMdThreads) {
        const int token = i >> 4;
        const int64_t f = f0 + (i & 15) * 4;
        if (f >= a.k) continue;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int j = 0; j < a.topk; ++j) {
            const int64_t choice = token * a.topk + j;
            const int64_t id = a.id64 ? (int64_t)__ldcg(static_cast<const long long*>(a.ids) + choice)
                                      : (int64_t)__ldcg(static_cast<const int*>(a.ids) + choice);
            if (id < 0 || id >= a.experts) continue;
            const float p = __ldcg(a.weights + choice);
            const float4 y = __ldcg(reinterpret_cast<const float4*>(a.y + choice * a.k + f));
            v.x = __fmaf_rn(p, y.x, v.x);
            v.y = __fmaf_rn(p, y.y, v.y);
            v.z = __fmaf_rn(p, y.z, v.z);
            v.w = __fmaf_rn(p, y.w, v.w);
        }
        *reinterpret_cast<uint2*>(a.out + token * a.k + f) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
}

// ------------------------------------------------------------- the products ----
// A block takes 32 features of an expert's gate and up weights, or 64 of its
// down weights.  Two of its warps share 16 rows of weights, one taking the even,
// one the odd groups of 128 columns of K: eight features' gate rows above their
// up rows, so that a lane gets both sums of a feature, or 16 features' down
// rows.  Such a unit of 16 rows of 128 bytes and their scales comes into a ring
// of the warp's own by asynchronous copies that run kMdDepth - 1 units ahead,
// across items, so that no barrier stops them.
//   The columns of a tensor-core tile are 8 rows of x, or the four terms of two
// rows of h.  Columns without a row repeat the first one's data; their sums are
// not read.
//   Down products wait for h in front of their first tile only; their weights
// are on the way by then.  The last block to store a tile of 64 features sums
// the choices for it, in their order.
constexpr int kMdDepth = 4;
constexpr int kMdScales = 16 * kMdRow;                  // where a stage's 16 scale lines lie
constexpr int kMdStage = kMdScales + 16 * 16;
constexpr int kMdRing = kMdWarps * kMdDepth * kMdStage;
constexpr int kMdSums = 2 * kMdWarps * 4 * 33 * 4;      // bytes of partial sums for each column tile

template <bool DOWN> __global__ void __launch_bounds__(kMdThreads, 2) moe_decode_kernel(const MdArgs a) {
    __shared__ int last_one;
    extern __shared__ __align__(16) unsigned char dyn[];
    float* red = reinterpret_cast<float*>(dyn + kMdRing);           // [2][warps][tiles][4][33]
    const int stride = list_stride(a.tokens * a.topk);
    int16_t* lists = reinterpret_cast<int16_t*>(dyn + kMdRing + a.tiles * kMdSums);
    MdList list = {lists, lists + stride, lists + 2 * stride, lists + 3 * stride, 0};
    uint32_t* xscales = reinterpret_cast<uint32_t*>(lists + 4 * stride);                    // [tokens][groups], of x
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t features = DOWN ? a.k : a.n, cols = DOWN ? a.n : a.k;
    const int kb = (int)(cols / 32), groups = (kb + 3) / 4;
    constexpr int kWidth = DOWN ? 64 : 32, kTile = DOWN ? 16 : 8, kRows = DOWN ? 2 : 8;
    const int blocks = (int)((features + kWidth - 1) / kWidth);
    // Ids and weights may be read by the second launch at once: the blocks of the first let it start only when
    // whatever wrote them had completed.
    if (!DOWN) {
        dependency_wait();
        allow_dependents();
        if (blockIdx.x == 0)
            for (int i = tid; i < (int)((a.k + 63) / 64); i += kMdThreads) a.done[i] = 0;
    }
    sort_choices(a, list, *reinterpret_cast<MdScratch*>(dyn));
    if (!DOWN)
        for (int i = tid; i < a.tokens * groups; i += kMdThreads) {
            const uint8_t* s = a.scales + (int64_t)(i / groups) * kb + i % groups * 4;
            uint32_t w = 0;
            for (int b = 0; b < 4; ++b)
                if (i % groups * 4 + b < kb) w |= (uint32_t)s[b] << (8 * b);
            xscales[i] = w;
        }
    const int pass_rows = kRows * a.tiles;
    const uint32_t ring = smem_addr(dyn) + warp * kMdDepth * kMdStage;
    const int q = lane >> 2, t = lane & 3;
    const int offset = (warp >> 1) * kTile, odd = warp & 1;
    const int warp_words = a.tiles * 4 * 33;
    const int items = list.active * blocks;

    // ---- the copies, ahead of the products
    // Gate and up go through all features of an expert before the next; down through all experts of a tile of
    // features, so that its sum over the choices can be formed while other tiles are on their way.
    int a_item = (int)blockIdx.x, a_ai = 0, a_r0 = 0, a_col = 0;
    const int c = (lane & 7) * 16;                      // eight lanes bring a row's 128 bytes
    const int64_t four = 4 * cols;
    const uint32_t to = ring + (lane >> 3) * kMdRow + c;
    const uint8_t *upper = nullptr, *lower = nullptr, *line = nullptr;
    auto aim = [&] {                                    // at the first group of an item
        a_col = odd * 128;
        int64_t f = 0;
        for (;; a_item += (int)gridDim.x) {             // the last tile of features may have none for this warp
            if (a_item >= items) return;
            f = (int64_t)(DOWN ? a_item / list.active : a_item % blocks) * kWidth + offset;
            if (f < features) break;
        }
        a_ai = DOWN ? a_item % list.active : a_item / blocks;
        const int64_t e = list.expert[a_ai];
        const int64_t at = (e * features + f + (lane >> 3)) * cols + a_col + c;
        const int64_t matrix = (features + 127) / 128 * groups * 512 * e + odd * 512;
        if (DOWN) {
            upper = a.down + at;
            lower = upper + 8 * cols;
            line = scale_line(a.down_scales, f + (lane & 15), 0, groups) + matrix;
        } else {
            upper = a.gate + at;
            lower = a.up + at;
            line = scale_line(lane < 8 ? a.gate_scales : a.up_scales, f + (lane & 7), 0, groups) + matrix;
        }
    };
    auto issue = [&](uint32_t stage) {
        if (a_item < items && odd < groups) {
            const uint32_t d = to + stage;
            if (a_col + 128 <= (int)cols) {
                copy16(d, upper);
                copy16(d + 4 * kMdRow, upper + four);
                copy16(d + 8 * kMdRow, lower);
                copy16(d + 12 * kMdRow, lower + four);
            } else {
                const bool in = a_col + c < (int)cols;
                const int64_t back = in ? 0 : -c;       // to a column that exists, of which nothing is read
                copy16_or_zero(d, upper + back, in);
                copy16_or_zero(d + 4 * kMdRow, upper + back + four, in);
                copy16_or_zero(d + 8 * kMdRow, lower + back, in);
                copy16_or_zero(d + 12 * kMdRow, lower + back + four, in);
            }
            if (lane < 16) copy16(ring + stage + kMdScales + lane * 16, line);
            upper += 256;
            lower += 256;
            line += 1024;
            a_col += 256;
            if (a_col >= (int)cols) {
                a_r0 += pass_rows;
                if (a_r0 >= list.start[a_ai + 1] - list.start[a_ai]) {
                    a_r0 = 0;
                    a_item += (int)gridDim.x;
                }
                aim();
            }
        }
        copy_commit();
    };
    aim();
#pragma unroll
    for (int i = 0; i < kMdDepth - 1; ++i) issue(i * kMdStage);
    if (DOWN) {
        dependency_wait();
        allow_dependents();
    } else {
        __syncthreads();                                // x's scales
    }

    uint32_t stage = 0;
    int flip = 0;
    for (int item = (int)blockIdx.x; item < items; item += (int)gridDim.x) {
        const int ai = DOWN ? item % list.active : item / blocks, block = DOWN ? item / list.active : item % blocks;
        const int first = list.start[ai], rows = list.start[ai + 1] - first;
        const int64_t f0 = (int64_t)block * kWidth;
        const uint32_t word = kMdScales + (uint32_t)((f0 + offset) >> 5 & 3) * 4 + q * 16;
        const bool idle = DOWN && f0 + offset >= features;
        for (int r0 = 0; r0 < rows; r0 += pass_rows) {
            const int left = rows - r0, nt = left > kRows && a.tiles > 1 ? 2 : 1;
            // this lane's column of B, and the scales of its sums' two columns
            const uint8_t* xb[kMdTiles];
            const uint32_t* cs[kMdTiles];
            uint32_t s0[kMdTiles], s1[kMdTiles];
#pragma unroll
            for (int i = 0; i < kMdTiles; ++i) {
                if (DOWN) {
                    const int rb = r0 + i * 2 + (q >> 2), rd = r0 + i * 2 + (t >> 1);
                    const int64_t cb = list.order[rb < rows ? first + rb : first], cd = list.order[rd < rows ? first + rd : first];
                    xb[i] = a.h + (cb * 4 + (q & 3)) * a.n + odd * 128 + t * 8;
                    cs[i] = reinterpret_cast<const uint32_t*>(a.hs) + cd * groups;
                } else {
                    const int rb = r0 + i * 8 + q, rd = r0 + i * 8 + t * 2;
                    xb[i] = a.codes + list.token[rb < rows ? first + rb : first] * a.k + odd * 128 + t * 8;
                    s0[i] = smem_addr(xscales + list.token[rd < rows ? first + rd : first] * groups);
                    s1[i] = smem_addr(xscales + list.token[rd + 1 < rows ? first + rd + 1 : first] * groups);
                }
            }
            uint64_t acc[kMdTiles][2];
#pragma unroll
            for (int i = 0; i < kMdTiles; ++i) acc[i][0] = acc[i][1] = 0;
            for (int g = idle ? groups : odd; g < groups; g += 2) {
                uint2 x[kMdTiles][4];
                uint32_t w0[kMdTiles], w1[kMdTiles];
                const bool whole = g * 4 + 4 <= kb;
#pragma unroll
                for (int i = 0; i < kMdTiles; ++i) {
                    if (i >= nt) break;
                    const uint8_t* from = xb[i] + (g - odd) * 128;
                    if (whole) {
#pragma unroll
                        for (int b = 0; b < 4; ++b) x[i][b] = *reinterpret_cast<const uint2*>(from + b * 32);
                    } else {
#pragma unroll
                        for (int b = 0; b < 3; ++b)
                            x[i][b] = g * 4 + b < kb ? *reinterpret_cast<const uint2*>(from + b * 32) : make_uint2(0u, 0u);
                    }
                    if (DOWN) {
                        // a term's scale is 2^-4 of the one's before it; the first is at least 2^(13 - 127)
                        w0[i] = cs[i][g] - (t & 1) * 0x08080808u;
                        w1[i] = w0[i] - 0x04040404u;
                    } else {
                        w0[i] = lds32(s0[i] + g * 4);
                        w1[i] = lds32(s1[i] + g * 4);
                    }
                }
                copy_wait<kMdDepth - 2>();
                __syncwarp();
                issue(stage == 0 ? (kMdDepth - 1) * kMdStage : stage - kMdStage);
                const uint32_t from = ring + stage;
                stage = stage + kMdStage < kMdDepth * kMdStage ? stage + kMdStage : 0;
                float su[4], sl[4];
                e8m0x4(lds32(from + word), su);
                e8m0x4(lds32(from + word + 128), sl);
                uint2 wu[4], wl[4];
                const uint32_t row = from + q * kMdRow + t * 8;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    wu[b] = lds64(row + b * 32);
                    wl[b] = lds64(row + 8 * kMdRow + b * 32);
                }
#pragma unroll
                for (int i = 0; i < kMdTiles; ++i) {
                    if (i >= nt) break;
                    float x0[4], x1[4];
                    e8m0x4(w0[i], x0);
                    e8m0x4(w1[i], x1);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (!whole && g * 4 + b >= kb) break;       // scales of no block may be anything
                        float d[4];
                        mma_e4m3(d, wu[b], wl[b], x[i][b]);
                        scaled_add(acc[i], d, su[b], sl[b], f2_pack(x0[b], x1[b]));
                    }
                }
            }
            float* p = red + (flip * kMdWarps + warp) * warp_words + lane;
#pragma unroll
            for (int i = 0; i < kMdTiles; ++i)
                if (i < nt) {
                    float v[4];
                    f2_unpack(acc[i][0], v[0], v[1]);
                    f2_unpack(acc[i][1], v[2], v[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[(i * 4 + j) * 33] = v[j];
                }
            __syncthreads();
            if (DOWN) {
                // 64 features of up to four rows: the sums of a feature's two warps over the four terms
                const int f = tid & 63, r = tid >> 6;
                if (r < left && r < nt * 2 && f0 + f < features) {
                    const float* s = red + (flip * kMdWarps + (f >> 4) * 2) * warp_words + ((r >> 1) * 4 + (f >> 3 & 1) * 2) * 33 +
                                     (f & 7) * 4 + (r & 1) * 2;
                    const float* z = s + warp_words;
                    a.y[(int64_t)list.order[first + r0 + r] * a.k + f0 + f] =
                        ((s[34] + z[34]) + (s[1] + z[1])) + ((s[33] + z[33]) + (s[0] + z[0]));
                }
            } else {
                // a warp takes a row, a lane a feature: the sums of its two warps, the activation, and the terms of h
                for (int r = warp; r < nt * 8 && r < left; r += kMdWarps) {
                    const float* s = red + (flip * kMdWarps + (lane >> 3) * 2) * warp_words + ((r >> 3) * 4 + (r & 1)) * 33 +
                                     (lane & 7) * 4 + ((r & 7) >> 1);
                    const float g = s[0] + s[warp_words], u = s[66] + s[warp_words + 66];
                    const float h = g / (1.0f + expf(-g)) * u;
                    // the block's largest value goes to [2^7, 2^8), and each term leaves at most 2^-4 of what it rounds
                    uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu) >> 23;
                    top = top < 20u ? 20u : top > 254u ? 254u : top;
                    float v = h * __uint_as_float((261u - top) << 23);
                    if (isinf(v)) v = __uint_as_float(0x7FFFFFFFu);     // the codes have no infinity
                    const int64_t choice = list.order[first + r0 + r];
                    uint8_t* out = a.h + choice * 4 * a.n + f0 + lane;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t code = cvt_fp8x2<kE4M3>(v, 0.0f) & 0xFFu;
                        out[j * a.n] = (uint8_t)code;
                        v = (v - decode_fp8x2<kE4M3>(code).x) * 16.0f;
                    }
                    if (lane == 0) a.hs[choice * a.hgroups * 4 + block] = (uint8_t)(top - 7u);
                }
            }
            flip ^= 1;                                  // the other half is free: its readers have met the barrier above
        }
        if (DOWN) {
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                last_one = atomicAdd(a.done + block, 1) == list.active - 1;
                __threadfence();
            }
            __syncthreads();
            if (last_one) sum_choices(a, f0);
        }
    }
    if (DOWN && list.active == 0)
        for (int block = (int)blockIdx.x; block < blocks; block += (int)gridDim.x) sum_choices(a, (int64_t)block * 64);
    copy_wait<0>();
}

}  // namespace fp8q

using namespace fp8q;

namespace {

// The down products, the four terms of h and a byte for every 32 of its values
// (rows of them filled up to words), and a counter for every 64 features.
size_t workspace_of(int64_t tokens, int topk, int64_t n, int64_t k) {
    const size_t choices = (size_t)tokens * (size_t)topk;
    return choices * (size_t)k * 4 + choices * (size_t)n * 4 + choices * (size_t)((n + 127) / 128) * 4 + (size_t)((k + 63) / 64) * 4;
}

bool valid_row(int64_t k) { return k > 0 && k % MXFP8_BLOCK == 0 && k <= FP8Q_MOE_DECODE_MAX_ROW; }

}  // namespace

extern "C" size_t mxfp8_moe_decode_workspace_bytes(int64_t tokens, int topk, int64_t n, int64_t k) {
    if (tokens < 0 || tokens > FP8Q_MOE_DECODE_MAX_TOKENS || topk < 1 || topk > FP8Q_MOE_MAX_TOPK || !valid_row(n) || !valid_row(k))
        return 0;
    return workspace_of(tokens, topk, n, k);
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
    const size_t need = workspace_of(tokens, topk, n, k);
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
    a.y = static_cast<float*>(workspace);
    a.h = reinterpret_cast<uint8_t*>(a.y + (size_t)choices * k);
    a.hs = a.h + (size_t)choices * n * 4;
    a.done = reinterpret_cast<int*>(a.hs + (size_t)choices * a.hgroups * 4);
    a.out = static_cast<uint16_t*>(out_bf16);
    a.tiles = (choices + 7) / 8 < kMdTiles ? (choices + 7) / 8 : kMdTiles;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    static_assert(kMdRing >= sizeof(MdScratch), "the sort works where the rings lie");
    constexpr size_t kMaxScales = FP8Q_MOE_DECODE_MAX_TOKENS * (FP8Q_MOE_DECODE_MAX_ROW / 128) * 4;
    constexpr size_t kMaxSmem = kMdRing + kMdTiles * kMdSums + 8 * (kMdMaxChoices + 8);
    const size_t smem = kMdRing + (size_t)a.tiles * kMdSums + 8 * (size_t)list_stride(choices);
    static KernelCache up_cache, down_cache;
    int resident = 0;
    const int most = choices < experts ? choices : experts;         // chosen experts
    fp8q_status_t st = prepare_kernel(up_cache, moe_decode_kernel<false>, kMdThreads, kMaxSmem, kMaxSmem + kMaxScales, &resident);
    if (st != FP8Q_OK) return st;
    st = launch(moe_decode_kernel<false>, grid_for((size_t)most * (size_t)(n / 32), 2), kMdThreads,
                smem + (size_t)tokens * (size_t)((k + 127) / 128) * 4, s, a);
    if (st != FP8Q_OK) return st;
    st = prepare_kernel(down_cache, moe_decode_kernel<true>, kMdThreads, kMaxSmem, kMaxSmem, &resident);
    if (st != FP8Q_OK) return st;
    return launch(moe_decode_kernel<true>, grid_for((size_t)most * (size_t)((k + 63) / 64), 2), kMdThreads, smem, s, a);
}
