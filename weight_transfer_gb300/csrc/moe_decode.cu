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
constexpr int kMdTiles = 4;                 // tiles of 8 rows that one pass over an expert's weights takes
constexpr int kMdMaxCluster = 8;

struct MdArgs {
    const uint8_t *codes, *scales;                  // [tokens, k], [tokens, k / 32]
    const void* ids;
    int id64;
    const float* weights;                           // [tokens, topk]
    int tokens, topk, experts;
    int64_t n, k;
    const uint8_t *gate, *gate_scales, *up, *up_scales, *down, *down_scales;
    uint16_t *hi, *lo;                              // [tokens * topk, n], h's halves
    uint8_t* hs;                                    // [tokens * topk, hgroups * 4], their scales
    int hgroups;                                    // groups of four blocks of 32
    uint16_t* out;                                  // [tokens, k]
    int tiles;                                      // tiles of 8 rows that the buffer of partial sums holds
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
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two e4m3 codes -> two f16, exactly.
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
// Four E8M0 bytes -> 2^(byte - 127) each, NaN for 255.
__device__ __forceinline__ void e8m0x4(uint32_t w, float (&f)[4]) {
    uint32_t a, b;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(a) : "h"((uint16_t)w));
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
    f[0] = bf16_lo(a); f[1] = bf16_hi(a); f[2] = bf16_lo(b); f[3] = bf16_hi(b);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t ld_nc32(const void* p) {
    uint32_t r;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ld_nc64(const void* p) {
    uint2 r;
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// Past the first-level cache, for what may be read before a kernel's dependency wait.
__device__ __forceinline__ uint32_t ld_l2_32(const void* p) {
    uint32_t r;
    asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ld_l2_64(const void* p) {
    uint2 r;
    asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// The four scales of blocks 4 j .. 4 j + 3 of row r in the 128 x 4 tiled layout.
__device__ __forceinline__ const uint8_t* scale_word(const uint8_t* s, int64_t r, int64_t j, int64_t tiles) {
    return s + ((r >> 7) * tiles + j) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}

// ------------------------------------------------------- choices by expert ----
// Every block sorts the choices by expert for itself.
struct MdList {
    int16_t expert[kMdMaxChoices];          // the experts that are chosen, rising
    int16_t start[kMdMaxChoices + 1];       // where their choices start in `order`
    int16_t order[kMdMaxChoices];           // choices by expert, and in their order
    int active;
    int twice;                              // some token names an expert twice
};
struct MdScratch {
    int count[FP8Q_MOE_MAX_EXPERTS];
    int16_t key[kMdMaxChoices], rank[kMdMaxChoices];
    int warp[kMdWarps];
};

// The ids are read past the first-level cache: the down kernel reads them
// before its own dependency wait.
__device__ __forceinline__ void sort_choices(const MdArgs& a, MdList& s, MdScratch& w) {
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int choices = a.tokens * a.topk;
    for (int i = tid; i < a.experts; i += kMdThreads) w.count[i] = 0;
    for (int i = tid; i < choices; i += kMdThreads) {
        const int64_t id = a.id64 ? (int64_t)__ldcg(static_cast<const long long*>(a.ids) + i)
                                  : (int64_t)__ldcg(static_cast<const int*>(a.ids) + i);
        w.key[i] = id >= 0 && id < a.experts ? (int16_t)id : (int16_t)-1;
    }
    if (tid == 0) s.twice = 0;
    __syncthreads();
    if (warp == 0) {
        for (int base = 0; base < choices; base += 32) {
            const int i = base + lane;
            const int key = i < choices ? w.key[i] : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, key);
            const int below = __popc(same & ((1u << lane) - 1u));
            const int had = key >= 0 ? w.count[key] : 0;
            if (key >= 0) w.rank[i] = (int16_t)(had + below);
            __syncwarp();
            if (key >= 0 && below == 0) w.count[key] = had + __popc(same);
            __syncwarp();
        }
    } else {
        for (int i = tid - 32; i < choices; i += kMdThreads - 32) {
            const int key = w.key[i];
            for (int j = i - i % a.topk; key >= 0 && j < i; ++j)
                if (w.key[j] == key) s.twice = 1;
        }
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
        s.active = (int)((before + sum) >> 16);
        s.start[s.active] = (int16_t)((before + sum) & 0xFFFFu);
    }
    __syncthreads();
    for (int i = tid; i < choices; i += kMdThreads) {
        const int key = w.key[i];
        if (key >= 0) s.order[w.count[key] + w.rank[i]] = (int16_t)i;
    }
    __syncthreads();
}

// ------------------------------------------------------ gate and up products ----
// A block takes 32 features of one expert, in four passes of 8 whose gate rows
// are the upper and whose up rows the lower half of a tensor-core tile, so that
// a lane gets both sums of a feature.  Its warps share K.
struct UpTile {
    uint2 w[2][4][2];           // two groups of four blocks of 32; gate, up
    uint32_t s[2][2];
};

__device__ __forceinline__ void load_up(UpTile& t, const MdArgs& a, int e, int64_t f0, int step, int chunks) {
    const int lane = (int)(threadIdx.x & 31u), warp = (int)(threadIdx.x >> 5);
    const int kb = (int)(a.k / 32), groups = (kb + 3) / 4;
    const int64_t f = f0 + (step / chunks) * 8 + (lane >> 2);
    const int first = (step % chunks) * 2 * kMdWarps + warp;
    const int64_t row = ((int64_t)e * a.n + f) * a.k + (lane & 3) * 8;
    const int64_t per = (a.n + 127) / 128 * groups * 512;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int g = first + q * kMdWarps;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const bool in = g * 4 + b < kb;
            const int64_t at = row + (g * 4 + b) * 32;
            t.w[q][b][0] = in ? ld_stream8(a.gate + at) : make_uint2(0u, 0u);
            t.w[q][b][1] = in ? ld_stream8(a.up + at) : make_uint2(0u, 0u);
        }
        const bool in = g < groups;
        t.s[q][0] = in ? ld_nc32(scale_word(a.gate_scales + e * per, f, g, groups)) : 0u;
        t.s[q][1] = in ? ld_nc32(scale_word(a.up_scales + e * per, f, g, groups)) : 0u;
    }
}

// Scales of blocks 4 g .. 4 g + 3 of a row-major row.
__device__ __forceinline__ uint32_t row_scales(const uint8_t* s, int g, int kb) {
    if ((kb & 3) == 0) return ld_nc32(s + 4 * g);
    uint32_t w = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (4 * g + b < kb) w |= (uint32_t)s[4 * g + b] << (8 * b);
    return w;
}

__global__ void __launch_bounds__(kMdThreads, 2) moe_decode_up_kernel(const MdArgs a) {
    __shared__ MdList list;
    extern __shared__ __align__(16) unsigned char dyn[];
    float* red = reinterpret_cast<float*>(dyn);         // [4 passes][warps][tiles][4][32], a pass one word further
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    dependency_wait();
    allow_dependents();
    sort_choices(a, list, *reinterpret_cast<MdScratch*>(dyn));
    const int kb = (int)(a.k / 32), groups = (kb + 3) / 4;
    const int chunks = (groups + 2 * kMdWarps - 1) / (2 * kMdWarps), steps = 4 * chunks;
    const int blocks = (int)(a.n / 32);
    const int pass_words = kMdWarps * a.tiles * 128 + 1;
    const int items = list.active * blocks;
    for (int item = (int)blockIdx.x; item < items; item += (int)gridDim.x) {
        const int ai = item / blocks;
        const int block = item % blocks;
        const int64_t f0 = (int64_t)block * 32;
        const int e = list.expert[ai], first = list.start[ai], rows = list.start[ai + 1] - first;
        for (int r0 = 0; r0 < rows; r0 += 8 * a.tiles) {
            const int left = rows - r0, nt = (left + 7) / 8 < a.tiles ? (left + 7) / 8 : a.tiles;
            UpTile next;
            load_up(next, a, e, f0, 0, chunks);
            float acc[kMdTiles][4];
            for (int step = 0; step < steps; ++step) {
                const UpTile t = next;
                if (step + 1 < steps) load_up(next, a, e, f0, step + 1, chunks);
                const int chunk = step % chunks;
                if (chunk == 0) {
#pragma unroll
                    for (int i = 0; i < kMdTiles; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kMdTiles; ++i) {
                    if (i >= nt) break;
                    // this lane's column of B, and the two columns of its sums
                    const int rb = r0 + i * 8 + (lane >> 2), rd = r0 + i * 8 + (lane & 3) * 2;
                    const bool inb = rb < rows;
                    const int64_t tb = inb ? list.order[first + rb] / a.topk : 0;
                    const int64_t t0 = rd < rows ? list.order[first + rd] / a.topk : 0;
                    const int64_t t1 = rd + 1 < rows ? list.order[first + rd + 1] / a.topk : 0;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int g = (chunk * 2 + q) * kMdWarps + warp;
                        if (g >= groups) break;
                        uint2 x[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            x[b] = inb && g * 4 + b < kb ? ld_nc64(a.codes + tb * a.k + (g * 4 + b) * 32 + (lane & 3) * 8)
                                                         : make_uint2(0u, 0u);
                        float s0[4], s1[4], sg[4], su[4];
                        e8m0x4(row_scales(a.scales + t0 * kb, g, kb), s0);
                        e8m0x4(row_scales(a.scales + t1 * kb, g, kb), s1);
                        e8m0x4(t.s[q][0], sg);
                        e8m0x4(t.s[q][1], su);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            float d[4];
                            mma_e4m3(d, t.w[q][b][0], t.w[q][b][1], x[b]);
                            acc[i][0] = __fmaf_rn(d[0] * sg[b], s0[b], acc[i][0]);
                            acc[i][1] = __fmaf_rn(d[1] * sg[b], s1[b], acc[i][1]);
                            acc[i][2] = __fmaf_rn(d[2] * su[b], s0[b], acc[i][2]);
                            acc[i][3] = __fmaf_rn(d[3] * su[b], s1[b], acc[i][3]);
                        }
                    }
                }
                if (chunk == chunks - 1) {
                    float* p = red + (step / chunks) * pass_words + warp * a.tiles * 128 + lane;
#pragma unroll
                    for (int i = 0; i < kMdTiles; ++i)
                        if (i < nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j) p[(i * 4 + j) * 32] = acc[i][j];
                }
            }
            __syncthreads();
            // a warp takes a row, a lane a feature
            for (int r = warp; r < nt * 8 && r < left; r += kMdWarps) {
                const float* p = red + (lane >> 3) * pass_words + ((r >> 3) * 4 + (r & 1)) * 32 + (lane & 7) * 4 + ((r & 7) >> 1);
                float g = 0.0f, u = 0.0f;
#pragma unroll
                for (int v = 0; v < kMdWarps; ++v) {
                    g += p[v * a.tiles * 128];
                    u += p[v * a.tiles * 128 + 64];
                }
                const float h = g / (1.0f + expf(-g)) * u;
                // the block's largest value goes to [2^14, 2^15): h = (hi + lo) * 2^(byte - 127)
                uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu) >> 23;
                top = top < 16u ? 16u : top > 254u ? 254u : top;
                const float v = h * __uint_as_float((268u - top) << 23);
                const uint32_t hi = pack_f16x2(v, 0.0f) & 0xFFFFu;
                const float back = __half2float(__ushort_as_half((unsigned short)hi));
                const uint32_t lo = (hi & 0x7C00u) == 0x7C00u ? 0u : pack_f16x2(v - back, 0.0f) & 0xFFFFu;
                const int64_t choice = list.order[first + r0 + r];
                a.hi[choice * a.n + f0 + lane] = (uint16_t)hi;
                a.lo[choice * a.n + f0 + lane] = (uint16_t)lo;
                if (lane == 0) a.hs[choice * a.hgroups * 4 + block] = (uint8_t)(top - 14u);
            }
            __syncthreads();
        }
    }
}

// -------------------------------------------- down product, sum over choices ----
// A cluster takes 32 output features of all tokens.  The pairs of a chosen
// expert and a group of 128 columns of n are cut evenly over its warps; a warp
// adds its products, times the choices' weights, to sums of its own, which are
// joined over the warps and over the cluster's blocks in a fixed order.
struct DownTile {
    uint2 w[2][4][2];           // two tiles of 16 features, four blocks of 32; features r, r + 8
    uint32_t s[2][2];
};

__device__ __forceinline__ void load_down(DownTile& t, const MdArgs& a, int e, int64_t f0, int g) {
    const int lane = (int)(threadIdx.x & 31u);
    const int nb = (int)(a.n / 32), groups = a.hgroups;
    const int64_t per = (a.k + 127) / 128 * groups * 512;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t f = f0 + m * 16 + r * 8 + (lane >> 2);
            const uint8_t* row = a.down + ((int64_t)e * a.k + f) * a.n + (lane & 3) * 8;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                t.w[m][b][r] = g * 4 + b < nb ? ld_l2_64(row + (g * 4 + b) * 32) : make_uint2(0u, 0u);
            t.s[m][r] = ld_l2_32(scale_word(a.down_scales + e * per, f, g, groups));
        }
}

__global__ void __launch_bounds__(kMdThreads, 2) moe_decode_down_kernel(const MdArgs a) {
    __shared__ MdList list;
    extern __shared__ __align__(16) unsigned char dyn[];
    float* part = reinterpret_cast<float*>(dyn);        // [warps][tokens][33]
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t ranks;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
    if (ranks > 1) cluster_arrive();
    const int sums = a.tokens * 33;
    float* gather = part + kMdWarps * sums;             // [ranks][tokens][32], in the first block
    // Ids and weights may be read at once: the blocks of the launch before this one let it start only when whatever
    // wrote them had completed.
    sort_choices(a, list, *reinterpret_cast<MdScratch*>(dyn));
    for (int i = tid; i < kMdWarps * sums; i += kMdThreads) part[i] = 0.0f;
    const int64_t f0 = (int64_t)(blockIdx.x / ranks) * 32;
    const int groups = a.hgroups, nb = (int)(a.n / 32);
    const int units = list.active * groups, shares = (int)ranks * kMdWarps, share = (int)rank * kMdWarps + warp;
    const int lo = (int)((int64_t)units * share / shares), hi = (int)((int64_t)units * (share + 1) / shares);
    DownTile next;
    if (lo < hi) load_down(next, a, list.expert[lo / groups], f0, lo % groups);
    dependency_wait();
    allow_dependents();
    __syncthreads();
    float* mine = part + warp * sums;
    for (int u = lo; u < hi; ++u) {
        const DownTile t = next;
        if (u + 1 < hi) load_down(next, a, list.expert[(u + 1) / groups], f0, (u + 1) % groups);
        const int ai = u / groups, g = u % groups;
        const int first = list.start[ai], rows = list.start[ai + 1] - first;
        for (int r0 = 0; r0 < rows; r0 += 8) {
            const int rb = r0 + (lane >> 2), rd = r0 + (lane & 3) * 2;
            const int64_t cb = rb < rows ? list.order[first + rb] : -1;
            const int c0 = rd < rows ? list.order[first + rd] : -1, c1 = rd + 1 < rows ? list.order[first + rd + 1] : -1;
            uint4 xh[4], xl[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const bool in = cb >= 0 && g * 4 + b < nb;
                const int64_t at = cb * a.n + (g * 4 + b) * 32 + (lane & 3) * 8;
                xh[b] = in ? __ldcg(reinterpret_cast<const uint4*>(a.hi + at)) : make_uint4(0u, 0u, 0u, 0u);
                xl[b] = in ? __ldcg(reinterpret_cast<const uint4*>(a.lo + at)) : make_uint4(0u, 0u, 0u, 0u);
            }
            float s0[4], s1[4];
            e8m0x4(c0 >= 0 ? __ldcg(reinterpret_cast<const uint32_t*>(a.hs) + (int64_t)c0 * groups + g) : 0u, s0);
            e8m0x4(c1 >= 0 ? __ldcg(reinterpret_cast<const uint32_t*>(a.hs) + (int64_t)c1 * groups + g) : 0u, s1);
            const float p0 = c0 >= 0 ? __ldcg(a.weights + c0) : 0.0f, p1 = c1 >= 0 ? __ldcg(a.weights + c1) : 0.0f;
            float acc[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float sa[4], sb[4];
                e8m0x4(t.s[m][0], sa);
                e8m0x4(t.s[m][1], sb);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][j] = 0.0f;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (g * 4 + b >= nb) break;
                    const uint2 w0 = t.w[m][b][0], w1 = t.w[m][b][1];
                    const uint32_t a0 = e4m3_f16(w0.x), a1 = e4m3_f16(w1.x), a2 = e4m3_f16(w0.x >> 16), a3 = e4m3_f16(w1.x >> 16);
                    const uint32_t a4 = e4m3_f16(w0.y), a5 = e4m3_f16(w1.y), a6 = e4m3_f16(w0.y >> 16), a7 = e4m3_f16(w1.y >> 16);
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_f16(d, a0, a1, a2, a3, xl[b].x, xl[b].y);
                    mma_f16(d, a4, a5, a6, a7, xl[b].z, xl[b].w);
                    mma_f16(d, a0, a1, a2, a3, xh[b].x, xh[b].y);
                    mma_f16(d, a4, a5, a6, a7, xh[b].z, xh[b].w);
                    acc[m][0] = __fmaf_rn(d[0] * sa[b], s0[b], acc[m][0]);
                    acc[m][1] = __fmaf_rn(d[1] * sa[b], s1[b], acc[m][1]);
                    acc[m][2] = __fmaf_rn(d[2] * sb[b], s0[b], acc[m][2]);
                    acc[m][3] = __fmaf_rn(d[3] * sb[b], s1[b], acc[m][3]);
                }
            }
            // columns of one tile are different tokens unless a token names an expert twice: then one column at a time
            const int turns = list.twice ? 4 : 1;
            for (int turn = 0; turn < turns; ++turn) {
                if (turns == 1 || (lane & 3) == turn) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int f = m * 16 + r * 8 + (lane >> 2);
                            if (c0 >= 0) {
                                float* o = mine + c0 / a.topk * 33 + f;
                                *o = __fmaf_rn(p0, acc[m][2 * r], *o);
                            }
                            if (c1 >= 0) {
                                float* o = mine + c1 / a.topk * 33 + f;
                                *o = __fmaf_rn(p1, acc[m][2 * r + 1], *o);
                            }
                        }
                }
                __syncwarp();
            }
        }
    }
    __syncthreads();
    if (ranks > 1) cluster_wait();                      // the first block has started
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_addr(gather + rank * a.tokens * 32)));
    for (int i = tid; i < a.tokens * 32; i += kMdThreads) {
        const float* p = part + (i >> 5) * 33 + (i & 31);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kMdWarps; ++w) v += p[w * sums];
        if (ranks > 1) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * i), "f"(v) : "memory");
        else a.out[(int64_t)(i >> 5) * a.k + f0 + (i & 31)] = (uint16_t)pack_bf16x2(v, 0.0f);
    }
    if (ranks == 1) return;
    cluster_sync();
    if (rank != 0) return;
    for (int i = tid; i < a.tokens * 32; i += kMdThreads) {
        float v = 0.0f;
        for (uint32_t r = 0; r < ranks; ++r) v += gather[r * a.tokens * 32 + i];
        a.out[(int64_t)(i >> 5) * a.k + f0 + (i & 31)] = (uint16_t)pack_bf16x2(v, 0.0f);
    }
}

}  // namespace fp8q

using namespace fp8q;

namespace {

// The two halves of h and a byte for every 32 values, rows of them filled up to words.
size_t workspace_of(int64_t tokens, int topk, int64_t n) {
    const size_t choices = (size_t)tokens * (size_t)topk;
    return choices * (size_t)n * 4 + choices * (size_t)((n + 127) / 128) * 4;
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
    a.hi = static_cast<uint16_t*>(workspace);
    a.lo = a.hi + (size_t)choices * n;
    a.hs = reinterpret_cast<uint8_t*>(a.lo + (size_t)choices * n);
    a.hgroups = (int)((n + 127) / 128);
    a.out = static_cast<uint16_t*>(out_bf16);
    a.tiles = (choices + 7) / 8 < kMdTiles ? (choices + 7) / 8 : kMdTiles;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    constexpr size_t kMaxUp = 4 * (kMdWarps * kMdTiles * 128 + 1) * sizeof(float);
    constexpr size_t kMaxDown = (kMdWarps * 33 + kMdMaxCluster * 32) * FP8Q_MOE_DECODE_MAX_TOKENS * sizeof(float);
    static KernelCache up_cache, down_cache;
    int resident = 0;
    const size_t up_smem = std::max(sizeof(MdScratch), 4 * (size_t)(kMdWarps * a.tiles * 128 + 1) * sizeof(float));
    fp8q_status_t st = prepare_kernel(up_cache, moe_decode_up_kernel, kMdThreads, kMaxUp, kMaxUp, &resident);
    if (st != FP8Q_OK) return st;
    const int most = choices < experts ? choices : experts;         // chosen experts
    const unsigned up_blocks = grid_for((size_t)most * (size_t)(n / 32), 2);
    st = launch(moe_decode_up_kernel, up_blocks, kMdThreads, up_smem, s, a);
    if (st != FP8Q_OK) return st;
    unsigned ranks = 1;
    while (ranks < kMdMaxCluster && (int64_t)(k / 32) * ranks < 2 * sm_count() &&
           (int64_t)ranks * kMdWarps < (int64_t)most * a.hgroups)
        ranks *= 2;
    const size_t down_smem = std::max(sizeof(MdScratch), (size_t)(kMdWarps * 33 + ranks * 32) * tokens * sizeof(float));
    st = prepare_kernel(down_cache, moe_decode_down_kernel, kMdThreads, kMaxDown, kMaxDown, &resident);
    if (st != FP8Q_OK) return st;
    return launch_clusters(moe_decode_down_kernel, (unsigned)(k / 32) * ranks, ranks, kMdThreads, down_smem, s, a);
}
