// Tokens to their experts and back.
//
// A token t has topk choices; choice i = t * topk + j names expert ids[i].  A
// stable counting sort by expert gives every choice a slot, the experts' rows
// lying one after the other (offsets[e] .. offsets[e + 1]) and the choices of
// no expert (an id outside [0, experts)) last, from offsets[experts] on.
// Everything after the sort is done from the token's side, so that no sum
// needs atomics and every result is the same on every run:
//     gather            rows[slots[t, j]] = x[t]                 (zero rows for dropped choices)
//     combine           out[t] = sum over j of w[t, j] * y[slots[t, j]]
//     combine, backward dy[slots[t, j]] = w[t, j] * dout[t],  dw[t, j] = <dout[t], y[slots[t, j]]>
// and the gradient of gather is combine without weights.
//
// The sort is bound by latency (65,536 choices in two launches: 12.3 us with
// the launches' own time), the row movement by HBM.  8192 tokens to 8 of 128
// experts, rows of 2048:
//     gather   MXFP8 24.8 us back to back: 138 MB written at 5.6 TB/s (bulk
//              copies through shared memory and wider segments 26.7 to 29.4);
//              bf16 46.0 us, 6.6 TB/s
//     combine  47.9 us, 6.3 TB/s: 4 KB rows in random order (fourteen shapes of
//              warps, columns and rows in flight 50.3 to 53.4)
//     backward 86 us, 6.7 TB/s
#include "fp8q_device.cuh"
#include "fp8q_host.cuh"

namespace fp8q {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 32;

// ------------------------------------------------------------------ sort ----
// (One cluster of eight blocks instead of the two launches took 26.6 us against
// 16.4 then: all its scattered stores leave through eight SMs.)
// Blocks of kSortWarps warps own consecutive chunks of choices, and each warp
// a consecutive segment of its block's chunk, taken 32 choices at a time.  A
// choice's rank among equal keys is the number of equal keys in earlier
// blocks, in earlier warps of its block, in earlier steps of its warp and in
// lower lanes: a sum of counts, so the order is stable without any atomics.
constexpr int kSortWarps = 16;
constexpr int kSortThreads = kSortWarps * 32;
constexpr int kSortMaxBlocks = 128;

struct SortArgs {
    const void* ids;
    int id64;
    int64_t n;
    int64_t chunk;              // choices per block, a multiple of kSortThreads
    int experts;
    int* counts;                // [blocks][experts + 1], unused with one block
    int* offsets;               // [experts + 1]
    int* order;                 // [n]
    int* slots;                 // [n]
};

// Past the first-level cache: the placing launch may read the ids before its
// own dependency wait, which is what would make that cache's lines current.
__device__ __forceinline__ int sort_key(const SortArgs& a, int64_t i) {
    const int64_t id = a.id64 ? (int64_t)__ldcg(static_cast<const long long*>(a.ids) + i)
                              : (int64_t)__ldcg(static_cast<const int*>(a.ids) + i);
    return id >= 0 && id < a.experts ? (int)id : a.experts;
}

// hist[warp][key] = number of this warp's choices with that key.
__device__ __forceinline__ void warp_histogram(const SortArgs& a, int* hist, int64_t lo, int64_t hi) {
    const int lane = (int)(threadIdx.x & 31u);
    for (int64_t i = lo; i < hi; i += 32) {
        const bool ok = i + lane < hi;
        const int key = ok ? sort_key(a, i + lane) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, key);
        if (ok && (same & ((1u << lane) - 1u)) == 0) hist[key] += __popc(same);
        __syncwarp();
    }
}

__device__ __forceinline__ void segment_of(const SortArgs& a, int64_t* lo, int64_t* hi) {
    const int64_t seg = a.chunk / kSortWarps;
    const int64_t begin = (int64_t)blockIdx.x * a.chunk + (int64_t)(threadIdx.x >> 5) * seg;
    *lo = begin < a.n ? begin : a.n;
    *hi = begin + seg < a.n ? begin + seg : a.n;
}

__global__ void __launch_bounds__(kSortThreads) moe_sort_count_kernel(const SortArgs a) {
    extern __shared__ int hist_all[];
    const int keys = a.experts + 1;
    const int t = (int)threadIdx.x;
    for (int i = t; i < kSortWarps * keys; i += kSortThreads) hist_all[i] = 0;
    dependency_wait();
    allow_dependents();
    __syncthreads();
    int64_t lo, hi;
    segment_of(a, &lo, &hi);
    warp_histogram(a, hist_all + (t >> 5) * keys, lo, hi);
    __syncthreads();
    for (int e = t; e < keys; e += kSortThreads) {
        int s = 0;
        for (int w = 0; w < kSortWarps; ++w) s += hist_all[w * keys + e];
        a.counts[(int64_t)blockIdx.x * keys + e] = s;
    }
}

template <bool COUNTED>
__global__ void __launch_bounds__(kSortThreads) moe_sort_place_kernel(const SortArgs a) {
    extern __shared__ int hist_all[];                       // [kSortWarps][keys], then first[keys], behind[keys]
    __shared__ int warp_total[kSortWarps];
    const int keys = a.experts + 1;
    int* first = hist_all + kSortWarps * keys;              // total of each key, then its first slot in this block
    int* behind = first + keys;                             // the earlier blocks' choices of each key
    const int t = (int)threadIdx.x, lane = t & 31, warp = t >> 5;
    for (int i = t; i < kSortWarps * keys; i += kSortThreads) hist_all[i] = 0;
    // Behind the counting launch the ids may be read at once: its blocks let
    // this launch start only when whatever wrote the ids had completed.
    if (!COUNTED) dependency_wait();
    __syncthreads();
    int64_t lo, hi;
    segment_of(a, &lo, &hi);
    int* hist = hist_all + warp * keys;
    warp_histogram(a, hist, lo, hi);
    __syncthreads();
    // per key: the counts of this block's warps become their offsets inside
    // the key's run; `first` gets the key's total
    for (int e = t; e < keys; e += kSortThreads) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = hist_all[w * keys + e];
            hist_all[w * keys + e] = run;
            run += c;
        }
        first[e] = run;
        behind[e] = 0;
    }
    if (COUNTED) {
        dependency_wait();
        // four threads a key: each a quarter of the blocks' counts
        const int blocks = (int)gridDim.x, q = t & 3;
        __syncthreads();
        for (int e0 = 0; e0 < keys; e0 += kSortThreads / 4) {
            const int e = e0 + (t >> 2);
            int before = 0, total = 0;
            if (e < keys) {
#pragma unroll 8
                for (int b = q; b < blocks; b += 4) {
                    const int c = a.counts[(int64_t)b * keys + e];
                    before += b < (int)blockIdx.x ? c : 0;
                    total += c;
                }
            }
#pragma unroll
            for (int m = 1; m < 4; m <<= 1) {
                before += __shfl_xor_sync(0xFFFFFFFFu, before, m);
                total += __shfl_xor_sync(0xFFFFFFFFu, total, m);
            }
            if (e < keys && q == 0) {
                first[e] = total;
                behind[e] = before;
            }
        }
    }
    allow_dependents();
    __syncthreads();
    // exclusive scan of the totals: each thread a run of consecutive keys
    const int per = (keys + kSortThreads - 1) / kSortThreads;
    const int e0 = t * per, e1 = e0 + per < keys ? e0 + per : keys;
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += first[e];
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    int at = incl - mine;
    at += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? warp_total[lane] : 0);
    for (int e = e0; e < e1; ++e) {
        const int c = first[e];
        first[e] = at + behind[e];
        if (blockIdx.x == 0) a.offsets[e] = at;
        at += c;
    }
    __syncthreads();
    for (int64_t i = lo; i < hi; i += 32) {
        const bool ok = i + lane < hi;
        const int key = ok ? sort_key(a, i + lane) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, key);
        const unsigned below = same & ((1u << lane) - 1u);
        const int run = ok ? hist[key] : 0;
        __syncwarp();
        if (ok) {
            const int s = first[key] + run + __popc(below);
            a.slots[i + lane] = s;
            a.order[s] = (int)(i + lane);
            if (below == 0) hist[key] = run + __popc(same);
        }
        __syncwarp();
    }
}

// Blocks of 4 warps: their turnover hides better than that of 8 (us back to back: combine of 8192 x 8 rows of 2048
// 49.2 and 47.9, of 200,000 x 1 of 256 50.3 and 38.1).
constexpr int kRowWarps = 4;

// The work of this warp where `segments` warps in a row share one token (or
// group of tokens): divisions in 32 bits, as the blocks fit into them.
struct WarpUnit {
    int64_t t;
    int segment;
    __device__ __forceinline__ explicit WarpUnit(int segments) {
        const uint32_t s = (uint32_t)segments, warp = threadIdx.x >> 5;
        const uint32_t q = blockIdx.x / s, r = (blockIdx.x - q * s) * kRowWarps + warp;
        t = (int64_t)q * kRowWarps + r / s;
        segment = (int)(r % s);
    }
};

// ---------------------------------------------------------------- gather ----
// A warp copies one 2 KB segment of one token's row to the slots of all its
// choices: the row is read once however many experts take it.  Of short rows
// with one or two choices it copies two or four at once (us back to back, MXFP8:
// 200,000 x 1 rows of 256 71.9 -> 25.6, 65,536 x 2 of 512 30.5 -> 17.8; with
// four choices or more it makes no difference).  The second launch bound lets
// the compiler have the registers to keep all the loads ahead of the stores
// (8192 x 8 rows of 2048: 25.4 -> 24.8; 5329 x 8 of 928: 13.3 -> 10.8).
struct RowCopy {
    const uint8_t* src;
    uint8_t* dst;
    int64_t bytes;              // per row
};
struct GatherArgs {
    RowCopy main, extra;        // extra: the scale rows, or bytes == 0
    const int* slots;
    const int* routed;          // &offsets[experts]
    int64_t tokens;
    int topk;
    int segments;               // of 2 KB in a main row
};
constexpr int kSegBytes = 2048;

// Short rows (scales) of `tokens` tokens from t0 on: the lanes share out all their choices' pieces at once.
template <class T, bool ONE>
__device__ __forceinline__ void copy_short(const RowCopy& r, int64_t t0, int tokens, const int* slots, int topk, int routed,
                                           int64_t n) {
    const int lane = (int)(threadIdx.x & 31u);
    const int pieces = (int)(r.bytes / (int64_t)sizeof(T));
    for (int u = lane; u < pieces * tokens * topk; u += 32) {
        const int c = u / pieces, i = u - c * pieces;
        const int s = slots[t0 * topk + c];
        const int64_t t = t0 + (ONE ? 0 : c / topk);
        if (s >= 0 && s < n)
            reinterpret_cast<T*>(r.dst + (int64_t)s * r.bytes)[i] =
                s < routed ? reinterpret_cast<const T*>(r.src + t * r.bytes)[i] : T{};
    }
}

template <int G>
__global__ void __launch_bounds__(kRowWarps * 32, 1) moe_gather_kernel(const GatherArgs a) {
    constexpr int U = 4, P = U / G;             // 512-byte pieces of a warp, and of a token
    const int lane = (int)(threadIdx.x & 31u);
    const WarpUnit unit(a.segments);
    const int64_t t0 = unit.t * G;
    dependency_wait();
    allow_dependents();
    if (t0 >= a.tokens) return;
    const int64_t n = a.tokens * a.topk;
    const int routed = *a.routed;
    const int tokens = a.tokens - t0 < G ? (int)(a.tokens - t0) : G;
    const int slot = lane < tokens * a.topk ? a.slots[t0 * a.topk + lane] : -1;
    const int64_t col = (int64_t)unit.segment * kSegBytes + lane * 16;
    const uint8_t* src = a.main.src + t0 * a.main.bytes + col;
    uint4 v[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        ok[u] = u / P < tokens && col + (u % P) * 512 < a.main.bytes;
        if (ok[u]) v[u] = *reinterpret_cast<const uint4*>(src + (u / P) * a.main.bytes + (u % P) * 512);
    }
#pragma unroll 1
    for (int j = 0; j < a.topk; ++j) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int s = __shfl_sync(0xFFFFFFFFu, slot, (g * a.topk + j) & 31);
            if (g < tokens && s >= 0 && s < n) {
                uint8_t* dst = a.main.dst + (int64_t)s * a.main.bytes + col;
#pragma unroll
                for (int u = g * P; u < (g + 1) * P; ++u)
                    if (ok[u]) *reinterpret_cast<uint4*>(dst + (u % P) * 512) = s < routed ? v[u] : make_uint4(0, 0, 0, 0);
            }
        }
    }
    if (unit.segment == 0 && a.extra.bytes > 0) {
        if (a.extra.bytes % 16 == 0)
            copy_short<uint4, G == 1>(a.extra, t0, tokens, a.slots, a.topk, routed, n);
        else if (a.extra.bytes % 4 == 0)
            copy_short<uint32_t, G == 1>(a.extra, t0, tokens, a.slots, a.topk, routed, n);
        else
            copy_short<uint8_t, G == 1>(a.extra, t0, tokens, a.slots, a.topk, routed, n);
    }
}

// --------------------------------------------------------------- combine ----
struct CombineArgs {
    const uint16_t* y;
    const int* slots;
    const int* routed;
    const float* weights;       // or NULL: all 1
    uint16_t* out;
    int64_t tokens;
    int topk;
    int k;
    int segments;               // of 256 * C columns (see moe_combine_kernel)
};

// A warp sums 256 * C columns of one token, 8 / C choices at a time: eight
// 16-byte pieces per lane on their way, however few choices there are (us, with
// C = 1 always -> with the C of fp8q_moe_combine: 22,255 tokens of 1600 columns,
// one choice 79.8 -> 34.8; 12,000 of 2048, two choices 57.2 -> 32.8; 8,000 of
// 2048, four 45.0 -> 32.8; 8,192 of 2048, six or eight 51.2 and 55.3 either way).
// Of rows shorter than that it sums those of G tokens (200,000 x 1 of 256, back
// to back: 89.1 -> 38.5; 65,536 x 2 of 512 38.9 and 38.0).
template <int C, int G>
__global__ void __launch_bounds__(kRowWarps * 32) moe_combine_kernel(const CombineArgs a) {
    constexpr int U = 8 / (C * G);
    const int lane = (int)(threadIdx.x & 31u);
    const WarpUnit unit(a.segments);
    const int64_t t0 = unit.t * G;
    const int col0 = unit.segment * (256 * C) + lane * 8;
    dependency_wait();
    allow_dependents();
    if (t0 >= a.tokens) return;
    const int64_t n = a.tokens * a.topk;
    const int64_t routed = *a.routed < n ? *a.routed : n;
    int slot = -1;
    float w = 1.0f;
    if (lane < G * a.topk && t0 * a.topk + lane < n) {
        slot = a.slots[t0 * a.topk + lane];
        if (a.weights) w = a.weights[t0 * a.topk + lane];
    }
    float acc[G][C][8];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[g][c][i] = 0.0f;
    for (int j0 = 0; j0 < a.topk; j0 += U) {
        uint4 v[G][U][C];
        float wj[G][U];
        bool live[G][U][C];
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = __shfl_sync(0xFFFFFFFFu, slot, (g * a.topk + j0 + u) & 31);
                wj[g][u] = __shfl_sync(0xFFFFFFFFu, w, (g * a.topk + j0 + u) & 31);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    live[g][u][c] = j0 + u < a.topk && s >= 0 && s < routed && col0 + c * 256 < a.k;
                    if (live[g][u][c]) v[g][u][c] = ld_stream(a.y + (int64_t)s * a.k + col0 + c * 256);
                }
            }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (live[g][u][c]) {
                        float f[8];
                        unpack8(v[g][u][c], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[g][c][i] = __fmaf_rn(wj[g][u], f[i], acc[g][c][i]);
                    }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (t0 + g < a.tokens && col0 + c * 256 < a.k) {
                const float(&f)[8] = acc[g][c];
                st_stream(a.out + (t0 + g) * a.k + col0 + c * 256,
                          make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                     pack_bf16x2(f[6], f[7])));
            }
}

struct CombineGradArgs {
    const uint16_t* dout;
    const uint16_t* y;
    const int* slots;
    const int* routed;
    const float* weights;
    uint16_t* dy;
    float* dweights;
    int64_t tokens;
    int topk;
    int k;
};

// A warp takes NC choices at once: as many as it can hold whole rows of, for
// short rows, so that it always has four 16-byte pieces per lane on their way.
// A dot product is summed in the lanes and joined by shuffles, dy leaves as the
// row of y passes by.  The choices of a token are neighbours, so that its row
// of dout comes from the first-level cache for all but one of them.
template <int NC>
__global__ void __launch_bounds__(kRowWarps * 32) moe_combine_backward_kernel(const CombineGradArgs a) {
    constexpr int U = 4 / NC;                   // pieces of a row per lane and step
    const int lane = (int)(threadIdx.x & 31u);
    const int64_t i0 = ((int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5)) * NC;
    const int64_t n = a.tokens * a.topk;
    dependency_wait();
    allow_dependents();
    if (i0 >= n) return;
    const int routed = *a.routed;
    const uint16_t *drow[NC], *yrow[NC];
    uint16_t* orow[NC];
    bool inside[NC], live[NC];
    float w[NC], dot[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t i = i0 + c < n ? i0 + c : n - 1;
        const int s = a.slots[i];
        inside[c] = i0 + c < n && s >= 0 && s < n;
        live[c] = inside[c] && s < routed;
        w[c] = a.weights[i];
        drow[c] = a.dout + i / a.topk * a.k;
        yrow[c] = a.y + (int64_t)(live[c] ? s : 0) * a.k;
        orow[c] = a.dy + (int64_t)(inside[c] ? s : 0) * a.k;
        dot[c] = 0.0f;
    }
    for (int c0 = lane * 8; c0 < a.k; c0 += 256 * U) {
        uint4 d[NC][U], y[NC][U];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int col = c0 + u * 256;
                d[c][u] = y[c][u] = make_uint4(0, 0, 0, 0);
                if (live[c] && col < a.k) {
                    d[c][u] = *reinterpret_cast<const uint4*>(drow[c] + col);
                    y[c][u] = ld_stream(yrow[c] + col);
                }
            }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int col = c0 + u * 256;
                float fd[8], fy[8];
                unpack8(d[c][u], fd);
                unpack8(y[c][u], fy);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot[c] = __fmaf_rn(fd[e], fy[e], dot[c]);
                    fd[e] = __fmul_rn(fd[e], w[c]);
                }
                if (inside[c] && col < a.k)
                    st_stream(orow[c] + col, live[c] ? make_uint4(pack_bf16x2(fd[0], fd[1]), pack_bf16x2(fd[2], fd[3]),
                                                                  pack_bf16x2(fd[4], fd[5]), pack_bf16x2(fd[6], fd[7]))
                                                     : make_uint4(0, 0, 0, 0));
            }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) dot[c] += __shfl_xor_sync(0xFFFFFFFFu, dot[c], m);
        if (lane == 0 && i0 + c < n) a.dweights[i0 + c] = dot[c];
    }
}

// Choices per sort block, and the number of blocks.
static int64_t sort_chunk(int64_t n, int64_t* blocks) {
    // one block up to 4 choices per thread; then blocks of 2 per thread while kSortMaxBlocks of them are enough
    int64_t chunk = n <= 4 * kSortThreads ? 4 * kSortThreads : 2 * kSortThreads;
    while ((n + chunk - 1) / chunk > kSortMaxBlocks) chunk *= 2;
    *blocks = (n + chunk - 1) / chunk;
    return chunk;
}

// The checks that all the routed operators share.
static fp8q_status_t route_sizes(int64_t tokens, int topk, int experts) {
    if (tokens < 0 || experts < 1 || experts > kMaxExperts) return FP8Q_ERR_SIZE;
    if (topk < 1 || topk > kMaxTopk) return FP8Q_ERR_K;
    if (tokens > ((int64_t)1 << 31) / topk - 1) return FP8Q_ERR_SIZE;
    return FP8Q_OK;
}

static fp8q_status_t row_sizes(int64_t tokens, int topk, int experts, int64_t k, int64_t multiple) {
    const fp8q_status_t st = route_sizes(tokens, topk, experts);
    if (st != FP8Q_OK) return st;
    if (k <= 0 || k % multiple != 0) return FP8Q_ERR_K;
    if (k > ((int64_t)1 << 30) || (tokens > 0 && (uint64_t)k > FP8Q_MAX_ELEMENTS / (uint64_t)(tokens * topk)))
        return FP8Q_ERR_SIZE;
    return FP8Q_OK;
}

template <int N>
static bool all_aligned(const void* const (&p)[N]) {
    for (const void* q : p)
        if (!aligned16(q)) return false;
    return true;
}

static fp8q_status_t units_grid(int64_t units, unsigned* grid) {
    const int64_t g = (units + kRowWarps - 1) / kRowWarps;
    if (g > 0x7FFFFFFF) return FP8Q_ERR_SIZE;
    *grid = (unsigned)g;
    return FP8Q_OK;
}

}  // namespace fp8q

using namespace fp8q;

extern "C" size_t fp8q_moe_sort_workspace_bytes(int64_t tokens, int topk, int experts) {
    if (route_sizes(tokens, topk, experts) != FP8Q_OK) return 0;
    int64_t blocks;
    sort_chunk(tokens * topk, &blocks);
    return blocks > 1 ? (size_t)blocks * (size_t)(experts + 1) * sizeof(int) : 0;
}

extern "C" fp8q_status_t fp8q_moe_sort(const void* ids, int id_bytes, int64_t tokens, int topk, int experts,
                                       int32_t* offsets, int32_t* order, int32_t* slots, void* workspace,
                                       size_t workspace_bytes, fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_moe_sort");
    if (id_bytes != 4 && id_bytes != 8) return FP8Q_ERR_FORMAT;
    const fp8q_status_t st = route_sizes(tokens, topk, experts);
    if (st != FP8Q_OK) return st;
    const int64_t n = tokens * topk;
    const size_t need = fp8q_moe_sort_workspace_bytes(tokens, topk, experts);
    if (!offsets || (n > 0 && (!ids || !order || !slots)) || (need > 0 && !workspace)) return FP8Q_ERR_NULL;
    if (workspace_bytes < need) return FP8Q_ERR_SIZE;
    const void* const all[] = {ids, offsets, order, slots, workspace};
    if (!all_aligned(all)) return FP8Q_ERR_ALIGN;
    const Range in = {ids, (size_t)n * id_bytes};
    const Range outs[] = {{offsets, 4 * (size_t)(experts + 1)}, {order, 4 * (size_t)n}, {slots, 4 * (size_t)n}, {workspace, need}};
    if (any_alias(outs, 4, &in, 1)) return FP8Q_ERR_ALIAS;
    int64_t blocks;
    const int64_t chunk = sort_chunk(n, &blocks);
    const SortArgs a = {ids, id_bytes == 8, n, chunk, experts, static_cast<int*>(workspace), offsets, order, slots};
    const size_t most = (size_t)(kSortWarps + 2) * (kMaxExperts + 1) * sizeof(int);
    const size_t smem = (size_t)(kSortWarps + 2) * (experts + 1) * sizeof(int);
    static KernelCache kc1, kc2, kc3;
    int resident = 0;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    fp8q_status_t s;
    if (blocks <= 1) {
        s = prepare_kernel(kc1, moe_sort_place_kernel<false>, kSortThreads, most, most, &resident);
        return s != FP8Q_OK ? s : launch(moe_sort_place_kernel<false>, 1, kSortThreads, smem, cs, a);
    }
    s = prepare_kernel(kc2, moe_sort_count_kernel, kSortThreads, most, most, &resident);
    if (s == FP8Q_OK) s = launch(moe_sort_count_kernel, (unsigned)blocks, kSortThreads, smem, cs, a);
    if (s == FP8Q_OK) s = prepare_kernel(kc3, moe_sort_place_kernel<true>, kSortThreads, most, most, &resident);
    return s != FP8Q_OK ? s : launch(moe_sort_place_kernel<true>, (unsigned)blocks, kSortThreads, smem, cs, a);
}

namespace fp8q {

static fp8q_status_t gather_launch(GatherArgs a, int experts, cudaStream_t stream) {
    const int64_t n = a.tokens * a.topk;
    if (!a.main.src || !a.main.dst || !a.slots || !a.routed || (a.extra.bytes > 0 && (!a.extra.src || !a.extra.dst)))
        return FP8Q_ERR_NULL;
    const void* const all[] = {a.main.src, a.main.dst, a.extra.src, a.extra.dst, a.slots, a.routed};
    if (!all_aligned(all)) return FP8Q_ERR_ALIGN;
    const Range ins[] = {{a.main.src, (size_t)(a.tokens * a.main.bytes)}, {a.extra.src, (size_t)(a.tokens * a.extra.bytes)},
                         {a.slots, 4 * (size_t)n}, {a.routed, 4 * (size_t)(experts + 1)}};
    const Range outs[] = {{a.main.dst, (size_t)(n * a.main.bytes)}, {a.extra.dst, (size_t)(n * a.extra.bytes)}};
    if (any_alias(outs, 2, ins, 4)) return FP8Q_ERR_ALIAS;
    a.routed += experts;
    a.segments = (int)((a.main.bytes + kSegBytes - 1) / kSegBytes);
    // as many tokens per warp as its lanes hold rows and slots of
    const int group = a.topk > 2 ? 1 : a.main.bytes <= kSegBytes / 4 ? 4 : a.main.bytes <= kSegBytes / 2 ? 2 : 1;
    unsigned grid;
    const fp8q_status_t st = units_grid((a.tokens + group - 1) / group * a.segments, &grid);
    if (st != FP8Q_OK) return st;
    return launch(group == 4 ? moe_gather_kernel<4> : group == 2 ? moe_gather_kernel<2> : moe_gather_kernel<1>, grid,
                  kRowWarps * 32, 0, stream, a);
}

}  // namespace fp8q

extern "C" fp8q_status_t fp8q_moe_gather(const void* x_bf16, const int32_t* slots, const int32_t* offsets,
                                         int64_t tokens, int topk, int experts, int64_t k, void* rows_bf16,
                                         fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_moe_gather");
    const fp8q_status_t st = row_sizes(tokens, topk, experts, k, 8);
    if (st != FP8Q_OK || tokens == 0) return st;
    GatherArgs a = {};
    a.main = {static_cast<const uint8_t*>(x_bf16), static_cast<uint8_t*>(rows_bf16), 2 * k};
    a.slots = slots;
    a.routed = offsets;
    a.tokens = tokens;
    a.topk = topk;
    return gather_launch(a, experts, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" fp8q_status_t mxfp8_moe_gather(const uint8_t* codes, const uint8_t* scales, const int32_t* slots,
                                          const int32_t* offsets, int64_t tokens, int topk, int experts, int64_t k,
                                          uint8_t* row_codes, uint8_t* row_scales, fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("mxfp8_moe_gather");
    const fp8q_status_t st = row_sizes(tokens, topk, experts, k, MXFP8_BLOCK);
    if (st != FP8Q_OK || tokens == 0) return st;
    GatherArgs a = {};
    a.main = {codes, row_codes, k};
    a.extra = {scales, row_scales, k / MXFP8_BLOCK};
    a.slots = slots;
    a.routed = offsets;
    a.tokens = tokens;
    a.topk = topk;
    return gather_launch(a, experts, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" fp8q_status_t fp8q_moe_combine(const void* y_bf16, const int32_t* slots, const int32_t* offsets,
                                          const float* weights, int64_t tokens, int topk, int experts, int64_t k,
                                          void* out_bf16, fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_moe_combine");
    const fp8q_status_t st = row_sizes(tokens, topk, experts, k, 8);
    if (st != FP8Q_OK || tokens == 0) return st;
    if (!y_bf16 || !slots || !offsets || !out_bf16) return FP8Q_ERR_NULL;
    const void* const all[] = {y_bf16, slots, offsets, weights, out_bf16};
    if (!all_aligned(all)) return FP8Q_ERR_ALIGN;
    const size_t n = (size_t)(tokens * topk);
    const Range ins[] = {{y_bf16, 2 * n * (size_t)k}, {slots, 4 * n}, {offsets, 4 * (size_t)(experts + 1)}, {weights, 4 * n}};
    const Range out = {out_bf16, 2 * (size_t)(tokens * k)};
    if (any_alias(&out, 1, ins, 4)) return FP8Q_ERR_ALIAS;
    const int pieces = topk <= 1 ? 8 : topk <= 2 ? 4 : topk <= 4 ? 2 : 1;      // C * G: all choices at once if topk <= 8
    int wide = pieces;
    while (wide > 1 && (wide / 2) * 256 >= k) wide /= 2;
    const int group = pieces / wide;
    const int segments = (int)((k + 256 * wide - 1) / (256 * wide));
    unsigned grid;
    const fp8q_status_t sg = units_grid((tokens + group - 1) / group * segments, &grid);
    if (sg != FP8Q_OK) return sg;
    const CombineArgs a = {static_cast<const uint16_t*>(y_bf16), slots, offsets + experts, weights,
                           static_cast<uint16_t*>(out_bf16), tokens, topk, (int)k, segments};
    void (*kernel)(const CombineArgs) = moe_combine_kernel<1, 1>;
    switch (pieces * 16 + wide) {
        case 8 * 16 + 8: kernel = moe_combine_kernel<8, 1>; break;
        case 8 * 16 + 4: kernel = moe_combine_kernel<4, 2>; break;
        case 8 * 16 + 2: kernel = moe_combine_kernel<2, 4>; break;
        case 8 * 16 + 1: kernel = moe_combine_kernel<1, 8>; break;
        case 4 * 16 + 4: kernel = moe_combine_kernel<4, 1>; break;
        case 4 * 16 + 2: kernel = moe_combine_kernel<2, 2>; break;
        case 4 * 16 + 1: kernel = moe_combine_kernel<1, 4>; break;
        case 2 * 16 + 2: kernel = moe_combine_kernel<2, 1>; break;
        case 2 * 16 + 1: kernel = moe_combine_kernel<1, 2>; break;
    }
    return launch(kernel, grid, kRowWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream), a);
}

extern "C" fp8q_status_t fp8q_moe_combine_backward(const void* dout_bf16, const void* y_bf16, const int32_t* slots,
                                                   const int32_t* offsets, const float* weights, int64_t tokens,
                                                   int topk, int experts, int64_t k, void* dy_bf16, float* dweights,
                                                   fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_moe_combine_backward");
    const fp8q_status_t st = row_sizes(tokens, topk, experts, k, 8);
    if (st != FP8Q_OK || tokens == 0) return st;
    if (!dout_bf16 || !y_bf16 || !slots || !offsets || !weights || !dy_bf16 || !dweights) return FP8Q_ERR_NULL;
    const void* const all[] = {dout_bf16, y_bf16, slots, offsets, weights, dy_bf16, dweights};
    if (!all_aligned(all)) return FP8Q_ERR_ALIGN;
    const size_t n = (size_t)(tokens * topk);
    const Range ins[] = {{dout_bf16, 2 * (size_t)(tokens * k)}, {y_bf16, 2 * n * (size_t)k}, {slots, 4 * n},
                         {offsets, 4 * (size_t)(experts + 1)}, {weights, 4 * n}};
    const Range outs[] = {{dy_bf16, 2 * n * (size_t)k}, {dweights, 4 * n}};
    if (any_alias(outs, 2, ins, 5)) return FP8Q_ERR_ALIAS;
    unsigned grid;
    const int per = k <= 256 ? 4 : k <= 512 ? 2 : 1;
    const fp8q_status_t sg = units_grid((tokens * topk + per - 1) / per, &grid);
    if (sg != FP8Q_OK) return sg;
    const CombineGradArgs a = {static_cast<const uint16_t*>(dout_bf16), static_cast<const uint16_t*>(y_bf16), slots,
                               offsets + experts, weights, static_cast<uint16_t*>(dy_bf16), dweights, tokens, topk, (int)k};
    return launch(per == 4   ? moe_combine_backward_kernel<4>
                  : per == 2 ? moe_combine_backward_kernel<2>
                             : moe_combine_backward_kernel<1>, grid, kRowWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream), a);
}
