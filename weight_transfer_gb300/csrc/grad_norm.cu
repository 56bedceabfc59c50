// The global norm of many gradient tensors, and the gradients clipped by it.
//
//     norm = scale * sqrt(sum of x^2 over all tensors),  coefficient = min(1, max_norm / (norm + 1e-6))
//     out = x * (scale * coefficient)
// The tensors are cut into chunks of a fixed number of bytes; a block sums one
// chunk's squares into its place of the workspace, and a single block joins the
// places in their order, so that the norm does not depend on timing.
// The table of tensors travels in the kernel's parameters, kGradGroup at a
// time: nothing is copied to the device ahead of the launch, and a captured
// graph keeps the table with its node.
//
// A thread sums 64 squares in binary32, in eight chains, a warp its threads'
// sums, and everything above is binary64 (of which this GPU does two additions
// a cycle and SM).  A warp's sum outside [2^-80, 2^100] would lose squares to the
// range of binary32; its elements are squared again under a power of two.
//
// Both passes are bound by HBM.  A layer of 623 million bf16 gradients takes 179 to
// 182 us for its norm (6.85 TB/s; blocks of 256 threads that each read one chunk
// into registers took 294 to 317).  Eight buckets of 13.1 million, averaged and
// clipped into others, 100 us in calls on other buffers than the last one's, 95.6
// from a graph on the same ones: the second reading finds some 40 MB in the
// second-level cache.  A thousand ragged views into 32-bit buffers, 99.6 and 97 us,
// as the copies into shared memory leave the output its own alignment (element by
// element 188).  Fourteen small tensors: 4.8 us in two launches of a graph (5.2
// where the first chunk was looked up behind the dependency wait).
#include "fp8q_device.cuh"
#include "fp8q_host.cuh"

#include <math.h>

#include <algorithm>
#include <type_traits>

namespace fp8q {

constexpr int kGradGroup = 1024;            // tensors per launch
constexpr int kGradFew = 64;                // a launch of no more has a smaller table
constexpr int kGradThreads = 256;
constexpr int kPiece = 32768;               // bytes of one copy
constexpr int kStages = 5;
constexpr uint64_t kGradMaxChunks = 4096;   // chunks grow from one piece so that there are not many more than this
constexpr int kJoinThreads = 256;
constexpr uint32_t kNear = 16;               // 8 and 32 take as long

// Element types and count share a word: count in the low 44 bits.
struct GradItem {
    const void* grad;
    void* out;
    uint64_t kind;
};
template <int N> struct GradTableN {
    static constexpr int kSize = N;
    GradItem item[N];
    uint32_t first[N + 1];                  // chunks of the group's earlier tensors
    // The tensor of every 16th chunk, and the last tensor, between which a look-up searches.  It reads the parameters
    // one after the other, 300 cycles for each line that is not at hand: 2200 cycles a chunk among a thousand ragged
    // views without these and with an item's members apart, 1400 as it is (clip_ragged 103 and 98.4 us).  A small
    // table needs none.
    uint16_t near[N > kGradFew ? (kGradMaxChunks + 1 + N) / kNear + 2 : 1];
    int count;
};
using GradTable = GradTableN<kGradGroup>;
static_assert(sizeof(GradTable) + 64 <= 32764, "a kernel's parameters");
constexpr uint64_t kCountMask = (1ull << 44) - 1;
constexpr uint64_t kGradF32 = 1ull << 62, kOutF32 = 1ull << 63;

template <int N> __device__ __forceinline__ int tensor_of(const GradTableN<N>& t, uint32_t chunk) {
    int lo = 0, hi = t.count - 1;
    if (N > kGradFew) lo = t.near[chunk / kNear], hi = t.near[chunk / kNear + 1];
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <int BYTES> __device__ __forceinline__ float load_grad(const void* p, int64_t i) {
    return BYTES == 2 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}

// Sum of the squares of a thread's vectors tid, tid + kGradThreads, ... of a
// piece, in eight chains of binary32 (up to 64 squares); SCALED: of the elements
// times `factor`, a power of two.
template <int BYTES, bool SCALED = false> __device__ __forceinline__ float squares(const uint4* piece, int vecs, float factor = 1.0f) {
    constexpr int kLoads = kPiece / 16 / kGradThreads;
    const uint64_t factors = f2_pack(factor, factor);
    uint64_t s[4] = {0, 0, 0, 0};
    uint4 v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
        const int i = (int)threadIdx.x + u * kGradThreads;
        v[u] = i < vecs ? piece[i] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        if (BYTES == 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint64_t x = f2_pack(bf16_lo(w[j]), bf16_hi(w[j]));
                if (SCALED) x = f2_mul(x, factors);
                s[j] = f2_fma(x, x, s[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint64_t x = f2_pack(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
                if (SCALED) x = f2_mul(x, factors);
                s[(u & 1) * 2 + j] = f2_fma(x, x, s[(u & 1) * 2 + j]);
            }
        }
    }
    float a, b;
    f2_unpack(f2_add(f2_add(s[0], s[1]), f2_add(s[2], s[3])), a, b);
    return a + b;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// A warp's sum of its vectors' squares, where binary32 loses some of them.
// Below 2^-80 all elements are below 2^-40, and times 2^86 the smallest still
// has a square of 2^-126; otherwise the elements go times 2^-70, where even 2048
// of the largest stay below 2^127, and squares that vanish have no weight beside
// one above 2^89.
template <int BYTES> __device__ __noinline__ double scaled_squares(const uint4* piece, int vecs, bool small) {
    const float v = warp_sum(squares<BYTES, true>(piece, vecs, small ? 0x1p86f : 0x1p-70f));
    return (double)v * (small ? 0x1p-172 : 0x1p140);
}

// A warp's sum of its vectors' squares.  Up to 2048 squares that vanish, or keep
// few bits, are off by 2^-150 each, which does not count beside 2^-80.  (64 Mi bf16
// gradients of 1e-14: 35 us, of 1e-3 27; with binary64 squares 408.)
template <int BYTES> __device__ __forceinline__ double piece_squares(const uint4* piece, int vecs) {
    const float v = squares<BYTES>(piece, vecs);
    const bool within = __all_sync(0xFFFFFFFFu, v <= 0x1p100f);     // a NaN is not
    const float sum = warp_sum(v);
    return within && sum >= 0x1p-80f ? (double)sum : scaled_squares<BYTES>(piece, vecs, within);
}

// The eviction priority in the second-level cache of what nothing reads again, and
// bulk_g2s with one.
__device__ __forceinline__ uint64_t evict_first() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void bulk_g2s_hint(void* smem_dst, const void* gmem_src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_addr(smem_dst)),
        "l"(gmem_src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// Where a chunk lies: `vecs` whole vectors from `from` on, element `first` of
// its tensor; `head` elements in front of the tensor's vectors and `tails`
// behind them, from element `tail` on, are in the care of its first and its last
// chunk.
struct Place {
    const unsigned char* from;
    const void* grad;
    void* out;
    int64_t first, vecs, tail;
    int f32, out32, head, tails;
};
template <int N> __device__ __forceinline__ Place locate(const GradTableN<N>& t, uint32_t chunk, int64_t chunk_bytes) {
    Place r;
    const int i = tensor_of(t, chunk);
    const uint64_t kind = t.item[i].kind;
    const uint32_t begin = t.first[i], end = t.first[i + 1];
    r.grad = t.item[i].grad;
    r.out = t.item[i].out;
    r.f32 = (kind & kGradF32) != 0;
    r.out32 = (kind & kOutF32) != 0;
    const int shift = r.f32 ? 2 : 1, per = 16 >> shift;
    const int64_t n = (int64_t)(kind & kCountMask), index = chunk - begin, most = chunk_bytes / 16;
    const unsigned char* p = static_cast<const unsigned char*>(r.grad);
    const int64_t to = (int64_t)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) >> shift;
    const int64_t head = to < n ? to : n, all = (n - head) >> (4 - shift);
    r.vecs = all - index * most < most ? all - index * most : most;
    if (r.vecs < 0) r.vecs = 0;                         // a last chunk of nothing but elements behind the vectors
    r.first = head + index * most * per;
    r.from = p + (r.first << shift);
    r.head = index == 0 ? (int)head : 0;
    r.tails = chunk + 1 == end ? (int)(n - head - all * per) : 0;
    r.tail = n - r.tails;
    return r;
}

// What the copying warp tells the summing ones about a stage.
struct Piece {
    const void* tensor;         // for the elements outside the vectors
    int64_t tail;               // where those behind them start
    int head, tails;            // how many there are in front and behind, in this piece's care
    int vecs;                   // -1: no more pieces
    int f32, last;              // last piece of its chunk
};

// Before the block's shared memory is given up: lets the copies land that were
// issued before stage s in the ring's current turn, but for those of stage
// `taken`, which the summing warps have had.
__device__ __noinline__ void land(uint64_t* full, uint32_t round, int s, int taken = -1) {
    for (int i = 0; i < kStages; ++i)
        if (i != taken && (i < s || round > 0)) mbar_wait(&full[i], (i < s ? round : round - 1) & 1);
}

// One block per SM walks over the chunks.  A warp of its own copies them, 32 KB
// at a time, into a ring of stages; eight warps sum.  A warp's sum of a chunk
// waits in the chunk's last stage, where the copying warp joins the eight when
// it takes the stage back.
template <int N>
__global__ void __launch_bounds__(kGradThreads + 32, 1) grad_squares_kernel(const __grid_constant__ GradTableN<N> t, uint32_t chunks,
                                                                            uint32_t kept, int64_t chunk_bytes, double* partial) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ Piece info[kStages];
    __shared__ double sums[kStages][kGradThreads / 32];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kGradThreads / 32);
        }
        fence_barrier_init();
    }
    __syncthreads();
    Place at;
    if (warp == kGradThreads / 32) at = locate(t, blockIdx.x, chunk_bytes);     // parameters need no wait
    dependency_wait();
    allow_dependents();
    if (warp == kGradThreads / 32) {
        if (lane != 0) return;
        const uint64_t drop = evict_first();
        int64_t chunk_of[kStages];                      // chunk that a stage ends, or -1
#pragma unroll
        for (int s = 0; s < kStages; ++s) chunk_of[s] = -1;
        uint32_t round = 0;                             // of the ring
        int s = 0;
        // Takes a stage back from the summing warps and stores the sum of the chunk that it ended.
        auto take = [&]() -> bool {
            if (round == 0) return true;
            if (!mbar_wait(&empty[s], (round - 1) & 1)) {
                raise_error(kErrCopyTimeout);
                return false;
            }
            int64_t done = -1;
#pragma unroll
            for (int i = 0; i < kStages; ++i)
                if (i == s) done = chunk_of[i];
            if (done >= 0) {
                double v[kGradThreads / 32];
                for (int w = 0; w < kGradThreads / 32; ++w) v[w] = sums[s][w];
#pragma unroll
                for (int n = kGradThreads / 64; n > 0; n /= 2)
#pragma unroll
                    for (int w = 0; w < n; ++w) v[w] += v[w + n];
                partial[done] = v[0];
            }
            return true;
        };
        auto next = [&](int64_t ends) {
#pragma unroll
            for (int i = 0; i < kStages; ++i)
                if (i == s) chunk_of[i] = ends;
            if (++s == kStages) s = 0, ++round;
        };
        for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
            if (c != blockIdx.x) at = locate(t, c, chunk_bytes);
            int64_t left = at.vecs;
            const unsigned char* from = at.from;
            for (bool first = true; first || left > 0; first = false) {
                const int v = (int)(left < kPiece / 16 ? left : kPiece / 16);
                left -= v;
                if (!take()) return land(full, round, s);
                info[s] = {at.grad, at.tail, first ? at.head : 0, left == 0 ? at.tails : 0, v, at.f32, left == 0};
                mbar_arrive_expect_tx(&full[s], (uint32_t)v * 16);
                if (v && c >= kept) bulk_g2s(ring + s * kPiece, from, (uint32_t)v * 16, &full[s]);
                else if (v) bulk_g2s_hint(ring + s * kPiece, from, (uint32_t)v * 16, &full[s], drop);
                from += (int64_t)v * 16;
                next(left == 0 ? (int64_t)c : -1);
            }
        }
        if (!take()) return land(full, round, s);
        info[s].vecs = -1;
        mbar_arrive_expect_tx(&full[s], 0);
        const uint32_t end_round = round;
        const int end = s;
        for (int i = 1; i < kStages; ++i) {             // the stages still on their way
            next(-1);
            if (!take()) return land(full, end_round, end, end);
        }
        return;
    }
    double sum = 0.0;                                   // lane 0: of the chunk so far
    uint32_t parity = 0;
    for (int s = 0;;) {
        if (!mbar_wait(&full[s], parity)) {
            if (lane == 0) raise_error(kErrCopyTimeout);
            return;
        }
        const Piece m = info[s];
        if (m.vecs < 0) return;
        const uint4* piece = reinterpret_cast<const uint4*>(ring + s * kPiece);
        sum += m.f32 ? piece_squares<4>(piece, m.vecs) : piece_squares<2>(piece, m.vecs);
        if (warp == 0 && m.head + m.tails > 0) {        // up to 7 on either side, one for a lane
            const int64_t at = lane < m.head ? lane : m.tail + (lane - m.head);
            double d = 0.0;
            if (lane < m.head + m.tails) d = (double)(m.f32 ? load_grad<4>(m.tensor, at) : load_grad<2>(m.tensor, at));
            sum += warp_sum(d * d);
        }
        __syncwarp();                                   // every lane is through with the stage
        if (lane == 0) {
            if (m.last) {
                sums[s][warp] = sum;
                sum = 0.0;
            }
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty[s])) : "memory");
        }
        if (++s == kStages) s = 0, parity ^= 1;
    }
}

struct JoinArgs {
    const double* partial;      // all chunks
    uint64_t chunks;
    double scale, max_norm;
    float* norm;                // [2], or NULL: another launch joins them
    const double* group;        // this group's chunks
    float* each;                // of this group, or NULL
};

// The first block joins all chunks, a warp of the others one tensor's.
template <int N> __global__ void __launch_bounds__(kJoinThreads) grad_join_kernel(const __grid_constant__ GradTableN<N> t, const JoinArgs a) {
    __shared__ double sh[kJoinThreads / 32];
    const int lane = (int)(threadIdx.x & 31u), warp = (int)(threadIdx.x >> 5);
    dependency_wait();
    allow_dependents();
    if (blockIdx.x > 0) {
        const int i = (int)(blockIdx.x - 1) * (kJoinThreads / 32) + warp;
        if (i >= t.count) return;
        double v = 0.0;
#pragma unroll 8
        for (uint32_t c = t.first[i] + (uint32_t)lane; c < t.first[i + 1]; c += 32) v += __ldcg(a.group + c);
        v = warp_sum(v);
        if (lane == 0) a.each[i] = (float)(sqrt(v) * a.scale);
        return;
    }
    if (!a.norm) return;
    double v = 0.0;
#pragma unroll 16
    for (uint64_t i = threadIdx.x; i < a.chunks; i += kJoinThreads) v += __ldcg(a.partial + i);
    v = warp_sum(v);
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        double sum = 0.0;
        for (int w = 0; w < kJoinThreads / 32; ++w) sum += sh[w];
        const double norm = sqrt(sum) * a.scale;
        const double ratio = a.max_norm / (norm + 1e-6);
        a.norm[0] = (float)norm;
        a.norm[1] = ratio >= 1.0 ? 1.0f : (float)ratio;     // a NaN stays one
    }
}

template <int BYTES> __device__ __forceinline__ void store_grad(void* q, int64_t i, float x) {
    if (BYTES == 2) static_cast<uint16_t*>(q)[i] = (uint16_t)pack_bf16x2(x, 0.0f);
    else static_cast<float*>(q)[i] = x;
}

// What the copying warp tells the scaling ones about a stage.
struct ScalePiece {
    const void* grad;           // for the elements outside the vectors
    void* out;
    int64_t first, tail;        // the first element of the vectors, and of those behind them
    int head, tails;
    int vecs;                   // -1: no more pieces
    int kind;                   // 2 * f32 of the input + f32 of the output
};

// `count` elements from shared memory, times f, to out: whole vectors of the
// output, single elements on either side of them.
template <int IN, int OUT> __device__ __forceinline__ void scale_piece(const unsigned char* in, void* out, int64_t first, int count, float f) {
    constexpr int OV = 16 / OUT;
    const int tid = (int)threadIdx.x;
    unsigned char* q = static_cast<unsigned char*>(out) + first * OUT;
    int head = (int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(q) & 15u)) & 15u) / OUT;
    if (head > count) head = count;
    const int vecs = (count - head) / OV, tail = head + vecs * OV;
    const unsigned char* body = in + head * IN;
    const bool whole = (head * IN) % (OV * IN < 16 ? OV * IN : 16) == 0;    // the elements of a vector lie in vectors of the input
#pragma unroll 4
    for (int i = tid; i < vecs; i += kGradThreads) {
        float x[OV];
        const unsigned char* p = body + i * (OV * IN);
        if (whole) {
            if constexpr (OV * IN == 8) {
                const uint2 v = *reinterpret_cast<const uint2*>(p);
                x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
            } else if constexpr (IN == 2) {
                unpack8(*reinterpret_cast<const uint4*>(p), x);
            } else {
#pragma unroll
                for (int j = 0; j < OV; j += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(p + j * 4);
                    x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < OV; ++j) x[j] = load_grad<IN>(p, j);
        }
#pragma unroll
        for (int j = 0; j < OV; ++j) x[j] *= f;
        uint4 v;
        if constexpr (OUT == 2)
            v = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        else
            v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        st_stream(q + (int64_t)(head + i * OV) * OUT, v);
    }
    if (tid < head) store_grad<OUT>(q, tid, load_grad<IN>(in, tid) * f);
    if (tid < count - tail) store_grad<OUT>(q, tail + tid, load_grad<IN>(in, tail + tid) * f);
}
template <int IN, int OUT> __device__ __forceinline__ void scale_stage(const unsigned char* stage, const ScalePiece& m, float f) {
    scale_piece<IN, OUT>(stage, m.out, m.first, m.vecs * (16 / IN), f);
    const int lane = (int)threadIdx.x;                  // up to 7 elements on either side of the vectors
    if (lane < m.head + m.tails) {
        const int64_t at = lane < m.head ? lane : m.tail + (lane - m.head);
        store_grad<OUT>(m.out, at, load_grad<IN>(m.grad, at) * f);
    }
}

// As the sums: one block per SM, a copying warp and eight that scale.  The
// chunks backwards: what the sums read last is still in the second-level cache.
// Reading through shared memory lets the output have its own alignment.
template <int N>
__global__ void __launch_bounds__(kGradThreads + 32, 1) grad_scale_kernel(const __grid_constant__ GradTableN<N> t, uint32_t chunks,
                                                                          int64_t chunk_bytes, double scale, const float* norm) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ ScalePiece info[kStages];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kGradThreads / 32);
        }
        fence_barrier_init();
    }
    __syncthreads();
    Place at;
    if (warp == kGradThreads / 32) at = locate(t, chunks - 1 - blockIdx.x, chunk_bytes);
    dependency_wait();
    allow_dependents();
    const float f = (float)(scale * (double)__ldcg(norm + 1));
    if (warp == kGradThreads / 32) {
        if (lane != 0) return;
        const uint64_t drop = evict_first();
        uint32_t round = 0;                             // of the ring
        int s = 0;
        auto take = [&]() -> bool {
            if (round == 0 || mbar_wait(&empty[s], (round - 1) & 1)) return true;
            raise_error(kErrCopyTimeout);
            return false;
        };
        for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
            if (c != blockIdx.x) at = locate(t, chunks - 1 - c, chunk_bytes);
            if (f == 1.0f && at.out == at.grad) continue;                   // in place and unchanged
            int64_t left = at.vecs, element = at.first;
            const unsigned char* from = at.from;
            for (bool first = true; first || left > 0; first = false) {
                const int v = (int)(left < kPiece / 16 ? left : kPiece / 16);
                left -= v;
                if (!take()) return land(full, round, s);
                info[s] = {at.grad, at.out, element, at.tail, first ? at.head : 0, left == 0 ? at.tails : 0, v,
                           2 * at.f32 + at.out32};
                mbar_arrive_expect_tx(&full[s], (uint32_t)v * 16);
                if (v) bulk_g2s_hint(ring + s * kPiece, from, (uint32_t)v * 16, &full[s], drop);
                from += (int64_t)v * 16;
                element += (int64_t)v * (at.f32 ? 4 : 8);
                if (++s == kStages) s = 0, ++round;
            }
        }
        if (!take()) return land(full, round, s);
        info[s].vecs = -1;
        mbar_arrive_expect_tx(&full[s], 0);
        return land(full, round, s, s);
    }
    uint32_t parity = 0;
    for (int s = 0;;) {
        if (!mbar_wait(&full[s], parity)) {
            if (lane == 0) raise_error(kErrCopyTimeout);
            return;
        }
        const ScalePiece m = info[s];
        if (m.vecs < 0) return;
        const unsigned char* stage = ring + s * kPiece;
        if (m.kind == 0) scale_stage<2, 2>(stage, m, f);
        else if (m.kind == 1) scale_stage<2, 4>(stage, m, f);
        else if (m.kind == 2) scale_stage<4, 2>(stage, m, f);
        else scale_stage<4, 4>(stage, m, f);
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty[s])) : "memory");
        if (++s == kStages) s = 0, parity ^= 1;
    }
}

unsigned unit_errors_grad_norm(bool clear) { return read_unit_errors(clear); }

}  // namespace fp8q

using namespace fp8q;

namespace {

constexpr uint64_t kPlanMark = 0x66703871677264ull;

// A plan in the caller's memory: this head, then the tables of the launches.
struct Plan {
    uint64_t mark;
    int count, groups;
    int64_t chunk_bytes;
    uint64_t chunks;
    int aliased;                // an output overlaps what it may not
    int spans;                  // behind the tables, sorted
    uint64_t pad;
};
static_assert(sizeof(Plan) % 16 == 0, "the tables behind it are aligned");

struct Span {
    uintptr_t lo, hi;
    int written;
};

int groups_of(int count) { return count > 0 ? (count + kGradGroup - 1) / kGradGroup : 1; }
size_t plan_bytes(int count) {
    return sizeof(Plan) + (size_t)groups_of(count) * sizeof(GradTable) + 2 * (size_t)count * sizeof(Span);
}
GradTable* tables(void* plan) { return reinterpret_cast<GradTable*>(static_cast<char*>(plan) + sizeof(Plan)); }
const GradTable* tables(const void* plan) {
    return reinterpret_cast<const GradTable*>(static_cast<const char*>(plan) + sizeof(Plan));
}

bool valid_type(int t) { return t == FP8Q_BF16 || t == FP8Q_F32; }
int type_bytes(int t) { return t == FP8Q_F32 ? 4 : 2; }

// Some written span overlaps another one.  Sorts the spans; `hi` becomes the
// furthest end up to each of them.
bool any_overlap(Span* s, int n) {
    bool found = false;
    std::sort(s, s + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t end = 0, written_end = 0;                     // of the spans so far
    for (int i = 0; i < n; ++i) {
        if (s[i].lo < (s[i].written ? end : written_end)) found = true;
        if (s[i].written && s[i].hi > written_end) written_end = s[i].hi;
        if (s[i].hi > end) end = s[i].hi;
        s[i].hi = end;
    }
    return found;
}

// The range overlaps one of the spans as any_overlap left them.
bool meets(const Span* s, int n, const Range& r) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(r.p), b = a + r.bytes;
    if (!r.p || r.bytes == 0) return false;
    int lo = 0, hi = n;                                     // spans that start below b
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s[mid].lo < b) lo = mid + 1; else hi = mid;
    }
    return lo > 0 && s[lo - 1].hi > a;
}

// One block per SM, or per chunk where there are fewer.
template <auto KERNEL, class... Args> fp8q_status_t launch_ring(uint32_t chunks, cudaStream_t stream, const Args&... args) {
    static KernelCache cache;
    int resident = 0;
    const fp8q_status_t s = prepare_kernel(cache, KERNEL, kGradThreads + 32, kStages * kPiece, kStages * kPiece, &resident);
    return s != FP8Q_OK ? s : launch(KERNEL, grid_for(chunks, 1), kGradThreads + 32, kStages * kPiece, stream, args...);
}

// The first of the chunks that the sums leave in the second-level cache for the
// clipping, which takes them first: 64 MB of the last launch's.  What is read
// before them is evicted first (clip_buckets 96.5 us; without priorities 101.7,
// forwards 108.7).  None is given that would outlive the call: with evict_last
// on the 64 MB, as fast, what ran next found them in its way (of 80 MB read a
// second time 47 MB came from HBM after a step that clipped nothing, 4 MB now).
uint32_t kept_from(const Plan& plan, uint32_t chunks, bool clips_next) {
    const uint64_t kept = (64ull << 20) / (uint64_t)plan.chunk_bytes;
    return clips_next && kept < chunks ? chunks - (uint32_t)kept : 0;
}

// f on the table, or on a smaller one that holds it: the launch carries it along.
template <class F> fp8q_status_t with_table(const GradTable& t, F f) {
    if (t.count > kGradFew) return f(t);
    GradTableN<kGradFew> few;
    for (int i = 0; i < t.count; ++i) {
        few.item[i].grad = t.item[i].grad;
        few.item[i].out = t.item[i].out;
        few.item[i].kind = t.item[i].kind;
        few.first[i] = t.first[i];
    }
    few.first[t.count] = t.first[t.count];
    few.count = t.count;
    return f(few);
}

fp8q_status_t grad_entry(const void* plan_memory, double scale, double max_norm, float* norm, float* each, void* workspace,
                         size_t workspace_bytes, bool clip, cudaStream_t stream) {
    if (!plan_memory || !norm) return FP8Q_ERR_NULL;
    if (!aligned16(plan_memory)) return FP8Q_ERR_ALIGN;
    const Plan& plan = *static_cast<const Plan*>(plan_memory);
    if (plan.mark != kPlanMark) return FP8Q_ERR_FORMAT;
    if (!(scale > 0.0) || !(scale < INFINITY) || !(max_norm > 0.0)) return FP8Q_ERR_SIZE;
    if (plan.chunks > 0 && !workspace) return FP8Q_ERR_NULL;
    if (plan.chunks * sizeof(double) > workspace_bytes) return FP8Q_ERR_SIZE;
    if (!aligned16(norm) || !aligned16(each) || !aligned16(workspace)) return FP8Q_ERR_ALIGN;
    const Range outs[] = {{norm, 8}, {each, 4 * (size_t)plan.count}, {workspace, (size_t)plan.chunks * sizeof(double)}};
    if (any_alias(outs, 3, nullptr, 0) || (clip && plan.aliased)) return FP8Q_ERR_ALIAS;
    const Span* spans = reinterpret_cast<const Span*>(tables(plan_memory) + plan.groups);
    for (const Range& r : outs)
        if (meets(spans, plan.spans, r)) return FP8Q_ERR_ALIAS;
    double* partial = static_cast<double*>(workspace);
    fp8q_status_t st = FP8Q_OK;
    uint64_t base = 0;
    for (int g = 0; g < plan.groups && st == FP8Q_OK; ++g)
        st = with_table(tables(plan_memory)[g], [&](const auto& t) {
            const uint32_t chunks = t.first[t.count];
            constexpr int N = std::decay_t<decltype(t)>::kSize;
            const fp8q_status_t s =
                chunks ? launch_ring<grad_squares_kernel<N>>(chunks, stream, t, chunks, kept_from(plan, chunks, clip && base + chunks == plan.chunks),
                                                             plan.chunk_bytes, partial + base)
                       : FP8Q_OK;
            base += chunks;
            return s;
        });
    base = 0;
    for (int g = 0; g < plan.groups && st == FP8Q_OK; ++g) {
        const bool last = g == plan.groups - 1;
        if (!each && !last) continue;
        const JoinArgs a = {partial, plan.chunks, scale, max_norm, last ? norm : nullptr, partial + base,
                            each ? each + (size_t)g * kGradGroup : nullptr};
        st = with_table(tables(plan_memory)[g], [&](const auto& t) {
            const unsigned blocks = 1 + (each ? (unsigned)(t.count + kJoinThreads / 32 - 1) / (kJoinThreads / 32) : 0);
            base += t.first[t.count];
            return launch(grad_join_kernel<std::decay_t<decltype(t)>::kSize>, blocks, kJoinThreads, 0, stream, t, a);
        });
    }
    for (int g = plan.groups - 1; clip && st == FP8Q_OK && g >= 0; --g)
        st = with_table(tables(plan_memory)[g], [&](const auto& t) {
            const uint32_t chunks = t.first[t.count];
            constexpr int N = std::decay_t<decltype(t)>::kSize;
            return chunks ? launch_ring<grad_scale_kernel<N>>(chunks, stream, t, chunks, plan.chunk_bytes, scale,
                                                              (const float*)norm)
                          : FP8Q_OK;
        });
    return st;
}

}  // namespace

extern "C" size_t fp8q_grad_plan_bytes(int count) {
    return count < 0 || count > FP8Q_MAX_GRADS ? 0 : plan_bytes(count);
}

extern "C" fp8q_status_t fp8q_grad_plan(const fp8q_grad_t* grads, int count, void* plan_memory, size_t bytes,
                                        size_t* workspace_bytes) {
    if (count < 0 || count > FP8Q_MAX_GRADS) return FP8Q_ERR_SIZE;
    if (!plan_memory || !workspace_bytes || (count > 0 && !grads)) return FP8Q_ERR_NULL;
    if (!aligned16(plan_memory)) return FP8Q_ERR_ALIGN;
    if (bytes < plan_bytes(count)) return FP8Q_ERR_SIZE;
    Plan& plan = *static_cast<Plan*>(plan_memory);
    plan = {};
    uint64_t total = 0;                                     // bytes, at most 2^14 * 2^44
    for (int i = 0; i < count; ++i) {
        const fp8q_grad_t& g = grads[i];
        if (!valid_type(g.grad_type) || (g.out && !valid_type(g.out_type))) return FP8Q_ERR_FORMAT;
        if (g.n > FP8Q_MAX_ELEMENTS) return FP8Q_ERR_SIZE;
        total += g.n * type_bytes(g.grad_type);
        if (g.n == 0) continue;
        if (!g.grad) return FP8Q_ERR_NULL;
        if (reinterpret_cast<uintptr_t>(g.grad) % type_bytes(g.grad_type)) return FP8Q_ERR_ALIGN;
        if (g.out && reinterpret_cast<uintptr_t>(g.out) % type_bytes(g.out_type)) return FP8Q_ERR_ALIGN;
    }
    plan.count = count;
    plan.groups = groups_of(count);                         // without tensors an empty one
    plan.chunk_bytes = kPiece;
    while (total / (uint64_t)plan.chunk_bytes > kGradMaxChunks) plan.chunk_bytes *= 2;
    GradTable* tab = tables(plan_memory);
    Span* spans = reinterpret_cast<Span*>(tab + plan.groups);
    int n = 0;
    for (int g = 0; g < plan.groups; ++g) {
        GradTable& t = tab[g];
        const int lo = g * kGradGroup, hi = lo + kGradGroup < count ? lo + kGradGroup : count;
        uint32_t chunks = 0;
        t.count = hi - lo;
        for (int k = 0; k < t.count; ++k) {
            const fp8q_grad_t& s = grads[lo + k];
            const int out_type = s.out ? s.out_type : s.grad_type;
            const uintptr_t in = reinterpret_cast<uintptr_t>(s.grad), out = s.out ? reinterpret_cast<uintptr_t>(s.out) : in;
            t.item[k].grad = s.grad;
            t.item[k].out = s.out ? s.out : const_cast<void*>(s.grad);
            t.item[k].kind = s.n | (s.grad_type == FP8Q_F32 ? kGradF32 : 0) | (out_type == FP8Q_F32 ? kOutF32 : 0);
            t.first[k] = chunks;
            chunks += (uint32_t)((s.n * type_bytes(s.grad_type) + (uint64_t)plan.chunk_bytes - 1) / (uint64_t)plan.chunk_bytes);
            if (s.n == 0) continue;
            spans[n++] = {out, out + s.n * type_bytes(out_type), 1};
            if (in != out || s.grad_type != out_type) spans[n++] = {in, in + s.n * type_bytes(s.grad_type), 0};
        }
        t.first[t.count] = chunks;
        int at = 0;
        for (uint32_t k = 0; k * kNear < chunks + kNear; ++k) {     // up to the first that lies behind the last chunk
            while (at + 1 < t.count && t.first[at + 1] <= k * kNear) ++at;
            t.near[k] = (uint16_t)at;
        }
        plan.chunks += chunks;
    }
    plan.aliased = any_overlap(spans, n);
    plan.spans = n;
    plan.mark = kPlanMark;
    *workspace_bytes = (size_t)plan.chunks * sizeof(double);
    return FP8Q_OK;
}

extern "C" fp8q_status_t fp8q_grad_norm(const void* plan, double scale, double max_norm, float* norm, float* each,
                                        void* workspace, size_t workspace_bytes, fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_grad_norm");
    return grad_entry(plan, scale, max_norm, norm, each, workspace, workspace_bytes, false,
                      reinterpret_cast<cudaStream_t>(stream));
}

extern "C" fp8q_status_t fp8q_grad_clip(const void* plan, double scale, double max_norm, float* norm, float* each,
                                        void* workspace, size_t workspace_bytes, fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_grad_clip");
    return grad_entry(plan, scale, max_norm, norm, each, workspace, workspace_bytes, true,
                      reinterpret_cast<cudaStream_t>(stream));
}
