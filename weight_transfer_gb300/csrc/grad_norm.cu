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
// a cycle and SM).  Sums outside [2^-80, 2^100] would lose squares to the range
// of binary32; their elements are summed again in binary64.
#include "fp8q_device.cuh"
#include "fp8q_host.cuh"

#include <math.h>

#include <algorithm>

namespace fp8q {

constexpr int kGradGroup = 1024;            // tensors per launch
constexpr int kGradFew = 64;                // a launch of no more has a smaller table
constexpr int kGradThreads = 256;
constexpr int kPiece = 32768;               // bytes of one copy
constexpr int kStages = 5;
constexpr uint64_t kGradMaxChunks = 4096;   // chunks grow from one piece so that there are not many more than this
constexpr int kJoinThreads = 1024;

// Element types and count share a word: count in the low 44 bits.
template <int N> struct GradTableN {
    const void* grad[N];
    void* out[N];
    uint64_t kind[N];
    uint32_t first[N + 1];                  // chunks of the group's earlier tensors
    int count;
};
using GradTable = GradTableN<kGradGroup>;
static_assert(sizeof(GradTable) + 64 <= 32764, "a kernel's parameters");
constexpr uint64_t kCountMask = (1ull << 44) - 1;
constexpr uint64_t kGradF32 = 1ull << 62, kOutF32 = 1ull << 63;

template <int N> __device__ __forceinline__ int tensor_of(const GradTableN<N>& t, uint32_t chunk) {
    int lo = 0, hi = t.count - 1;
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
// piece, in eight chains of binary32 (up to 64 squares).
template <int BYTES> __device__ __forceinline__ float squares(const uint4* piece, int vecs) {
    constexpr int kLoads = kPiece / 16 / kGradThreads;
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
                const uint64_t x = f2_pack(bf16_lo(w[j]), bf16_hi(w[j]));
                s[j] = f2_fma(x, x, s[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint64_t x = f2_pack(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
                s[(u & 1) * 2 + j] = f2_fma(x, x, s[(u & 1) * 2 + j]);
            }
        }
    }
    float a, b;
    f2_unpack(f2_add(f2_add(s[0], s[1]), f2_add(s[2], s[3])), a, b);
    return a + b;
}

// The same in binary64: squares whose sum left the range in which binary32
// keeps them all.  Nothing but zeros needs no binary64.
template <int BYTES> __device__ __noinline__ double exact_squares(const uint4* piece, int vecs) {
    double d = 0.0;
    uint32_t any = 0;
    for (int i = (int)threadIdx.x; i < vecs; i += kGradThreads) any |= piece[i].x | piece[i].y | piece[i].z | piece[i].w;
    if ((any & (BYTES == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) == 0) return 0.0;
    for (int i = (int)threadIdx.x; i < vecs; i += kGradThreads)
        for (int j = 0; j < 16 / BYTES; ++j) {
            const double x = (double)load_grad<BYTES>(piece + i, j);
            d += x * x;
        }
    return d;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// A warp's sum of its vectors' squares, in lane 0: over the lanes in binary32
// where all their sums are within range.
template <int BYTES> __device__ __forceinline__ double piece_squares(const uint4* piece, int vecs) {
    float v = squares<BYTES>(piece, vecs);
    if (__all_sync(0xFFFFFFFFu, v == 0.0f || (v >= 0x1p-80f && v <= 0x1p100f))) {
        // a sum of 0 may be one of squares that vanished: then nothing larger than 2^-74 is among them, which counts
        // only where the whole warp has no more
        if (__any_sync(0xFFFFFFFFu, v != 0.0f)) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            return (double)v;
        }
    }
    return warp_sum(exact_squares<BYTES>(piece, vecs));
}

// Sum of a value over the block, in thread 0.
template <int NT> __device__ __forceinline__ double block_sum(double v, double* sh) {
    const int lane = (int)(threadIdx.x & 31u), warp = (int)(threadIdx.x >> 5);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    v = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < NT / 32; ++w) v += sh[w];
    return v;
}

// What the copying warp tells the summing ones about a stage.
struct Piece {
    const void* tensor;         // for the elements outside the vectors
    int64_t tail;               // where those behind them start
    int head, tails;            // how many there are in front and behind, in this piece's care
    int vecs;                   // -1: no more pieces
    int f32, last;              // last piece of its chunk
};

// One block per SM walks over the chunks.  A warp of its own copies them, 32 KB
// at a time, into a ring of stages; eight warps sum.  A warp's sum of a chunk
// waits in the chunk's last stage, where the copying warp joins the eight when
// it takes the stage back.
template <int N>
__global__ void __launch_bounds__(kGradThreads + 32, 1) grad_squares_kernel(const __grid_constant__ GradTableN<N> t, uint32_t chunks,
                                                                            int64_t chunk_bytes, double* partial) {
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
    dependency_wait();
    allow_dependents();
    if (warp == kGradThreads / 32) {
        if (lane != 0) return;
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
                double v = 0.0;
                for (int w = 0; w < kGradThreads / 32; ++w) v += sums[s][w];
                partial[done] = v;
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
            const int i = tensor_of(t, c);
            const int f32 = (t.kind[i] & kGradF32) != 0, shift = f32 ? 2 : 1, per = 16 >> shift;
            const int64_t n = (int64_t)(t.kind[i] & kCountMask), index = c - t.first[i];
            const unsigned char* p = static_cast<const unsigned char*>(t.grad[i]);
            const int64_t to = (int64_t)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) >> shift;
            const int64_t head = to < n ? to : n, vecs = (n - head) / per, mine = index * (chunk_bytes / 16);
            int64_t left = vecs - mine < chunk_bytes / 16 ? vecs - mine : chunk_bytes / 16;
            if (left < 0) left = 0;                     // a last chunk of nothing but elements behind the vectors
            const bool ends_tensor = c + 1 == t.first[i + 1];
            const unsigned char* from = p + (head << shift) + mine * 16;
            for (bool first = true; first || left > 0; first = false) {
                const int v = (int)(left < kPiece / 16 ? left : kPiece / 16);
                left -= v;
                if (!take()) return;
                Piece& m = info[s];
                m.tensor = p;
                m.head = first && index == 0 ? (int)head : 0;
                m.tail = head + vecs * per;
                m.tails = left == 0 && ends_tensor ? (int)(n - m.tail) : 0;
                m.vecs = v;
                m.f32 = f32;
                m.last = left == 0;
                mbar_arrive_expect_tx(&full[s], (uint32_t)v * 16);
                if (v) bulk_g2s(ring + s * kPiece, from, (uint32_t)v * 16, &full[s]);
                from += (int64_t)v * 16;
                next(left == 0 ? (int64_t)c : -1);
            }
        }
        if (!take()) return;
        info[s].vecs = -1;
        mbar_arrive_expect_tx(&full[s], 0);
        for (int i = 1; i < kStages; ++i) {             // the stages still on their way
            next(-1);
            if (!take()) return;
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
        if (lane == 0) {
            if (m.last) {
                sums[s][warp] = sum;
                sum = 0.0;
            }
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty[s])) : "memory");
        }
        __syncwarp();
        if (++s == kStages) s = 0, parity ^= 1;
    }
}

struct JoinArgs {
    const double* partial;      // all chunks
    uint64_t chunks;
    double scale, max_norm;
    float* norm;                // [2]
};

__global__ void __launch_bounds__(kJoinThreads) grad_join_kernel(const JoinArgs a) {
    __shared__ double sh[kJoinThreads / 32];
    dependency_wait();
    allow_dependents();
    double v = 0.0;
#pragma unroll 8
    for (uint64_t i = threadIdx.x; i < a.chunks; i += kJoinThreads) v += __ldcg(a.partial + i);
    const double sum = block_sum<kJoinThreads>(v, sh);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum) * a.scale;
        const double ratio = a.max_norm / (norm + 1e-6);
        a.norm[0] = (float)norm;
        a.norm[1] = ratio >= 1.0 ? 1.0f : (float)ratio;     // a NaN stays one
    }
}

// A warp joins one tensor's chunks.
template <int N>
__global__ void __launch_bounds__(256) grad_each_kernel(const __grid_constant__ GradTableN<N> t, const double* partial, double scale,
                                                        float* each) {
    const int lane = (int)(threadIdx.x & 31u);
    const int i = (int)(blockIdx.x * 8 + (threadIdx.x >> 5));
    dependency_wait();
    allow_dependents();
    if (i >= t.count) return;
    double v = 0.0;
#pragma unroll 8
    for (uint32_t c = t.first[i] + (uint32_t)lane; c < t.first[i + 1]; c += 32) v += __ldcg(partial + c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) each[i] = (float)(sqrt(v) * scale);
}

template <int BYTES> __device__ __forceinline__ void store_grad(void* q, int64_t i, float x) {
    if (BYTES == 2) static_cast<uint16_t*>(q)[i] = (uint16_t)pack_bf16x2(x, 0.0f);
    else static_cast<float*>(q)[i] = x;
}

// Eight elements, in and out on 16-byte boundaries.
template <int BYTES> __device__ __forceinline__ void load8(const unsigned char* p, float (&f)[8]) {
    if (BYTES == 2) {
        unpack8(ld_once(p), f);
    } else {
        const uint4 a = ld_once(p), b = ld_once(p + 16);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
    }
}
template <int BYTES> __device__ __forceinline__ void store8(unsigned char* q, const float (&f)[8]) {
    if (BYTES == 2) {
        st_stream(q, make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
    } else {
        st_stream(q, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
        st_stream(q + 16, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
    }
}

// One by one, sixteen on their way: where the input and the output lie
// differently relative to 16-byte boundaries.
template <int IN, int OUT>
__device__ __forceinline__ void scale_each(const void* p, void* q, int64_t lo, int64_t hi, float f) {
    constexpr int U = 16;
    for (int64_t b = lo + threadIdx.x; b < hi; b += U * kGradThreads) {
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = b + u * kGradThreads < hi ? load_grad<IN>(p, b + u * kGradThreads) : 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (b + u * kGradThreads < hi) store_grad<OUT>(q, b + u * kGradThreads, x[u] * f);
    }
}

template <int IN, int OUT>
__device__ __forceinline__ void scale_chunk(const void* p, void* q, int64_t n, int64_t index, int64_t size, float f) {
    const int64_t lo = index * size, hi = lo + size < n ? lo + size : n;
    // elements to the first place where eight are whole vectors of both
    constexpr int IV = IN == 2 ? 8 : 4, OV = OUT == 2 ? 8 : 4, V = IV > OV ? IV : OV;
    const int in_off = (int)((reinterpret_cast<uintptr_t>(p) / IN + (uintptr_t)lo) % IV);
    const int out_off = (int)((reinterpret_cast<uintptr_t>(q) / OUT + (uintptr_t)lo) % OV);
    const int head = (V - (IV == V ? in_off : out_off)) % V;
    if ((in_off + head) % IV != 0 || (out_off + head) % OV != 0 || hi - lo < head + 8) {
        scale_each<IN, OUT>(p, q, lo, hi, f);
        return;
    }
    const int tid = (int)threadIdx.x;
    const int64_t body = lo + head;
    const int eights = (int)((hi - body) / 8);
    const unsigned char* pb = static_cast<const unsigned char*>(p) + body * IN;
    unsigned char* qb = static_cast<unsigned char*>(q) + body * OUT;
    constexpr int U = IN == 2 ? 4 : 2;
    for (int b = tid; b < eights; b += U * kGradThreads) {
        float x[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (b + u * kGradThreads < eights) load8<IN>(pb + (int64_t)(b + u * kGradThreads) * 8 * IN, x[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b + u * kGradThreads >= eights) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[u][j] *= f;
            store8<OUT>(qb + (int64_t)(b + u * kGradThreads) * 8 * OUT, x[u]);
        }
    }
    if (tid < head) store_grad<OUT>(q, lo + tid, load_grad<IN>(p, lo + tid) * f);
    const int64_t tail = body + (int64_t)eights * 8 + tid;
    if (tail < hi) store_grad<OUT>(q, tail, load_grad<IN>(p, tail) * f);
}

// The chunks backwards: what the sums read last is still in the second-level cache.
template <int N>
__global__ void __launch_bounds__(kGradThreads) grad_scale_kernel(const __grid_constant__ GradTableN<N> t, uint32_t pieces,
                                                                  float scale, const float* norm) {
    // `pieces` blocks to a chunk
    const uint32_t at = gridDim.x - 1 - blockIdx.x, chunk = at / pieces;
    const int i = tensor_of(t, chunk);
    const int64_t n = (int64_t)(t.kind[i] & kCountMask);
    const int64_t index = (int64_t)(chunk - t.first[i]) * pieces + at % pieces;
    dependency_wait();
    allow_dependents();
    const float f = scale * __ldcg(norm + 1);
    const void* p = t.grad[i];
    void* q = t.out[i];
    const bool in4 = (t.kind[i] & kGradF32) != 0, out4 = (t.kind[i] & kOutF32) != 0;
    if (p == q && f == 1.0f) return;                        // in place and unchanged
    const int64_t size = kPiece / (in4 ? 4 : 2);
    if (index * size >= n) return;
    if (in4) {
        if (out4) scale_chunk<4, 4>(p, q, n, index, size, f);
        else scale_chunk<4, 2>(p, q, n, index, size, f);
    } else {
        if (out4) scale_chunk<2, 4>(p, q, n, index, size, f);
        else scale_chunk<2, 2>(p, q, n, index, size, f);
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

int groups_of(int count) { return (count + kGradGroup - 1) / kGradGroup; }
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

// f on the table, or on a smaller one that holds it: the launch carries it along.
template <class F> fp8q_status_t with_table(const GradTable& t, F f) {
    if (t.count > kGradFew) return f(t);
    GradTableN<kGradFew> few;
    for (int i = 0; i < t.count; ++i) {
        few.grad[i] = t.grad[i];
        few.out[i] = t.out[i];
        few.kind[i] = t.kind[i];
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
    for (int g = 0; g < plan.groups; ++g) {
        const GradTable& t = tables(plan_memory)[g];
        st = with_table(t, [&](const auto& tab) {
            constexpr int N = sizeof(tab.grad) / sizeof(void*);
            const uint32_t chunks = tab.first[tab.count];
            fp8q_status_t s = FP8Q_OK;
            if (chunks) {
                static KernelCache cache;
                int resident = 0;
                s = prepare_kernel(cache, grad_squares_kernel<N>, kGradThreads + 32, kStages * kPiece, kStages * kPiece, &resident);
                if (s == FP8Q_OK)
                    s = launch(grad_squares_kernel<N>, grid_for(chunks, 1), kGradThreads + 32, kStages * kPiece, stream, tab, chunks,
                               plan.chunk_bytes, partial + base);
            }
            if (s == FP8Q_OK && each)
                s = launch(grad_each_kernel<N>, (unsigned)(tab.count + 7) / 8, 256, 0, stream, tab, (const double*)(partial + base),
                           scale, each + (size_t)g * kGradGroup);
            return s;
        });
        if (st != FP8Q_OK) return st;
        base += t.first[t.count];
    }
    const JoinArgs a = {partial, plan.chunks, scale, max_norm, norm};
    st = launch(grad_join_kernel, 1, kJoinThreads, 0, stream, a);
    for (int g = plan.groups - 1; clip && st == FP8Q_OK && g >= 0; --g)
        st = with_table(tables(plan_memory)[g], [&](const auto& tab) {
            constexpr int N = sizeof(tab.grad) / sizeof(void*);
            const uint32_t chunks = tab.first[tab.count];
            const uint32_t pieces = (uint32_t)(plan.chunk_bytes / kPiece);
            if (chunks == 0) return FP8Q_OK;
            if ((uint64_t)chunks * pieces > 0x7FFFFFFFull) return FP8Q_ERR_SIZE;
            return launch(grad_scale_kernel<N>, chunks * pieces, kGradThreads, 0, stream, tab, pieces, (float)scale,
                          (const float*)norm);
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
    plan.groups = groups_of(count);
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
            t.grad[k] = s.grad;
            t.out[k] = s.out ? s.out : const_cast<void*>(s.grad);
            t.kind[k] = s.n | (s.grad_type == FP8Q_F32 ? kGradF32 : 0) | (out_type == FP8Q_F32 ? kOutF32 : 0);
            t.first[k] = chunks;
            chunks += (uint32_t)((s.n * type_bytes(s.grad_type) + (uint64_t)plan.chunk_bytes - 1) / (uint64_t)plan.chunk_bytes);
            if (s.n == 0) continue;
            spans[n++] = {out, out + s.n * type_bytes(out_type), 1};
            if (in != out || s.grad_type != out_type) spans[n++] = {in, in + s.n * type_bytes(s.grad_type), 0};
        }
        t.first[t.count] = chunks;
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
