// The global norm of many gradient tensors, and the gradients clipped by it.
//
//     norm = scale * sqrt(sum of x^2 over all tensors),  coefficient = min(1, max_norm / (norm + 1e-6))
//     out = x * (scale * coefficient)
// The tensors are cut into chunks of a fixed number of elements; a block sums
// one chunk's squares into its place of the workspace, and a single block
// joins the places in their order, so that the norm does not depend on timing.
// The table of tensors travels in the kernel's parameters, kGradGroup at a
// time: nothing is copied to the device ahead of the launch, and a captured
// graph keeps the table with its node.
//
// A thread's squares are summed in binary32 (up to 64 of them) and everything
// above in binary64.  Sums outside [2^-80, 2^100] would lose squares to the
// range of binary32; their elements are summed again in binary64.
#include "fp8q_device.cuh"
#include "fp8q_host.cuh"

#include <math.h>

#include <algorithm>

namespace fp8q {

constexpr int kGradGroup = 1024;            // tensors per launch
constexpr int kGradThreads = 256;
constexpr int64_t kGradChunk = 16384;       // elements of the smallest chunk
constexpr int64_t kGradMaxChunks = 16384;   // larger chunks keep their number near this
constexpr int kJoinThreads = 1024;

// Element types and count share a word: count in the low 44 bits.
struct GradTable {
    const void* grad[kGradGroup];
    void* out[kGradGroup];
    uint64_t kind[kGradGroup];
    uint32_t first[kGradGroup + 1];         // chunks of the group's earlier tensors
    int count;
};
static_assert(sizeof(GradTable) + 64 <= 32764, "a kernel's parameters");
constexpr uint64_t kCountMask = (1ull << 44) - 1;
constexpr uint64_t kGradF32 = 1ull << 62, kOutF32 = 1ull << 63;

__device__ __forceinline__ int tensor_of(const GradTable& t, uint32_t chunk) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The elements [lo, hi) of a tensor that a chunk holds, and the first of them
// that lies on a 16-byte boundary.
struct Chunk {
    int64_t lo, hi, body;
    int64_t vecs;
};
template <int BYTES> __device__ __forceinline__ Chunk cut_chunk(const void* p, int64_t n, int64_t index, int64_t size) {
    Chunk c;
    c.lo = index * size;
    c.hi = c.lo + size < n ? c.lo + size : n;
    const uint32_t off = (uint32_t)((reinterpret_cast<uintptr_t>(p) + (uintptr_t)c.lo * BYTES) & 15u);
    const int64_t to = c.lo + (int64_t)((16u - off) & 15u) / BYTES;
    c.body = to < c.hi ? to : c.hi;
    c.vecs = (c.hi - c.body) / (16 / BYTES);
    return c;
}

template <int BYTES> __device__ __forceinline__ float load_grad(const void* p, int64_t i) {
    return BYTES == 2 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}

template <int BYTES, int N> __device__ __forceinline__ double squares(const uint4 (&v)[N]) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (BYTES == 2) {
                s[j & 1] = __fmaf_rn(bf16_lo(w[j]), bf16_lo(w[j]), s[j & 1]);
                s[2 + (j & 1)] = __fmaf_rn(bf16_hi(w[j]), bf16_hi(w[j]), s[2 + (j & 1)]);
            } else {
                s[j] = __fmaf_rn(__uint_as_float(w[j]), __uint_as_float(w[j]), s[j]);
            }
            any |= w[j];
        }
    }
    const float total = (s[0] + s[1]) + (s[2] + s[3]);
    if (total >= 0x1p-80f && total <= 0x1p100f) return (double)total;
    if (total == 0.0f && (any & (BYTES == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) == 0) return 0.0;
    double d = 0.0;
#pragma unroll 1
    for (int u = 0; u < N; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        for (int j = 0; j < 4; ++j) {
            if (BYTES == 2) {
                const double a = (double)bf16_lo(w[j]), b = (double)bf16_hi(w[j]);
                d += a * a + b * b;
            } else {
                const double a = (double)__uint_as_float(w[j]);
                d += a * a;
            }
        }
    }
    return d;
}

template <int BYTES> __device__ __forceinline__ double chunk_squares(const void* p, int64_t n, int64_t index, int64_t size) {
    constexpr int per = 16 / BYTES, U = 8;
    const int tid = (int)threadIdx.x;
    const Chunk c = cut_chunk<BYTES>(p, n, index, size);
    double sum = 0.0;
    if (c.lo + tid < c.body) {
        const double x = (double)load_grad<BYTES>(p, c.lo + tid);
        sum += x * x;
    }
    const int64_t tail = c.body + c.vecs * per + tid;
    if (tail < c.hi) {
        const double x = (double)load_grad<BYTES>(p, tail);
        sum += x * x;
    }
    const unsigned char* body = static_cast<const unsigned char*>(p) + c.body * BYTES;
    for (int64_t b = 0; b < c.vecs; b += (int64_t)kGradThreads * U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = b + u * kGradThreads + tid;
            v[u] = i < c.vecs ? ld_stream(body + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
        }
        sum += squares<BYTES>(v);
    }
    return sum;
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

__global__ void __launch_bounds__(kGradThreads) grad_squares_kernel(const __grid_constant__ GradTable t, int64_t size,
                                                                    double* partial) {
    __shared__ double sh[kGradThreads / 32];
    const int i = tensor_of(t, blockIdx.x);
    const int64_t n = (int64_t)(t.kind[i] & kCountMask);
    const int64_t index = blockIdx.x - t.first[i];
    dependency_wait();
    allow_dependents();
    const double mine = (t.kind[i] & kGradF32) ? chunk_squares<4>(t.grad[i], n, index, size)
                                               : chunk_squares<2>(t.grad[i], n, index, size);
    const double sum = block_sum<kGradThreads>(mine, sh);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
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
__global__ void __launch_bounds__(256) grad_each_kernel(const __grid_constant__ GradTable t, const double* partial, double scale,
                                                        float* each) {
    const int lane = (int)(threadIdx.x & 31u);
    const int i = (int)(blockIdx.x * 8 + (threadIdx.x >> 5));
    dependency_wait();
    allow_dependents();
    if (i >= t.count) return;
    double v = 0.0;
    for (uint32_t c = t.first[i] + (uint32_t)lane; c < t.first[i + 1]; c += 32) v += __ldcg(partial + c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) each[i] = (float)(sqrt(v) * scale);
}

template <int IN, int OUT>
__device__ __forceinline__ void scale_chunk(const void* p, void* q, int64_t n, int64_t index, int64_t size, float f) {
    const int64_t lo = index * size, hi = lo + size < n ? lo + size : n;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kGradThreads) {
        const float x = load_grad<IN>(p, i) * f;
        if (OUT == 2) static_cast<uint16_t*>(q)[i] = (uint16_t)pack_bf16x2(x, 0.0f);
        else static_cast<float*>(q)[i] = x;
    }
}

__global__ void __launch_bounds__(kGradThreads) grad_scale_kernel(const __grid_constant__ GradTable t, int64_t size, float scale,
                                                                  const float* norm) {
    const uint32_t chunk = gridDim.x - 1 - blockIdx.x;
    const int i = tensor_of(t, chunk);
    const int64_t n = (int64_t)(t.kind[i] & kCountMask);
    const int64_t index = chunk - t.first[i];
    dependency_wait();
    allow_dependents();
    const float f = scale * __ldcg(norm + 1);
    const void* p = t.grad[i];
    void* q = t.out[i];
    const bool in4 = (t.kind[i] & kGradF32) != 0, out4 = (t.kind[i] & kOutF32) != 0;
    if (p == q && f == 1.0f) return;                        // in place and unchanged
    if (in4) {
        if (out4) scale_chunk<4, 4>(p, q, n, index, size, f);
        else scale_chunk<4, 2>(p, q, n, index, size, f);
    } else {
        if (out4) scale_chunk<2, 4>(p, q, n, index, size, f);
        else scale_chunk<2, 2>(p, q, n, index, size, f);
    }
}

}  // namespace fp8q

using namespace fp8q;

namespace {

constexpr uint64_t kPlanMark = 0x66703871677264ull;

// A plan in the caller's memory: this head, then the tables of the launches.
struct Plan {
    uint64_t mark;
    int count, groups;
    int64_t size;               // elements per chunk
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
        const uint32_t chunks = t.first[t.count];
        if (chunks) st = launch(grad_squares_kernel, chunks, kGradThreads, 0, stream, t, plan.size, partial + base);
        if (st == FP8Q_OK && each)
            st = launch(grad_each_kernel, (unsigned)(t.count + 7) / 8, 256, 0, stream, t, (const double*)(partial + base), scale,
                        each + (size_t)g * kGradGroup);
        if (st != FP8Q_OK) return st;
        base += chunks;
    }
    const JoinArgs a = {partial, plan.chunks, scale, max_norm, norm};
    st = launch(grad_join_kernel, 1, kJoinThreads, 0, stream, a);
    for (int g = plan.groups - 1; clip && st == FP8Q_OK && g >= 0; --g) {
        const GradTable& t = tables(plan_memory)[g];
        if (t.first[t.count])
            st = launch(grad_scale_kernel, t.first[t.count], kGradThreads, 0, stream, t, plan.size, (float)scale,
                        (const float*)norm);
    }
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
    uint64_t total = 0;                                     // at most 2^14 * 2^42
    for (int i = 0; i < count; ++i) {
        const fp8q_grad_t& g = grads[i];
        if (!valid_type(g.grad_type) || (g.out && !valid_type(g.out_type))) return FP8Q_ERR_FORMAT;
        if (g.n > FP8Q_MAX_ELEMENTS) return FP8Q_ERR_SIZE;
        total += g.n;
        if (g.n == 0) continue;
        if (!g.grad) return FP8Q_ERR_NULL;
        if (reinterpret_cast<uintptr_t>(g.grad) % type_bytes(g.grad_type)) return FP8Q_ERR_ALIGN;
        if (g.out && reinterpret_cast<uintptr_t>(g.out) % type_bytes(g.out_type)) return FP8Q_ERR_ALIGN;
    }
    plan.count = count;
    plan.groups = groups_of(count);
    plan.size = kGradChunk;
    while (total / (uint64_t)plan.size > kGradMaxChunks) plan.size *= 2;
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
            chunks += (uint32_t)((s.n + (uint64_t)plan.size - 1) / (uint64_t)plan.size);
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
