// Log probabilities of given tokens, with entropy and the best alternatives,
// and their gradient.
//
// For a row x of logits and z = x / T, m = max x:
//     S = sum of exp((x_j - m) / T),   log p_j = (x_j - m) / T - log S
//     entropy = - sum of p_j log p_j = log S - (sum of e_j (x_j - m) / T) / S
// One pass: every thread keeps a running maximum m of what it has read, the
// sum S relative to it and the sum E of 2^t * t with t = (x - m) c, c = log2(e) /
// T, so that a larger maximum m' turns them into
//     S' = S * 2^d,   E' = 2^d * (E + d * S),   d = (m - m') c
// and the same step joins threads, warps and the blocks of a cluster, in a
// fixed order.
//
// Gradient, from the statistics that the forward pass wrote:
//     dx_j = ([j = t] g - p_j (g + dH (log p_j + entropy))) / T
//
// All of it is bound by HBM.  4096 rows of 151,936 bf16 logits: 180 to 185 us
// forward with entropy (6.74 to 6.93 TB/s, from one GPU to another; scalar
// arithmetic on unpacked logits, 12 instructions each instead of 5, took 261), 385
// to 389 for the gradient in calls on other buffers than the last one's (6.4 TB/s)
// and 360 to 380 from a graph on the same ones (a comparison with the target at
// every logit cost 30 us more).  256 rows of 151,669 binary32 logits with five
// alternatives: 36 to 37 us, without them 26.  Four rows: 6.5 us from a graph, of
// which the launch and the joins are most (an earlier state, whose lanes joined
// their sums pair by pair and whose joins waited for the sorting, took 8.8).
#include "fp8q_device.cuh"
#include "fp8q_host.cuh"

#include <math.h>

namespace fp8q {

constexpr int kLpMaxTop = FP8Q_MAX_TOP;
constexpr int kLpCap = 128;             // candidates that a warp holds in shared memory
constexpr int kLpMaxCluster = 8;
// Blocks per SM up to which rows are divided: 256 rows of 151,669 normal binary32
// logits with five alternatives 30.6 us, with 2 36.1, with 8 35.5.
constexpr int kLpBlocksPerSm = 4;
// Places of stored maxima a thread.  1024 such rows 106 us, 8 places 109; 48 137,
// as what a block then holds of the shared memory leaves little first-level cache
// for loads on their way.
constexpr int kLpPlaces = 24;
constexpr int kLpUnroll = 4;            // 16-byte vectors per thread and step
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLowest = -3.402823466e38f;

struct LpArgs {
    const void* logits;
    const void* targets;        // or NULL
    int id64;
    int64_t vocab, stride;
    float temperature, c;       // c = log2(e) / temperature
    int top;
    int fold;                   // steps that share a place of the stored maxima
    int far;                    // where the far sums lie in the dynamic shared memory
    float* logprobs;            // each NULL when not wanted
    float* entropy;
    float* top_logprobs;
    int32_t* top_ids;
    float* stats;
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int BYTES> struct Logit;
template <> struct Logit<2> {
    static constexpr int kPerVec = 8;
    static constexpr uint32_t kNothing = 0xFF80FF80u;       // two -inf
    static __device__ __forceinline__ float load(const void* p, int64_t i) {
        return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) { unpack8(v, f); }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, float f) {
        static_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16x2(f, 0.0f);
    }
};
template <> struct Logit<4> {
    static constexpr int kPerVec = 4;
    static constexpr uint32_t kNothing = 0xFF800000u;
    static __device__ __forceinline__ float load(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, float f) { static_cast<float*>(p)[i] = f; }
};

// Elements in front of the first 16-byte boundary of a row, its whole vectors
// and the elements behind them.
struct RowCut {
    int head, tail;
    int64_t vecs;
};
template <int BYTES> __device__ __forceinline__ RowCut cut_row(const void* p, int64_t n) {
    constexpr int per = 16 / BYTES;
    RowCut r;
    const int64_t to = (int64_t)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / BYTES;
    r.head = (int)(to < n ? to : n);
    r.vecs = (n - r.head) / per;
    r.tail = (int)(n - r.head - r.vecs * per);
    return r;
}

__device__ __forceinline__ int64_t load_id(const void* p, int id64, int64_t i) {
    return id64 ? (int64_t)static_cast<const long long*>(p)[i] : (int64_t)static_cast<const int*>(p)[i];
}

// Sums over a set of logits relative to one of them, m: s of 2^t and e of 2^t * t
// with t = (x - m) c; and the set's largest logit.
struct Soft {
    float m, s, e, top;
};
__device__ __forceinline__ void raise(Soft& a, float m, float c) {
    const float d = fmaxf((a.m - m) * c, -1000.0f);         // a.m <= m; 2^-1000 is 0
    const float f = ex2(d);
    a.e = f * (a.e + d * a.s);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
    return r;
}
// Joins the sums of a warp's lanes; the first LANES of them have the result.
template <int LANES> __device__ __forceinline__ void join_lanes(Soft& a, float c) {
    raise(a, warp_max(a.m), c);
    a.top = warp_max(a.top);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(0xFFFFFFFFu, a.s, o);
        a.e += __shfl_xor_sync(0xFFFFFFFFu, a.e, o);
    }
}

// The far sums.  A thread's own chains take no more than 256 terms one after
// another; then what they hold is added, with what that addition rounds off, to
// sums in shared memory, so that a row's error does not grow with its length:
// equal terms that are rounded the same way every time were off by 1e-4 at 200
// million logits, 5e-7 at 151,936, and are 9e-7 at any length now (one row of 16
// million bf16 logits 87.5 us, without them 84.8).  They have an instance of the
// kernel of their own (FAR): rows of which a block's share is shorter would take
// 0.7% longer, four rows 3%.
constexpr int kLpChain = 256;
template <int BYTES> constexpr int kLpFarSteps = kLpChain * BYTES / 16;     // a step adds 8 bf16 or 4 binary32 terms to a chain
template <int NT> struct LpFar {
    float m[NT], s[NT], s_off[NT], e[NT], e_off[NT];
};
__device__ __forceinline__ void add_off(float& sum, float& off, float x) {  // sum + off += x, what is rounded off goes to off
    const float t = sum + x, b = t - sum;
    off += (sum - (t - b)) + (x - b);
    sum = t;
}
// Brings a thread's far sums to the reference m, not below theirs, and adds s and e.
template <int NT> __device__ __noinline__ void add_far(LpFar<NT>& far, float m, float s, float e, float c) {
    const int i = (int)threadIdx.x;
    const float d = fmaxf((far.m[i] - m) * c, -1000.0f), f = ex2(d);
    float fe = f * (far.e[i] + d * far.s[i]), fe_off = f * (far.e_off[i] + d * far.s_off[i]);
    float fs = f * far.s[i], fs_off = f * far.s_off[i];
    add_off(fs, fs_off, s);
    add_off(fe, fe_off, e);
    far.m[i] = m;
    far.s[i] = fs;
    far.s_off[i] = fs_off;
    far.e[i] = fe;
    far.e_off[i] = fe_off;
}

// A thread's sums.  The reference m is raised only where a logit exceeds it by 4
// units of t, so that most steps raise nothing (score_rollouts 179.9 us, 183.0
// where every larger logit raises it; 256 rows with alternatives 30.6 and 34.2); t is rounded by up to 4 * 2^-24 then, in
// the terms that count, which a slack of 40 would make 40 * 2^-24.
// t is taken as x * c - mc with mc = RN(m * c), one instruction for two logits;
// settle() and take() go between that reference and m itself.  Logits below
// m - 4000 / c count as that, whose 2^t is 0, so that no 0 * -inf arises in e.
// All that holds for |m| c below 2^18, where bf16 still tells m from that bound;
// otherwise (no finite logit yet, the type's extremes, a temperature near 0)
// logits are added one by one.
constexpr float kSlack = 4.0f;
constexpr float kBound = 4000.0f;
__device__ __forceinline__ bool ordinary(float m, float c) { return fabsf(m) * c < 0x1p18f; }

template <int BYTES, bool ENT> struct Sums {
    float m, mc, top;
    bool fast;                                               // ordinary(m, c)
    uint32_t low;                                            // m - kBound / c: in binary32, or twice in bf16
    uint64_t s[2], e[2];

    __device__ __forceinline__ void reset() {
        m = mc = kLowest;
        top = -INFINITY;
        fast = false;
        low = 0;
        forget();
    }
    __device__ __forceinline__ Soft settle(float c) const {
        float a, b, x, y;
        f2_unpack(f2_add(s[0], s[1]), a, b);
        f2_unpack(f2_add(e[0], e[1]), x, y);
        Soft r = {m, a + b, x + y, top};
        if (fast) {                                          // 2^(x c - mc) = 2^t * 2^(m c - mc)
            const float d = __fmaf_rn(m, c, -mc), f = ex2(-d);
            r.e = f * (r.e - d * r.s);
            r.s *= f;
        }
        return r;
    }
    __device__ __forceinline__ void take(const Soft& v, float c) {
        m = v.m;
        mc = m;
        float d = 0.0f, f = 1.0f;
        fast = ordinary(m, c);
        if (fast) {
            mc = m * c;
            d = __fmaf_rn(m, c, -mc);
            f = ex2(d);
            const float l = m - __fdiv_rn(kBound, c);
            low = BYTES == 2 ? pack_bf16x2(l, l) : __float_as_uint(l);
        }
        s[0] = f2_pack(v.s * f, 0.0f);
        e[0] = f2_pack(f * (v.e + d * v.s), 0.0f);
        s[1] = e[1] = 0;
    }
    __device__ __forceinline__ void forget() { s[0] = s[1] = e[0] = e[1] = 0; }    // what has been added elsewhere
    // Before logits of which the largest is `most` are added.
    __device__ __forceinline__ void meet(float most, float c) {
        top = fmaxf(top, most);
        if ((most - m) * c > kSlack) {
            Soft v = settle(c);
            raise(v, most, c);
            take(v, c);
        }
    }
    __device__ __forceinline__ void add_one(float x, float c) {
        if (x == -INFINITY) return;
        float d = fast ? __fmaf_rn(x, c, -mc) : (x - m) * c;
        if (ENT) d = max_nan(d, -kBound);
        const float p = ex2(d);
        s[0] = f2_add(s[0], f2_pack(p, 0.0f));
        if (ENT) e[0] = f2_fma(f2_pack(p, 0.0f), f2_pack(d, 0.0f), e[0]);
    }
    template <int V> __device__ __forceinline__ void add(const uint4 (&v)[V], float c) {
        if (!fast) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                float f[16 / BYTES];
                Logit<BYTES>::unpack(v[u], f);
#pragma unroll
                for (int j = 0; j < 16 / BYTES; ++j) add_one(f[j], c);
            }
            return;
        }
        const uint64_t c2 = f2_pack(c, c), mc2 = f2_pack(-mc, -mc);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int j = 0; j < 4; j += BYTES / 2) {
                uint64_t x;
                if (BYTES == 2) {
                    const uint32_t y = ENT ? max_nan_bf16x2(w[j], low) : w[j];
                    x = f2_pack(bf16_lo(y), bf16_hi(y));
                } else {
                    const float a = __uint_as_float(w[j]), b = __uint_as_float(w[j + 1]), l = __uint_as_float(low);
                    x = ENT ? f2_pack(max_nan(a, l), max_nan(b, l)) : f2_pack(a, b);
                }
                const uint64_t d = f2_fma(x, c2, mc2);
                float d0, d1;
                f2_unpack(d, d0, d1);
                const uint64_t p = f2_pack(ex2(d0), ex2(d1));
                const int k = (j / (BYTES / 2)) & 1;
                s[k] = f2_add(s[k], p);
                if (ENT) e[k] = f2_fma(p, d, e[k]);
            }
        }
    }
};

template <int BYTES, int V> __device__ __forceinline__ float largest(const uint4 (&v)[V]) {
    if (BYTES == 2) {
        uint32_t m = max_bf16x2(max_bf16x2(v[0].x, v[0].y), max_bf16x2(v[0].z, v[0].w));
#pragma unroll
        for (int u = 1; u < V; ++u) m = max_bf16x2(m, max_bf16x2(max_bf16x2(v[u].x, v[u].y), max_bf16x2(v[u].z, v[u].w)));
        return fmaxf(bf16_lo(m), bf16_hi(m));
    }
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        m = fmaxf(m, fmaxf(__uint_as_float(v[u].x), __uint_as_float(v[u].y)));
        m = fmaxf(m, fmaxf(__uint_as_float(v[u].z), __uint_as_float(v[u].w)));
    }
    return m;
}

// Candidates are ordered by one 64-bit key, larger logits first and among
// equal ones the lower index; +0 and -0 are equal.  No key is 0.
__device__ __forceinline__ uint64_t key_of(float x, int64_t i) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t o = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
    return ((uint64_t)o << 32) | (0xFFFFFFFFu - (uint32_t)i);
}
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ int32_t key_index(uint64_t k) { return (int32_t)(0xFFFFFFFFu - (uint32_t)k); }

__device__ __forceinline__ uint32_t map_rank0(const void* p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
    return r;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t a, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

template <int NT> struct LpShared {
    Soft warp[NT / 32];
    Soft part[kLpMaxCluster];
    float m, log_s;             // of the row; m = -inf without any logit
};
// The alternatives.  Every thread stores the largest logit of each of its steps.
// When the row is through, the top-th largest of 64 groups' maxima is a floor:
// as many logits are not below it, and few more.  The steps that reach the
// floor, a few dozen, are read again, one to a thread, and what is in them and
// not below the floor is sorted.  Where that is too much (many equal logits),
// the warps go through their steps one by one, each keeping its best.
constexpr int kLpGather = kLpMaxCluster * kLpMaxTop;
struct __align__(16) WarpTop {
    uint64_t keys[kLpCap];
    int count;
};
template <int NT> struct LpTopShared {
    WarpTop warp[NT / 32];
    uint64_t gather[kLpGather];
    uint64_t parts[kLpGather];  // what the blocks of a cluster found, in the first of them
    uint64_t sorted[kLpMaxTop], best[kLpMaxTop];        // of gather, and of parts
    float group[64];
    int list[kLpGather];
    float floor;
    int listed, gathered;
    float most[1];              // [steps / fold][NT]
};

// Leaves the `top` largest of the warp's n > top keys as keys[0 .. top) and
// returns the smallest of them, which is found bit by bit.
__device__ __noinline__ uint64_t narrow(WarpTop& t, int top, int n) {
    const int lane = (int)(threadIdx.x & 31u);
    uint64_t k[kLpCap / 32];
#pragma unroll
    for (int j = 0; j < kLpCap / 32; ++j) k[j] = lane + 32 * j < n ? t.keys[lane + 32 * j] : 0;
    uint64_t lo = 0;
#pragma unroll 1
    for (int i = 63; i >= 0; --i) {
        const uint64_t mid = lo | (1ull << i);
        int c = 0;
#pragma unroll
        for (int j = 0; j < kLpCap / 32; ++j) c += k[j] >= mid;
        if (__reduce_add_sync(0xFFFFFFFFu, c) >= top) lo = mid;
    }
    int at = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kLpCap / 32; ++j) {
        const unsigned m = __ballot_sync(0xFFFFFFFFu, k[j] >= lo);
        if (k[j] >= lo) t.keys[at + __popc(m & ((1u << lane) - 1u))] = k[j];
        at += __popc(m);
    }
    if (lane == 0) t.count = top;
    __syncwarp();
    return lo;
}

// The `top` largest keys of keys[0 .. n) in falling order into sorted, which was
// all 0 before.  Keys are unique, but for 0, which is none; n at most kLpGather,
// keys behind n up to the next multiple of 8 are 0; keys 16-byte aligned.
template <int NT> __device__ __forceinline__ void sort_top(const uint64_t* keys, int n, int top, uint64_t* sorted) {
    for (int i = (int)threadIdx.x; i < n; i += NT) {
        const uint64_t k = keys[i];
        int above = 0;
        for (int j = 0; j < n; j += 8) {
            ulonglong2 o[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) o[u] = *reinterpret_cast<const ulonglong2*>(keys + j + 2 * u);
#pragma unroll
            for (int u = 0; u < 4; ++u) above += (o[u].x > k) + (o[u].y > k);
        }
        if (k != 0 && above < top) sorted[above] = k;
    }
    __syncthreads();
}

// Joins n <= 8 partial results; for a whole warp, whose first lanes have the result.
__device__ __forceinline__ Soft join_parts(const Soft* parts, int n, float c) {
    const int lane = (int)(threadIdx.x & 31u);
    Soft v = lane < n ? parts[lane] : Soft{kLowest, 0.0f, 0.0f, -INFINITY};
    join_lanes<8>(v, c);
    return v;
}

// A row's scores and statistics from its sums.
template <bool ENT>
__device__ __forceinline__ void write_row(const LpArgs& a, int64_t row, int64_t target, float target_logit, Soft v, float& m, float& log_s) {
    // a row of -inf alone has no distribution: its scores are -inf, its entropy 0
    raise(v, v.top == -INFINITY ? v.m : v.top, a.c);
    const bool none = v.top == -INFINITY && v.s == 0.0f;
    log_s = none ? 0.0f : logf(v.s);
    m = none ? -INFINITY : v.m;
    if (a.logprobs)
        a.logprobs[row] = target < 0 ? 0.0f : none ? -INFINITY : __fdiv_rn(target_logit - m, a.temperature) - log_s;
    if (ENT) a.entropy[row] = none ? 0.0f : log_s - __fdiv_rn(v.e, v.s) * kLn2;
    if (a.stats) {
        a.stats[2 * row] = m;
        a.stats[2 * row + 1] = log_s;
    }
}

// Many short rows: one for each warp, without a barrier.  From eight rows per SM
// on, of up to 48 KB (9728 rows of 1 KB bf16 logits 6.5 us, of 16 KB 25.9, of 48
// KB 69.1; with a block to each 29.8, 44.9 and 84.3.  1216 rows of 48 KB 10.0 and
// 10.7, 608 rows of 48 KB 7.9 and 6.0.  Of 64 KB 1216 rows take as long either way
// and 9728 97.5 and 104, but a lane's chains are then as long as the error's bound
// allows).
constexpr int kLpRowThreads = 128;
constexpr int64_t kLpRowBytes = 49152;
constexpr int kLpRowsPerSm = 8;
template <int BYTES, bool ENT>
__global__ void __launch_bounds__(kLpRowThreads, 8) token_logprobs_rows_kernel(const LpArgs a, int64_t rows) {
    using L = Logit<BYTES>;
    const int lane = (int)(threadIdx.x & 31u);
    const int64_t row = (int64_t)blockIdx.x * (kLpRowThreads / 32) + (threadIdx.x >> 5);
    dependency_wait();
    allow_dependents();
    if (row >= rows) return;
    const unsigned char* x = static_cast<const unsigned char*>(a.logits) + row * a.stride * BYTES;
    const RowCut cut = cut_row<BYTES>(x, a.vocab);
    const unsigned char* body = x + (int64_t)cut.head * BYTES;
    const int vecs = (int)cut.vecs;
    auto load = [&](uint4 (&v)[kLpUnroll], int base) {
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
            const int i = base + u * 32 + lane;
            v[u] = i < vecs ? ld_stream(body + 16 * (int64_t)i) : make_uint4(L::kNothing, L::kNothing, L::kNothing, L::kNothing);
        }
    };
    uint4 next[kLpUnroll];
    load(next, 0);
    // the elements outside the row's vectors, up to 7 on either side, one for a lane
    float extra = -INFINITY;
    if (lane < cut.head) extra = L::load(x, lane);
    if (lane >= 8 && lane - 8 < cut.tail) extra = L::load(x, cut.head + cut.vecs * L::kPerVec + (lane - 8));
    int64_t target = -1;
    float target_logit = 0.0f;
    if (lane == 0 && a.targets) {
        target = load_id(a.targets, a.id64, row);
        if (target < 0 || target >= a.vocab) target = -1;
        else target_logit = L::load(x, target);
    }
    Sums<BYTES, ENT> sums;
    sums.reset();
    for (int base = 0; base < vecs; base += 32 * kLpUnroll) {
        uint4 v[kLpUnroll];
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) v[u] = next[u];
        if (base + 32 * kLpUnroll < vecs) load(next, base + 32 * kLpUnroll);
        sums.meet(largest<BYTES>(v), a.c);
        sums.add(v, a.c);
    }
    if (!(extra == -INFINITY)) {
        sums.meet(extra, a.c);
        sums.add_one(extra, a.c);
    }
    Soft acc = sums.settle(a.c);
    join_lanes<32>(acc, a.c);
    float m, log_s;
    if (lane == 0) write_row<ENT>(a, row, target, target_logit, acc, m, log_s);
}

template <int BYTES, bool TOP, bool ENT, int NT, bool FAR>
__global__ void __launch_bounds__(NT, NT == 256 ? 4 : 1) token_logprobs_kernel(const LpArgs a) {
    using L = Logit<BYTES>;
    constexpr int per = L::kPerVec;
    __shared__ LpShared<NT> sh;
    extern __shared__ __align__(16) unsigned char dyn[];
    LpTopShared<NT>& t = *reinterpret_cast<LpTopShared<NT>*>(dyn);
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    WarpTop& mine = t.warp[warp];
    uint32_t ranks;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
    const int64_t row = blockIdx.x / ranks;
    const unsigned char* x = static_cast<const unsigned char*>(a.logits) + row * a.stride * BYTES;
    const RowCut cut = cut_row<BYTES>(x, a.vocab);
    const int64_t v0 = cut.vecs * rank / ranks, v1 = cut.vecs * (rank + 1) / ranks;
    const unsigned char* body = x + (int64_t)cut.head * BYTES;
    if (TOP) {
        if (tid == 0) t.listed = t.gathered = 0;
        if (tid < kLpMaxTop) t.sorted[tid] = t.best[tid] = 0;
        for (int i = tid; i < kLpGather; i += NT) t.gather[i] = t.parts[i] = 0;
    }
    if (ranks > 1) cluster_arrive();
    dependency_wait();
    allow_dependents();

    auto load = [&](uint4 (&v)[kLpUnroll], int64_t base) {
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
            const int64_t i = base + u * NT + tid;
            v[u] = i < v1 ? ld_stream(body + 16 * i) : make_uint4(L::kNothing, L::kNothing, L::kNothing, L::kNothing);
        }
    };
    uint4 next[kLpUnroll];
    load(next, v0);
    // the elements outside the row's vectors, one for a thread
    float extra = -INFINITY;
    int64_t extra_at = 0;
    if (rank == 0 && tid < cut.head) extra_at = tid, extra = L::load(x, extra_at);
    if (rank == ranks - 1 && tid >= 32 && tid - 32 < cut.tail)
        extra_at = cut.head + cut.vecs * per + (tid - 32), extra = L::load(x, extra_at);
    // the lead joins the warps' sums while others sort; its first lane writes the row's scores
    constexpr int kLead = TOP ? NT / 32 - 1 : 0;
    int64_t target = -1;
    float target_logit = 0.0f;
    if (rank == 0 && tid == kLead * 32 && a.targets) {
        target = load_id(a.targets, a.id64, row);
        if (target < 0 || target >= a.vocab) target = -1;
        else target_logit = L::load(x, target);
    }

    Sums<BYTES, ENT> sums;
    sums.reset();
    LpFar<NT>& far = *reinterpret_cast<LpFar<NT>*>(dyn + a.far);
    if (FAR) {
        far.m[tid] = kLowest;
        far.s[tid] = far.s_off[tid] = far.e[tid] = far.e_off[tid] = 0.0f;
    }
    int places = 0, sharing = 0;                     // places of stored maxima begun, and steps in the last of them
    float held = -INFINITY;
    auto step = [&](int64_t base) {
        uint4 v[kLpUnroll];
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) v[u] = next[u];
        if (base + (int64_t)NT * kLpUnroll < v1) load(next, base + (int64_t)NT * kLpUnroll);
        const float most = largest<BYTES>(v);
        sums.meet(most, a.c);
        sums.add(v, a.c);
        if (TOP) {
            if (sharing == 0) held = -INFINITY, ++places;
            held = fmaxf(held, most);
            t.most[(places - 1) * NT + tid] = held;
            if (++sharing == a.fold) sharing = 0;
        }
    };
    if constexpr (FAR) {
        constexpr int64_t kTurn = (int64_t)NT * kLpUnroll * kLpFarSteps<BYTES>;
        for (int64_t turn = v0;; turn += kTurn) {
            const int64_t end = turn + kTurn < v1 ? turn + kTurn : v1;
#pragma unroll 1
            for (int64_t base = turn; base < end; base += (int64_t)NT * kLpUnroll) step(base);
            if (end == v1) break;
            const Soft now = sums.settle(a.c);
            add_far<NT>(far, now.m, now.s, now.e, a.c);
            sums.forget();
        }
    } else {
        for (int64_t base = v0; base < v1; base += (int64_t)NT * kLpUnroll) step(base);
    }
    if (!(extra == -INFINITY)) {
        sums.meet(extra, a.c);
        sums.add_one(extra, a.c);
    }

    Soft acc = sums.settle(a.c);
    if (FAR) {
        add_far<NT>(far, acc.m, acc.s, acc.e, a.c);
        acc.s = far.s[tid] + far.s_off[tid];
        acc.e = far.e[tid] + far.e_off[tid];
    }
    join_lanes<32>(acc, a.c);
    if (lane == 0) sh.warp[warp] = acc;
    if (TOP) {
        float g = sums.top;
#pragma unroll
        for (int o = 1; o < NT / 64; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
        if (tid % (NT / 64) == 0) t.group[tid / (NT / 64)] = g;
    }
    __syncthreads();
    if (ranks > 1) cluster_wait();                   // the first block has started
    if (warp == kLead) {
        acc = join_parts(sh.warp, NT / 32, a.c);
        if (lane == 0 && ranks > 1) {
            const uint32_t to = map_rank0(&sh.part[rank]);
            st_cluster_f32(to, acc.m);
            st_cluster_f32(to + 4, acc.s);
            st_cluster_f32(to + 8, acc.e);
            st_cluster_f32(to + 12, acc.top);
        } else if (lane == 0) {
            write_row<ENT>(a, row, target, target_logit, acc, sh.m, sh.log_s);
        }
    }
    if (TOP) {
        if (tid < 64) {
            const float own = t.group[tid];
            int above = 0;
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
                const float4 o = *reinterpret_cast<const float4*>(&t.group[j]);
                above += (o.x > own || (o.x == own && j < tid)) + (o.y > own || (o.y == own && j + 1 < tid)) +
                         (o.z > own || (o.z == own && j + 2 < tid)) + (o.w > own || (o.w == own && j + 3 < tid));
            }
            if (above == a.top - 1) t.floor = own;
        }
        __syncthreads();
        const float floor_value = t.floor;
#pragma unroll 4
        for (int i = 0; i < places; ++i) {
            const float m = t.most[i * NT + tid];
            if (m >= floor_value && m > -INFINITY) {
                const int pos = atomicAdd(&t.listed, 1);
                if (pos < kLpGather) t.list[pos] = i * NT + tid;
            }
        }
        if (extra >= floor_value && extra > -INFINITY) {
            const int pos = atomicAdd(&t.gathered, 1);
            if (pos < kLpGather) t.gather[pos] = key_of(extra, extra_at);
        }
        __syncthreads();
        const int listed = t.listed;
        if (listed <= kLpGather) {
            for (int e = tid; e < listed * kLpUnroll; e += NT) {        // one of a step's vectors to a thread
                const int step = t.list[e / kLpUnroll], place = step / NT, owner = step % NT;
                for (int f = 0; f < a.fold; ++f) {
                    const int64_t i = v0 + ((int64_t)(place * a.fold + f) * kLpUnroll + e % kLpUnroll) * NT + owner;
                    if (i >= v1) break;
                    float x8[per];
                    L::unpack(ld_stream(body + 16 * i), x8);
                    unsigned hits = 0;
#pragma unroll
                    for (int j = 0; j < per; ++j) hits |= (x8[j] >= floor_value && x8[j] > -INFINITY ? 1u : 0u) << j;
                    if (hits == 0) continue;
                    int pos = atomicAdd(&t.gathered, __popc(hits));
#pragma unroll
                    for (int j = 0; j < per; ++j) {
                        if (!(hits >> j & 1)) continue;
                        if (pos < kLpGather) t.gather[pos] = key_of(x8[j], cut.head + i * per + j);
                        ++pos;
                    }
                }
            }
            __syncthreads();
        }
        int n = t.gathered;
        if (listed > kLpGather || n > kLpGather) {
            // too many: every warp goes through its steps again and keeps its best
            if (lane == 0) mine.count = 0;
            __syncwarp();
            uint64_t floor_key = 0;
            float floor_own = floor_value;
            auto offer = [&](float f, int64_t i) {   // one logit of each lane
                bool pending = f > -INFINITY && f >= floor_own && key_of(f, i) >= floor_key;
                while (__any_sync(0xFFFFFFFFu, pending)) {
                    if (pending) {
                        const int pos = atomicAdd(&mine.count, 1);
                        if (pos < kLpCap) mine.keys[pos] = key_of(f, i), pending = false;
                    }
                    __syncwarp();
                    const int c = mine.count;
                    __syncwarp();
                    if (c > kLpCap - 32) {
                        floor_key = narrow(mine, a.top, c < kLpCap ? c : kLpCap);
                        floor_own = fmaxf(floor_own, key_value(floor_key));
                        pending = pending && key_of(f, i) >= floor_key;
                    }
                }
            };
            offer(extra, extra_at);
#pragma unroll 1
            for (int s = 0; s < places; ++s) {
                if (!__any_sync(0xFFFFFFFFu, t.most[s * NT + tid] >= floor_own)) continue;
#pragma unroll 1
                for (int u = 0; u < kLpUnroll * a.fold; ++u) {
                    const int64_t i = v0 + ((int64_t)s * a.fold * kLpUnroll + u) * NT + tid;
                    const uint4 v = i < v1 ? ld_stream(body + 16 * i) : make_uint4(L::kNothing, L::kNothing, L::kNothing, L::kNothing);
                    float x8[per];
                    L::unpack(v, x8);
#pragma unroll
                    for (int j = 0; j < per; ++j)
                        if (__any_sync(0xFFFFFFFFu, x8[j] >= floor_own)) offer(x8[j], cut.head + i * per + j);
                }
            }
            int own = mine.count;
            if (own > a.top) {
                narrow(mine, a.top, own);
                own = a.top;
            }
            __syncthreads();                         // the gathered ones have been counted
            n = NT / 32 * a.top;
            if (lane < a.top) t.gather[warp * a.top + lane] = lane < own ? mine.keys[lane] : 0;
            if (tid < 8 && n + tid < kLpGather) t.gather[n + tid] = 0;
            __syncthreads();
        }
        sort_top<NT>(t.gather, n, a.top, t.sorted);
    }
    if (ranks > 1) {
        if (TOP && tid < a.top) st_cluster_u64(map_rank0(&t.parts[rank * a.top + tid]), t.sorted[tid]);
        cluster_sync();
        if (rank != 0) return;
        if (warp == kLead) {
            acc = join_parts(sh.part, (int)ranks, a.c);
            if (lane == 0) write_row<ENT>(a, row, target, target_logit, acc, sh.m, sh.log_s);
        }
        if (TOP) sort_top<NT>(t.parts, (int)ranks * a.top, a.top, t.best);
    }
    if (TOP) {
        uint64_t* list = ranks > 1 ? t.best : t.sorted;
        if (list[a.top - 1] == 0) {
            // fewer candidates than asked for: the first logits that are -inf (or NaN) fill the list; fewer than `top`
            // are neither, so that they lie among the first 2 * top
            __syncthreads();
            if (tid == 0) {
                int n = 0;
                while (list[n] != 0) ++n;
                for (int64_t i = 0; n < a.top; ++i)
                    if (!(L::load(x, i) > -INFINITY)) list[n++] = key_of(-INFINITY, i);
            }
            __syncthreads();
        }
        if (tid < a.top) {
            const uint64_t k = list[tid];
            const float m = sh.m;
            a.top_ids[row * a.top + tid] = key_index(k);
            a.top_logprobs[row * a.top + tid] =
                m == -INFINITY ? -INFINITY : __fdiv_rn(key_value(k) - m, a.temperature) - sh.log_s;
        }
    }
}

// ------------------------------------------------------------- gradient ----
struct LpGradArgs {
    const void* logits;
    const void* targets;
    int id64;
    int64_t rows, vocab, stride, dstride;
    float inv_t, c;             // 1 / temperature, log2(e) / temperature
    const float* stats;
    const float* dlogprobs;     // or NULL
    const float* entropy;       // with dentropy
    const float* dentropy;      // or NULL
    void* dlogits;
    unsigned parts;             // blocks per row
};

// Blocks of 128 threads with four vectors each: a narrower window of memory on
// its way than with 256 threads (score_grad_long in a row 385.8 us where 393.8, 512
// threads 451; two vectors 463, eight 385).
constexpr int kLpGradThreads = 128;
constexpr int kLpGradUnroll = 4;
// Many short rows go to a warp each: of up to 4 KB from eight rows per SM on (1216
// rows of 2 KB bf16 logits 2.1 us, with a block to each 2.4, of 4 KB 2.8 and 2.8;
// 608 rows of 2 KB 2.0 and 1.9), of up to 6 KB from twelve (1824 rows of 6 KB 3.8
// and 4.1, 19,456 37.2 and 38.7; 1520 rows 3.7 and 3.4, 1216 3.4 and 3.2; of 8 KB
// 40,000 rows 97.6 and 95.6).
constexpr int64_t kLpGradShort = 4096, kLpGradMedium = 6000;
constexpr int kLpGradShortRowsPerSm = 8, kLpGradMediumRowsPerSm = 12;

// NT threads take one part of one row, or all of it where a block has several rows.
// VEC: the rows of logits and dlogits lie
// alike relative to 16-byte boundaries.
//   With t = (x - m) c - log2 S:  dx = 2^t (base + slope t), plus g at the
// target, the last taken after the others.  Logits below m - 4000 / c count as
// that, whose 2^t is 0, so that no 0 * -inf arises; where bf16 does not tell m
// from that bound, logits go one by one.
template <int BYTES, bool ENT, bool VEC, int NT>
__global__ void __launch_bounds__(kLpGradThreads) token_logprobs_backward_kernel(const LpGradArgs a) {
    using L = Logit<BYTES>;
    constexpr int per = L::kPerVec;
    constexpr int kRows = kLpGradThreads / NT;
    const int tid = (int)threadIdx.x % NT;
    const int64_t row = kRows > 1 ? (int64_t)blockIdx.x * kRows + threadIdx.x / NT : blockIdx.x / a.parts;
    const unsigned part = kRows > 1 ? 0u : blockIdx.x - (unsigned)row * a.parts;
    const unsigned char* x = static_cast<const unsigned char*>(a.logits) + row * a.stride * BYTES;
    unsigned char* dx = static_cast<unsigned char*>(a.dlogits) + row * a.dstride * BYTES;
    const RowCut cut = cut_row<BYTES>(x, a.vocab);
    const int64_t v0 = cut.vecs * part / a.parts, v1 = cut.vecs * (part + 1) / a.parts;
    const unsigned char* body = x + (int64_t)cut.head * BYTES;
    unsigned char* dbody = dx + (int64_t)cut.head * BYTES;
    dependency_wait();
    allow_dependents();
    if (row >= a.rows) return;
    int64_t target = a.targets ? load_id(a.targets, a.id64, row) : -1;
    if (target < 0 || target >= a.vocab) target = -1;
    const float m = a.stats[2 * row], log_s = a.stats[2 * row + 1];
    const float g = target >= 0 && a.dlogprobs ? a.dlogprobs[row] * a.inv_t : 0.0f;
    const float dh = ENT ? a.dentropy[row] * a.inv_t : 0.0f;
    const float base = ENT ? -(g + dh * a.entropy[row]) : -g;
    const float slope = ENT ? -dh * kLn2 : 0.0f;
    const float shift = -log_s * kLog2e;
    const bool zero = m == -INFINITY || (g == 0.0f && dh == 0.0f);  // nothing reaches this row: zeros, whatever it holds
    const bool fast = ordinary(m, a.c);
    auto grad = [&](float v, int64_t i) {
        if (zero) return 0.0f;
        float d = __fmaf_rn(v - m, a.c, shift);
        if (ENT) d = max_nan(d, -200.0f);            // 2^-200 is 0 here
        float r = ex2(d) * (ENT ? __fmaf_rn(slope, d, base) : base);
        if (i == target) r += g;
        return r;
    };
    if (!VEC) {
        const int64_t lo = a.vocab * part / a.parts, hi = a.vocab * (part + 1) / a.parts;
#pragma unroll 8
        for (int64_t i = lo + tid; i < hi; i += NT) L::store(dx, i, grad(L::load(x, i), i));
        return;
    }
    if (part == 0 && tid < cut.head) L::store(dx, tid, grad(L::load(x, tid), tid));
    if (part == a.parts - 1 && tid < cut.tail) {
        const int64_t i = cut.head + cut.vecs * per + tid;
        L::store(dx, i, grad(L::load(x, i), i));
    }
    const int64_t target_vec = target >= cut.head ? (target - cut.head) / per : -1;
    const float lowest = m - __fdiv_rn(kBound, a.c);
    const uint32_t low = BYTES == 2 ? pack_bf16x2(lowest, lowest) : __float_as_uint(lowest);
    const uint64_t c2 = f2_pack(a.c, a.c), m2 = f2_pack(-m, -m), shift2 = f2_pack(shift, shift);
    const uint64_t base2 = f2_pack(base, base), slope2 = f2_pack(slope, slope);
    for (int64_t b = v0; b < v1; b += (int64_t)NT * kLpGradUnroll) {
        uint4 v[kLpGradUnroll];
#pragma unroll
        for (int u = 0; u < kLpGradUnroll; ++u) {
            const int64_t i = b + u * NT + tid;
            if (i < v1 && !zero) v[u] = ld_once(body + 16 * i);     // dlogits may be the logits themselves
        }
#pragma unroll
        for (int u = 0; u < kLpGradUnroll; ++u) {
            const int64_t i = b + u * NT + tid;
            if (i >= v1) break;
            float f[per];
            if (zero) {
                st_stream(dbody + 16 * i, make_uint4(0u, 0u, 0u, 0u));
                continue;
            }
            if (fast) {
                const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                for (int j = 0; j < per; j += 2) {
                    uint64_t y;
                    if (BYTES == 2) {
                        const uint32_t k = ENT ? max_nan_bf16x2(w[j / 2], low) : w[j / 2];
                        y = f2_pack(bf16_lo(k), bf16_hi(k));
                    } else {
                        const float p = __uint_as_float(w[j & 3]), q = __uint_as_float(w[(j + 1) & 3]), l = __uint_as_float(low);
                        y = ENT ? f2_pack(max_nan(p, l), max_nan(q, l)) : f2_pack(p, q);
                    }
                    const uint64_t d = f2_fma(f2_add(y, m2), c2, shift2);
                    float d0, d1;
                    f2_unpack(d, d0, d1);
                    const uint64_t p = f2_pack(ex2(d0), ex2(d1));
                    f2_unpack(f2_mul(p, ENT ? f2_fma(slope2, d, base2) : base2), f[j], f[j + 1]);
                }
                if (i == target_vec) {
                    const int at = (int)(target - cut.head - i * per);
#pragma unroll
                    for (int j = 0; j < per; ++j)
                        if (j == at) f[j] += g;
                }
            } else {
                L::unpack(v[u], f);
#pragma unroll
                for (int j = 0; j < per; ++j) f[j] = grad(f[j], cut.head + i * per + j);
            }
            st_stream(dbody + 16 * i, L::pack(f));
        }
    }
}

}  // namespace fp8q

using namespace fp8q;

namespace {

bool valid_temperature(float t) { return t >= 0x1p-20f && t <= 0x1p20f; }

// Bytes from the first row's first element to the last one's last.
size_t span(int64_t rows, int64_t cols, int64_t stride, int bytes) {
    return rows ? ((size_t)(rows - 1) * (size_t)stride + (size_t)cols) * (size_t)bytes : 0;
}

fp8q_status_t check_logits(int64_t rows, int64_t vocab, int64_t stride, int logit_bytes, int id_bytes, float temperature) {
    if (logit_bytes != 2 && logit_bytes != 4) return FP8Q_ERR_FORMAT;
    if (id_bytes != 4 && id_bytes != 8) return FP8Q_ERR_FORMAT;
    if (vocab < 1 || vocab > FP8Q_MAX_VOCAB) return FP8Q_ERR_K;
    if (rows < 0 || rows >= (1ll << 27)) return FP8Q_ERR_SIZE;
    if (stride < vocab || (uint64_t)stride > FP8Q_MAX_ELEMENTS) return FP8Q_ERR_SIZE;
    if (rows > 0 && (uint64_t)stride > FP8Q_MAX_ELEMENTS / (uint64_t)rows) return FP8Q_ERR_SIZE;
    if (!valid_temperature(temperature)) return FP8Q_ERR_SIZE;
    return FP8Q_OK;
}

template <int BYTES, bool TOP, bool ENT, int NT, bool FAR>
fp8q_status_t launch_logprobs_kernel(const LpArgs& a, unsigned rows, unsigned ranks, size_t smem, cudaStream_t stream) {
    constexpr size_t kMax = TOP ? sizeof(LpTopShared<NT>) + (size_t)kLpPlaces * NT * 4 + (FAR ? sizeof(LpFar<NT>) : 0) : 0;
    static KernelCache cache;
    int resident = 0;
    const fp8q_status_t st = prepare_kernel(cache, token_logprobs_kernel<BYTES, TOP, ENT, NT, FAR>, NT, smem, kMax, &resident);
    if (st != FP8Q_OK) return st;
    return launch_clusters(token_logprobs_kernel<BYTES, TOP, ENT, NT, FAR>, rows * ranks, ranks, NT, smem, stream, a);
}

template <int BYTES, bool TOP, bool ENT, int NT>
fp8q_status_t launch_logprobs(LpArgs a, int64_t rows, cudaStream_t stream) {
    // blocks of a cluster share a row while there are few rows; clusters of four and eight do not fill every slot (72
    // rows of 151,669 binary32 logits with five alternatives in clusters of eight took 1.25 times as long as of four, 152
    // in clusters of four 1.29 times as long as of two; 10.9 and 19.1 us now)
    unsigned ranks = 1;
    const int64_t slots = kLpBlocksPerSm * sm_count();
    const int64_t steps = (a.vocab * BYTES + NT * kLpUnroll * 16 - 1) / (NT * kLpUnroll * 16);
    while (ranks < kLpMaxCluster && rows * ranks * 2 <= (ranks > 1 ? slots - slots / 16 : slots) && (int64_t)ranks * 2 <= steps) ranks *= 2;
    const int64_t mine = steps / ranks + 1;          // of one block, at most
    size_t smem = 0;
    if (TOP) {
        a.fold = (int)((mine + kLpPlaces - 1) / kLpPlaces);
        smem = sizeof(LpTopShared<NT>) + (size_t)((mine + a.fold - 1) / a.fold) * NT * 4;
    }
    if constexpr (NT == 256) {                       // rows of so many steps
        if (mine > kLpFarSteps<BYTES>) {
            a.far = (int)smem;
            return launch_logprobs_kernel<BYTES, TOP, ENT, NT, true>(a, (unsigned)rows, ranks, smem + sizeof(LpFar<NT>), stream);
        }
    }
    return launch_logprobs_kernel<BYTES, TOP, ENT, NT, false>(a, (unsigned)rows, ranks, smem, stream);
}

template <int BYTES, bool TOP, bool ENT>
fp8q_status_t launch_logprobs_size(const LpArgs& a, int64_t rows, cudaStream_t stream) {
    if (!TOP && a.vocab * BYTES <= kLpRowBytes && rows >= kLpRowsPerSm * sm_count())
        return launch(token_logprobs_rows_kernel<BYTES, ENT>, (unsigned)((rows + kLpRowThreads / 32 - 1) / (kLpRowThreads / 32)),
                      kLpRowThreads, 0, stream, a, rows);
    return a.vocab * BYTES <= 16384 ? launch_logprobs<BYTES, TOP, ENT, 128>(a, rows, stream)
                                    : launch_logprobs<BYTES, TOP, ENT, 256>(a, rows, stream);
}

template <int BYTES> fp8q_status_t launch_logprobs_kind(const LpArgs& a, int64_t rows, cudaStream_t stream) {
    if (a.top) return a.entropy ? launch_logprobs_size<BYTES, true, true>(a, rows, stream)
                                : launch_logprobs_size<BYTES, true, false>(a, rows, stream);
    return a.entropy ? launch_logprobs_size<BYTES, false, true>(a, rows, stream)
                     : launch_logprobs_size<BYTES, false, false>(a, rows, stream);
}

template <int BYTES, int NT> fp8q_status_t launch_backward_size(const LpGradArgs& a, bool vec, unsigned grid, cudaStream_t stream) {
    const bool ent = a.dentropy != nullptr;
    if (vec)
        return ent ? launch(token_logprobs_backward_kernel<BYTES, true, true, NT>, grid, kLpGradThreads, 0, stream, a)
                   : launch(token_logprobs_backward_kernel<BYTES, false, true, NT>, grid, kLpGradThreads, 0, stream, a);
    return ent ? launch(token_logprobs_backward_kernel<BYTES, true, false, NT>, grid, kLpGradThreads, 0, stream, a)
               : launch(token_logprobs_backward_kernel<BYTES, false, false, NT>, grid, kLpGradThreads, 0, stream, a);
}
template <int BYTES> fp8q_status_t launch_backward(LpGradArgs a, bool vec, cudaStream_t stream) {
    const int64_t bytes = a.vocab * BYTES;
    if (bytes <= kLpGradMedium && a.rows >= (bytes <= kLpGradShort ? kLpGradShortRowsPerSm : kLpGradMediumRowsPerSm) * sm_count()) {
        a.parts = 1;
        return launch_backward_size<BYTES, 32>(a, vec, (unsigned)((a.rows + kLpGradThreads / 32 - 1) / (kLpGradThreads / 32)), stream);
    }
    const int64_t per_block = (int64_t)kLpGradThreads * kLpGradUnroll * 16 / BYTES;
    const int64_t parts = (a.vocab + per_block - 1) / per_block, most = 0x7FFFFFFFll / a.rows;
    a.parts = (unsigned)(parts < most ? parts : most);
    return launch_backward_size<BYTES, kLpGradThreads>(a, vec, (unsigned)a.rows * a.parts, stream);
}

// A row's ids and numbers are read and written one by one, so that their own size is all the alignment they need.
bool aligned_for(const void* p, int bytes, unsigned flags) {
    return reinterpret_cast<uintptr_t>(p) % (flags & FP8Q_ELEMENT_ALIGNED ? (unsigned)bytes : 16u) == 0;
}

fp8q_status_t logprobs_entry(const void* logits, int logit_bytes, int64_t rows, int64_t vocab, int64_t stride, const void* targets,
                             int id_bytes, float temperature, int top, float* logprobs, float* entropy, float* top_logprobs,
                             int32_t* top_ids, float* stats, unsigned flags, fp8q_stream_t stream) {
    if (flags & ~FP8Q_ELEMENT_ALIGNED) return FP8Q_ERR_FLAGS;
    const fp8q_status_t st = check_logits(rows, vocab, stride, logit_bytes, id_bytes, temperature);
    if (st != FP8Q_OK) return st;
    if (top < 0 || top > FP8Q_MAX_TOP || top > vocab) return FP8Q_ERR_K;
    if (rows == 0) return FP8Q_OK;
    if (!logits || (targets == nullptr) != (logprobs == nullptr)) return FP8Q_ERR_NULL;
    if ((top > 0) != (top_logprobs != nullptr) || (top > 0) != (top_ids != nullptr)) return FP8Q_ERR_NULL;
    if (!logprobs && !entropy && !top && !stats) return FP8Q_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(logits) % (unsigned)logit_bytes) return FP8Q_ERR_ALIGN;
    if (!aligned_for(targets, id_bytes, flags)) return FP8Q_ERR_ALIGN;
    for (const void* p : {(const void*)logprobs, (const void*)entropy, (const void*)top_logprobs, (const void*)top_ids, (const void*)stats})
        if (!aligned_for(p, 4, flags)) return FP8Q_ERR_ALIGN;
    const size_t r = (size_t)rows;
    const Range outs[] = {{logprobs, 4 * r}, {entropy, 4 * r}, {top_logprobs, 4 * r * top}, {top_ids, 4 * r * top},
                          {stats, 8 * r}};
    const Range ins[] = {{logits, span(rows, vocab, stride, logit_bytes)}, {targets, r * id_bytes}};
    if (any_alias(outs, 5, ins, 2)) return FP8Q_ERR_ALIAS;
    const LpArgs a = {logits, targets, id_bytes == 8, vocab, stride, temperature,
                      (float)(1.44269504088896340736 / (double)temperature), top, 1, 0, logprobs, entropy, top_logprobs, top_ids, stats};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return logit_bytes == 2 ? launch_logprobs_kind<2>(a, rows, s) : launch_logprobs_kind<4>(a, rows, s);
}

fp8q_status_t logprobs_backward_entry(const void* logits, int logit_bytes, int64_t rows, int64_t vocab, int64_t stride,
                                      const void* targets, int id_bytes, float temperature, const float* stats,
                                      const float* dlogprobs, const float* entropy, const float* dentropy, void* dlogits,
                                      int64_t dstride, unsigned flags, fp8q_stream_t stream) {
    if (flags & ~FP8Q_ELEMENT_ALIGNED) return FP8Q_ERR_FLAGS;
    fp8q_status_t st = check_logits(rows, vocab, stride, logit_bytes, id_bytes, temperature);
    if (st == FP8Q_OK) st = check_logits(rows, vocab, dstride, logit_bytes, id_bytes, temperature);
    if (st != FP8Q_OK) return st;
    if (rows == 0) return FP8Q_OK;
    if (!logits || !stats || !dlogits) return FP8Q_ERR_NULL;
    if ((targets == nullptr) != (dlogprobs == nullptr) || (entropy == nullptr) != (dentropy == nullptr)) return FP8Q_ERR_NULL;
    if (!dlogprobs && !dentropy) return FP8Q_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(logits) % (unsigned)logit_bytes || reinterpret_cast<uintptr_t>(dlogits) % (unsigned)logit_bytes)
        return FP8Q_ERR_ALIGN;
    if (!aligned_for(targets, id_bytes, flags)) return FP8Q_ERR_ALIGN;
    for (const float* p : {stats, dlogprobs, entropy, dentropy})
        if (!aligned_for(p, 4, flags)) return FP8Q_ERR_ALIGN;
    const size_t r = (size_t)rows;
    const Range out[] = {{dlogits, span(rows, vocab, dstride, logit_bytes)}};
    const bool in_place = dlogits == logits && dstride == stride;
    const Range ins[] = {{in_place ? nullptr : logits, span(rows, vocab, stride, logit_bytes)}, {targets, r * id_bytes},
                         {stats, 8 * r}, {dlogprobs, 4 * r}, {entropy, 4 * r}, {dentropy, 4 * r}};
    if (any_alias(out, 1, ins, 6)) return FP8Q_ERR_ALIAS;
    const LpGradArgs a = {logits, targets, id_bytes == 8, rows, vocab, stride, dstride, (float)(1.0 / (double)temperature),
                          (float)(1.44269504088896340736 / (double)temperature), stats, dlogprobs, entropy, dentropy, dlogits, 1};
    const uintptr_t apart = reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(dlogits);
    const bool vec = apart % 16 == 0 && (rows == 1 || (uint64_t)(stride - dstride) * (unsigned)logit_bytes % 16 == 0);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return logit_bytes == 2 ? launch_backward<2>(a, vec, s) : launch_backward<4>(a, vec, s);
}

}  // namespace

extern "C" fp8q_status_t fp8q_token_logprobs(const void* logits, int logit_bytes, int64_t rows, int64_t vocab, int64_t stride,
                                             const void* targets, int id_bytes, float temperature, int top,
                                             float* logprobs, float* entropy, float* top_logprobs, int32_t* top_ids,
                                             float* stats, fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_token_logprobs");
    return logprobs_entry(logits, logit_bytes, rows, vocab, stride, targets, id_bytes, temperature, top, logprobs, entropy,
                          top_logprobs, top_ids, stats, 0, stream);
}

extern "C" fp8q_status_t fp8q_token_logprobs_ex(const void* logits, int logit_bytes, int64_t rows, int64_t vocab, int64_t stride,
                                                const void* targets, int id_bytes, float temperature, int top,
                                                float* logprobs, float* entropy, float* top_logprobs, int32_t* top_ids,
                                                float* stats, unsigned int flags, fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_token_logprobs_ex");
    return logprobs_entry(logits, logit_bytes, rows, vocab, stride, targets, id_bytes, temperature, top, logprobs, entropy,
                          top_logprobs, top_ids, stats, flags, stream);
}

extern "C" fp8q_status_t fp8q_token_logprobs_backward(const void* logits, int logit_bytes, int64_t rows, int64_t vocab,
                                                      int64_t stride, const void* targets, int id_bytes, float temperature,
                                                      const float* stats, const float* dlogprobs, const float* entropy,
                                                      const float* dentropy, void* dlogits, int64_t dstride,
                                                      fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_token_logprobs_backward");
    return logprobs_backward_entry(logits, logit_bytes, rows, vocab, stride, targets, id_bytes, temperature, stats, dlogprobs,
                                   entropy, dentropy, dlogits, dstride, 0, stream);
}

extern "C" fp8q_status_t fp8q_token_logprobs_backward_ex(const void* logits, int logit_bytes, int64_t rows, int64_t vocab,
                                                         int64_t stride, const void* targets, int id_bytes,
                                                         float temperature, const float* stats, const float* dlogprobs,
                                                         const float* entropy, const float* dentropy, void* dlogits,
                                                         int64_t dstride, unsigned int flags, fp8q_stream_t stream) {
    FP8Q_NVTX_RANGE("fp8q_token_logprobs_backward_ex");
    return logprobs_backward_entry(logits, logit_bytes, rows, vocab, stride, targets, id_bytes, temperature, stats, dlogprobs,
                                   entropy, dentropy, dlogits, dstride, flags, stream);
}
