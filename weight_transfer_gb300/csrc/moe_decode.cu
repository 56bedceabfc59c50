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

namespace fp8q {

constexpr int kMdThreads = 256;
constexpr int kMdWarps = kMdThreads / 32;

struct MdArgs {
    const uint8_t *codes, *scales;                  // [tokens, k], [tokens, k / 32]
    const void* ids;
    int id64;
    const float* weights;                           // [tokens, topk]
    int tokens, topk, experts;
    int64_t n, k;
    const uint8_t *gate, *gate_scales, *up, *up_scales, *down, *down_scales;
    float* h;                                       // [tokens * topk, n]
    uint16_t* out;                                  // [tokens, k]
};

__device__ __forceinline__ int expert_of(const MdArgs& a, int64_t i) {
    const int64_t id = a.id64 ? (int64_t)static_cast<const long long*>(a.ids)[i] : (int64_t)static_cast<const int*>(a.ids)[i];
    return id >= 0 && id < a.experts ? (int)id : -1;
}

// 2^(s - 127), NaN for 255.
__device__ __forceinline__ float e8m0(uint32_t s) {
    return s == 255u ? __uint_as_float(0x7FFFFFFFu) : s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}

// Place of scale (r, j) in a matrix of the 128 x 4 tiled layout.
__device__ __forceinline__ int64_t tiled(int64_t r, int64_t j, int64_t tiles) {
    return ((r >> 7) * tiles + (j >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (j & 3);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ void decode32(const uint8_t* p, float (&f)[32]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 16);
    decode_fp8x4<kE4M3>(a.x, f); decode_fp8x4<kE4M3>(a.y, f + 4); decode_fp8x4<kE4M3>(a.z, f + 8); decode_fp8x4<kE4M3>(a.w, f + 12);
    decode_fp8x4<kE4M3>(b.x, f + 16); decode_fp8x4<kE4M3>(b.y, f + 20); decode_fp8x4<kE4M3>(b.z, f + 24); decode_fp8x4<kE4M3>(b.w, f + 28);
}

// A warp takes one feature of one choice.
__global__ void __launch_bounds__(kMdThreads) moe_decode_up_kernel(const MdArgs a) {
    const int lane = (int)(threadIdx.x & 31u);
    dependency_wait();
    allow_dependents();
    const int64_t choice = blockIdx.x / (unsigned)((a.n + kMdWarps - 1) / kMdWarps);
    const int64_t f = (blockIdx.x % (unsigned)((a.n + kMdWarps - 1) / kMdWarps)) * kMdWarps + (threadIdx.x >> 5);
    const int e = expert_of(a, choice);
    if (f >= a.n || e < 0) return;
    const int64_t kb = a.k / 32, tiles = (kb + 3) / 4, per = (a.n + 127) / 128 * tiles * 512, token = choice / a.topk;
    const uint8_t *x = a.codes + token * a.k, *xs = a.scales + token * kb;
    const uint8_t *g = a.gate + ((int64_t)e * a.n + f) * a.k, *gs = a.gate_scales + e * per;
    const uint8_t *u = a.up + ((int64_t)e * a.n + f) * a.k, *us = a.up_scales + e * per;
    float sg = 0.0f, su = 0.0f;
    for (int64_t b = lane; b < kb; b += 32) {
        float xv[32], w[32];
        decode32(x + 32 * b, xv);
        const float sx = e8m0(xs[b]);
        decode32(g + 32 * b, w);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s = __fmaf_rn(w[i], xv[i], s);
        sg += s * sx * e8m0(gs[tiled(f, b, tiles)]);
        decode32(u + 32 * b, w);
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s = __fmaf_rn(w[i], xv[i], s);
        su += s * sx * e8m0(us[tiled(f, b, tiles)]);
    }
    sg = warp_sum(sg);
    su = warp_sum(su);
    if (lane == 0) a.h[choice * a.n + f] = sg / (1.0f + expf(-sg)) * su;
}

// A warp takes one output feature of one token.
__global__ void __launch_bounds__(kMdThreads) moe_decode_down_kernel(const MdArgs a) {
    const int lane = (int)(threadIdx.x & 31u);
    dependency_wait();
    allow_dependents();
    const int64_t token = blockIdx.x / (unsigned)((a.k + kMdWarps - 1) / kMdWarps);
    const int64_t f = (blockIdx.x % (unsigned)((a.k + kMdWarps - 1) / kMdWarps)) * kMdWarps + (threadIdx.x >> 5);
    if (f >= a.k) return;
    const int64_t nb = a.n / 32, tiles = (nb + 3) / 4, per = (a.k + 127) / 128 * tiles * 512;
    float out = 0.0f;
    for (int j = 0; j < a.topk; ++j) {
        const int64_t choice = token * a.topk + j;
        const int e = expert_of(a, choice);
        if (e < 0) continue;
        const uint8_t *d = a.down + ((int64_t)e * a.k + f) * a.n, *ds = a.down_scales + e * per;
        const float* h = a.h + choice * a.n;
        float sum = 0.0f;
        for (int64_t b = lane; b < nb; b += 32) {
            float w[32];
            decode32(d + 32 * b, w);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) s = __fmaf_rn(w[i], __ldcg(h + 32 * b + i), s);
            sum += s * e8m0(ds[tiled(f, b, tiles)]);
        }
        out = __fmaf_rn(a.weights[choice], warp_sum(sum), out);
    }
    if (lane == 0) a.out[token * a.k + f] = (uint16_t)pack_bf16x2(out, 0.0f);
}

}  // namespace fp8q

using namespace fp8q;

namespace {

size_t workspace_of(int64_t tokens, int topk, int64_t n) { return (size_t)tokens * (size_t)topk * (size_t)n * sizeof(float); }

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
    const MdArgs a = {codes, scales, ids, id_bytes == 8, weights, (int)tokens, topk, experts, n, k, gate_codes, gate_scales,
                      up_codes, up_scales, down_codes, down_scales, static_cast<float*>(workspace), static_cast<uint16_t*>(out_bf16)};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned up_blocks = (unsigned)(tokens * topk * ((n + kMdWarps - 1) / kMdWarps));
    const unsigned down_blocks = (unsigned)(tokens * ((k + kMdWarps - 1) / kMdWarps));
    const fp8q_status_t st = launch(moe_decode_up_kernel, up_blocks, kMdThreads, 0, s, a);
    return st != FP8Q_OK ? st : launch(moe_decode_down_kernel, down_blocks, kMdThreads, 0, s, a);
}
