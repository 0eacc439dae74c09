// Cached-latent decode over the fp4 latent cache (latent_fp4.cu): r = 512, d_v = 128, 1 <= H <= 96.
//
// Sequence b's absorbed query q_abs[b] (all H heads) attends to its cache rows [0, lens[b]); steps 2-4 of section
// "完整计算流（四步）" of the page "Gated MLA（矩阵吸收版）" follow: scores against c itself, softmax, the latent
// weighting by c itself, W_UV^T, gate.
//
// Split kernel: a warp takes one head and one of the `nsplit` runs of a sequence's rows; lane j holds latent elements
// 16j .. 16j + 15 and the warp keeps a running maximum, sum and weighted row, all fp32.
// Merge kernel: a block per (head, sequence) joins the runs with the log-sum-exp rule, multiplies by W_UV^T and applies
// the gate.
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kR = 512;
constexpr int kDV = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct Fp4Params {
    const __nv_bfloat16 *q_abs, *w_uv, *gate;
    const uint8_t *c4;
    long long ld;
    const int *lens;
    __nv_bfloat16 *out;
    float *ws_o, *ws_m, *ws_l;   // [nsplit][B][H] (x kR)
    int *err;
    int B, H, max_len, nsplit;
    float scale_log2;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__global__ void __launch_bounds__(128) fp4_split_kernel(const Fp4Params p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = static_cast<int>(blockIdx.x) * 4 + warp, split = blockIdx.y, b = blockIdx.z;
    if (h >= p.H) return;
    const int raw = __ldg(p.lens + b);
    if (raw < 0 || raw > p.max_len) record_error(p.err, kDevErrBounds);
    const int len = min(max(raw, 0), p.max_len);
    const int per = (len + p.nsplit - 1) / p.nsplit;
    const int k0 = static_cast<int>(min(static_cast<long long>(per) * split, static_cast<long long>(len)));
    const int k1 = min(len - k0, per) + k0;
    float q[16], o[16], m = -INFINITY, l = 0.f;
    const uint4 *qs = reinterpret_cast<const uint4 *>(p.q_abs + (static_cast<size_t>(b) * p.H + h) * kR) + lane * 2;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint4 v = __ldg(qs + half);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            q[8 * half + 2 * k] = __uint_as_float(w[k] << 16) * p.scale_log2;
            q[8 * half + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u) * p.scale_log2;
        }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
    for (int u = k0; u < k1; ++u) {
        const uint8_t *row = p.c4 + (static_cast<long long>(b) * p.max_len + u) * p.ld;
        const uint2 codes = __ldg(reinterpret_cast<const uint2 *>(row) + lane);
        const float scale = fp4_scale(__ldg(row + kR / 2 + (lane >> 1)));
        float c[16], (&lo)[8] = *reinterpret_cast<float (*)[8]>(c), (&hi)[8] = *reinterpret_cast<float (*)[8]>(c + 8);
        unpack_e2m1x8(codes.x, lo);
        unpack_e2m1x8(codes.y, hi);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += q[k] * (c[k] *= scale);
        s = warp_sum(s);
        const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - base), w = exp2f(s - base);
        l = l * f + w;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = o[k] * f + w * c[k];
        m = mn;
    }
    const size_t slot = (static_cast<size_t>(split) * p.B + b) * p.H + h;
    float4 *dst = reinterpret_cast<float4 *>(p.ws_o + slot * kR) + lane * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    if (lane == 0) {
        p.ws_m[slot] = m;
        p.ws_l[slot] = l;
    }
}

__global__ void __launch_bounds__(128) fp4_merge_kernel(const Fp4Params p) {
    __shared__ float o_lat[kR];
    const int h = blockIdx.x, b = blockIdx.y, t = threadIdx.x;
    const int len = min(max(__ldg(p.lens + b), 0), p.max_len);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    auto slot = [&](int i) { return (static_cast<size_t>(i) * p.B + b) * p.H + h; };
    for (int i = 0; i < p.nsplit; ++i) m = fmaxf(m, p.ws_m[slot(i)]);
    const float base = m == -INFINITY ? 0.f : m;
    for (int i = 0; i < p.nsplit; ++i) {
        const float w = exp2f(p.ws_m[slot(i)] - base), li = p.ws_l[slot(i)];
        l += w * li;
        if (w == 0.f && li == li) continue;
        const float4 v = *(reinterpret_cast<const float4 *>(p.ws_o + slot(i) * kR) + t);
        o[0] += w * v.x, o[1] += w * v.y, o[2] += w * v.z, o[3] += w * v.w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) o_lat[4 * t + k] = len > 0 ? o[k] / l : 0.f;
    __syncthreads();
    float y = 0.f;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p.w_uv + (static_cast<size_t>(h) * kDV + t) * kR);
    for (int j = 0; j < kR / 2; ++j) {
        const uint32_t v = __ldg(w + j);
        y += __uint_as_float(v << 16) * o_lat[2 * j] + __uint_as_float(v & 0xFFFF0000u) * o_lat[2 * j + 1];
    }
    const size_t at = (static_cast<size_t>(b) * p.H + h) * kDV + t;
    if (p.gate) y /= 1.f + exp2f(-__bfloat162float(p.gate[at]) * kLog2e);
    p.out[at] = __float2bfloat16(y);
}

int splits(int B, int H, int max_len, int num_sms) {
    const long long warps = static_cast<long long>(num_sms) * 32, want = (warps + B * H - 1) / (static_cast<long long>(B) * H);
    const long long most = (max_len + 63) / 64;
    const long long n = want < most ? want : most;
    return static_cast<int>(n < 1 ? 1 : (n > 4096 ? 4096 : n));
}

}  // namespace

size_t decode_fp4_workspace_bytes(int B, int H, int max_len, int num_sms) {
    return static_cast<size_t>(splits(B, H, max_len, num_sms)) * B * H * (kR + 2) * sizeof(float);
}

cudaError_t launch_decode_fp4(const DecodeArgs &a, cudaStream_t s) {
    if (!decode_bf16_supports(a.H, a.d_v, a.r) || a.B > 65535) return cudaErrorInvalidValue;
    Fp4Params p;
    p.q_abs = static_cast<const __nv_bfloat16 *>(a.q_abs);
    p.w_uv = static_cast<const __nv_bfloat16 *>(a.w_uv);
    p.gate = static_cast<const __nv_bfloat16 *>(a.gate);
    p.c4 = static_cast<const uint8_t *>(a.c_cache);
    p.ld = a.ld_cache;
    p.lens = a.lens;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.nsplit = splits(a.B, a.H, a.max_len, a.num_sms);
    const size_t slots = static_cast<size_t>(p.nsplit) * a.B * a.H;
    p.ws_o = static_cast<float *>(a.workspace);
    p.ws_m = p.ws_o + slots * kR;
    p.ws_l = p.ws_m + slots;
    p.err = a.dev_err;
    p.B = a.B;
    p.H = a.H;
    p.max_len = a.max_len;
    p.scale_log2 = a.scale * kLog2e;
    note_launch();
    fp4_split_kernel<<<dim3((a.H + 3) / 4, p.nsplit, a.B), 128, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    note_launch();
    fp4_merge_kernel<<<dim3(a.H, a.B), 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mla
