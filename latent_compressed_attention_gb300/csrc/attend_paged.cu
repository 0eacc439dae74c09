// Attention of each sequence's new tokens over the paged latent cache (r = 512, d_v = 128).
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kR = 512, kDV = 128;
constexpr float kLog2e = 1.4426950408889634f;

// Which cache rows a token sees: [0, head) and [lo, hi), and of the rows from `tree` on those whose bit is set.
struct Sight {
    int head, lo, hi, tree;
    unsigned long long bits;
    __device__ bool sees(int u) const {
        return u < tree ? (u < head || u >= lo) && u < hi : u - tree < 64 && ((bits >> (u - tree)) & 1);
    }
};

__device__ Sight sight(const AttendPagedArgs &p, int b, int t, int len) {
    Sight s;
    if (p.parents) {
        const int *const up = p.parents + static_cast<long long>(b) * p.T;
        int depth = -1;
        for (int a = t; a >= 0; ++depth) {
            const int q = up[a];
            if (q < -1 || q >= a) record_error(p.dev_err, kDevErrBounds);
            a = q < a ? max(q, -1) : -1;
        }
        s.bits = 0;
        int d = depth;
        for (int a = t; a >= 0; --d) {
            if (p.window == 0 || depth - d < p.window || len + d < p.sinks) s.bits |= 1ull << a;
            const int q = up[a];
            a = q < a ? max(q, -1) : -1;
        }
        s.tree = s.hi = len;
        s.lo = p.window ? max(len + depth - p.window + 1, 0) : 0;
    } else {
        s.bits = 0;
        s.hi = s.tree = len + t + 1;
        s.lo = p.window ? max(len + t - p.window + 1, 0) : 0;
    }
    s.head = min(p.sinks, s.lo);
    return s;
}

__global__ void __launch_bounds__(256) attend_paged_simple_kernel(const AttendPagedArgs p) {
    const int h = blockIdx.x % p.H, t = blockIdx.x / p.H % p.T, b = blockIdx.x / (p.H * p.T);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    const int len = p.lens[b], count = p.counts ? p.counts[b] : p.T;
    const long long cap = static_cast<long long>(p.max_blocks) * p.bs;
    if (len < 0 || count < 0 || count > p.T || static_cast<long long>(len) + count > cap) {
        if (threadIdx.x == 0) record_error(p.dev_err, kDevErrBounds);
        return;
    }
    if (t >= count) return;
    const Sight s = sight(p, b, t, len);
    const long long row = (static_cast<long long>(b) * p.T + t) * p.H + h;
    const auto *q = static_cast<const __nv_bfloat16 *>(p.q_abs) + row * kR;
    float qv[16], o[16] = {};
    for (int i = 0; i < 16; ++i) qv[i] = __bfloat162float(q[lane * 16 + i]) * p.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    for (int u = warp; u < len + count; u += 8) {
        if (!s.sees(u)) continue;
        const int block = p.table[b * p.ld_table + u / p.bs];
        float c[16] = {}, dot = 0.f;
        if (block >= 0 && block < p.num_blocks) {
            const auto *src = static_cast<const __nv_bfloat16 *>(p.pool) +
                              (static_cast<long long>(block) * p.bs + u % p.bs) * p.ld_pool + lane * 16;
            for (int i = 0; i < 16; ++i) c[i] = __bfloat162float(src[i]);
        } else if (lane == 0) {
            record_error(p.dev_err, kDevErrBounds);
        }
        for (int i = 0; i < 16; ++i) dot = fmaf(qv[i], c[i], dot);
        for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        const float top = fmaxf(m, dot), f = exp2f(m - top), w = exp2f(dot - top);
        for (int i = 0; i < 16; ++i) o[i] = o[i] * f + w * c[i];
        l = l * f + w;
        m = top;
    }
    __shared__ float sm[8], sl[8], so[8][kR], lat[kR];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    for (int i = 0; i < 16; ++i) so[warp][lane * 16 + i] = o[i];
    __syncthreads();
    float top = -INFINITY, all = 0.f;
    for (int w = 0; w < 8; ++w) top = fmaxf(top, sm[w]);
    for (int w = 0; w < 8; ++w) all += sl[w] > 0.f || sl[w] != sl[w] ? sl[w] * exp2f(sm[w] - top) : 0.f;
    for (int i = threadIdx.x; i < kR; i += 256) {
        float v = 0.f;
        for (int w = 0; w < 8; ++w) v += sl[w] > 0.f || sl[w] != sl[w] ? so[w][i] * exp2f(sm[w] - top) : 0.f;
        lat[i] = v / all;
    }
    __syncthreads();
    for (int v = warp; v < kDV; v += 8) {
        const auto *w = static_cast<const __nv_bfloat16 *>(p.w_uv) + (static_cast<long long>(h) * kDV + v) * kR;
        float x = 0.f;
        for (int i = lane; i < kR; i += 32) x = fmaf(lat[i], __bfloat162float(w[i]), x);
        for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (lane == 0) {
            if (p.gate) x /= 1.f + __expf(-__bfloat162float(static_cast<const __nv_bfloat16 *>(p.gate)[row * kDV + v]));
            static_cast<__nv_bfloat16 *>(p.out)[row * kDV + v] = __float2bfloat16(x);
        }
    }
}

}  // namespace

bool attend_paged_supports(int H, int d_v, int r) { return r == kR && d_v == kDV && H >= 1 && H <= 128; }

size_t attend_paged_workspace_bytes(long long, long long, int, int) { return 256; }

cudaError_t launch_attend_paged(const AttendPagedArgs &a, cudaStream_t s) {
    note_launch();
    return launch_dependent(attend_paged_simple_kernel, dim3(static_cast<unsigned>(a.B) * a.T * a.H), 256, 0, s, a);
}

}  // namespace mla
