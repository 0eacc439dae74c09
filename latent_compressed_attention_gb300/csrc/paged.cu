// The paged latent cache: block tables and slot maps kept on the GPU, and latent rows written through them.
//
// Only the latent c is cached (page "Gated MLA（矩阵吸收版）", KV-cache table in section "形状与参数对比": r values
// per token).  Here its rows live in a pool of blocks of `bs` rows, and sequence b's row u is row u % bs of block
// table[b][u / bs], so that sequences of any length share the pool.
//
//   reserve  need_b = ceil((lens_b + counts_b) / bs) blocks.  Sequences that hold more give the rest up, numbered
//            k = 0 .. R - 1 in order of (sequence, index); those that need more take, in the same order, number k of what
//            was given up for k < R and then free[F - 1 - (k - R)], the top of the free stack.  What nobody took goes to
//            free[F + R - 1 - k], so that number A, the first left over, is not on top of number A + 1 by chance: a
//            growth and the same shrinking leave the stack as it was.
//   append   pool row slots[i] = c[i].
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kReserveThreads = 1024;

struct ReserveParams {
    const int *lens, *counts;
    int *table, *held, *free_blocks, *free_count, *slots;
    long long ld_table;
    int B, T, max_blocks, capacity, bs;
    int *err;
};

// Number of the sequence whose part of [0, pre[B]) holds k.
__device__ __forceinline__ int owner(const int *pre, int B, int k) {
    int lo = 0, hi = B;   // pre[lo] <= k < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        (pre[mid] <= k ? lo : hi) = mid;
    }
    return lo;
}

template <bool kCluster>
__device__ __forceinline__ void sync_all() {
    if constexpr (kCluster) {
        __threadfence();
        cluster_sync_all();
    } else {
        __syncthreads();
    }
}

// Every CTA adds up all sequences' needs (they fit one CTA's threads); after a barrier, when no one reads the old state
// any more, all of them change it, each thread a block at a time.
template <bool kCluster>
__global__ void __launch_bounds__(kReserveThreads) reserve_latent_blocks_kernel(const ReserveParams p) {
    extern __shared__ int pre[];   // [B + 1] blocks taken, [B + 1] blocks given up by the sequences before
    __shared__ long long warp_sum[2][32];
    __shared__ long long all_sum[2];
    int *const take = pre, *const give = pre + p.B + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int F = *p.free_count;
    const int per = (p.B + kReserveThreads - 1) / kReserveThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    auto need = [&](int b) {
        return static_cast<int>((static_cast<long long>(p.lens[b]) + p.counts[b] + p.bs - 1) / p.bs);
    };
    long long sum[2] = {0, 0};
    bool bad = F < 0 || F > p.capacity;
    for (int b = b0; b < b1; ++b) {
        const int len = p.lens[b], count = p.counts[b], h = p.held[b];
        const long long n = (static_cast<long long>(len) + count + p.bs - 1) / p.bs;
        bad |= len < 0 || count < 0 || (p.slots != nullptr && count > p.T) || n > p.max_blocks || h < 0 || h > p.max_blocks;
        sum[0] += max(n - h, 0ll), sum[1] += max(h - n, 0ll);
    }
    long long before[2] = {sum[0], sum[1]};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, before[i], off);
            if (lane >= off) before[i] += v;
        }
        if (lane == 31) warp_sum[i][warp] = before[i];
    }
    bad = __syncthreads_or(bad);
    if (warp < 2) {
        const long long v = warp_sum[warp][lane];
        long long incl = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long w = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += w;
        }
        warp_sum[warp][lane] = incl - v;
        if (lane == 31) all_sum[warp] = incl;
    }
    __syncthreads();
    const long long A = all_sum[0], R = all_sum[1];
    bad |= A > F + R || F + R - A > p.capacity;   // what does not fit changes nothing
    if (!bad) {
        long long t = warp_sum[0][warp] + before[0] - sum[0], g = warp_sum[1][warp] + before[1] - sum[1];
        for (int b = b0; b < b1; ++b) {
            take[b] = static_cast<int>(t), give[b] = static_cast<int>(g);
            const int n = need(b), h = p.held[b];
            t += max(n - h, 0), g += max(h - n, 0);
        }
        if (tid == 0) take[p.B] = static_cast<int>(A), give[p.B] = static_cast<int>(R);
    }
    const int step = kCluster ? kReserveThreads * static_cast<int>(gridDim.x) : kReserveThreads;
    const int me = kCluster ? tid + kReserveThreads * static_cast<int>(blockIdx.x) : tid;
    if (bad) {
        if (me == 0) record_error(p.err, kDevErrBounds);
        if (p.slots != nullptr)
            for (long long i = me; i < static_cast<long long>(p.B) * p.T; i += step) p.slots[i] = -1;
        return;
    }
    sync_all<kCluster>();   // the prefix sums are there; held and free_count have been read
    const int a_all = static_cast<int>(A), r_all = static_cast<int>(R);
    // Only sequences that keep no more than they need take blocks, and only the others give some up: the entries read
    // here and those written are of different sequences, as are the stack's places below F and from F on.
    auto given = [&](int k) {
        const int b = owner(give, p.B, k);
        return p.table[b * p.ld_table + need(b) + (k - give[b])];
    };
    for (int k = me; k < a_all; k += step) {
        const int b = owner(take, p.B, k), n = need(b), had = n - (take[b + 1] - take[b]);
        p.table[b * p.ld_table + had + (k - take[b])] = k < r_all ? given(k) : p.free_blocks[F - 1 - (k - r_all)];
    }
    for (int k = a_all + me; k < r_all; k += step) p.free_blocks[F + r_all - 1 - k] = given(k);
    for (int b = me; b < p.B; b += step) p.held[b] = need(b);
    if (me == 0) *p.free_count = F + r_all - a_all;
    if (p.slots == nullptr) return;
    sync_all<kCluster>();   // the tables are whole
    const int quads = (p.T + 3) / 4;
    const bool wide = p.T % 4 == 0;
    for (long long i = me; i < static_cast<long long>(p.B) * quads; i += step) {
        const int b = static_cast<int>(i / quads), t0 = static_cast<int>(i - static_cast<long long>(b) * quads) * 4;
        const int len = p.lens[b], count = p.counts[b];
        int s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s[k] = -1;
            if (t0 + k < count) {
                const int u = len + t0 + k, j = u / p.bs;
                const long long row = static_cast<long long>(p.table[b * p.ld_table + j]) * p.bs + (u - j * p.bs);
                if (row >= 0 && row <= 0x7FFFFFFF)
                    s[k] = static_cast<int>(row);
                else
                    record_error(p.err, kDevErrBounds);
            }
        }
        int *const dst = p.slots + static_cast<long long>(b) * p.T + t0;
        if (wide) {
            *reinterpret_cast<int4 *>(dst) = make_int4(s[0], s[1], s[2], s[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (t0 + k < p.T) dst[k] = s[k];
        }
    }
}

constexpr int kAppendThreads = 256;
constexpr int kMany = 4;   // pieces of 8 elements that a thread of a long run has in flight

struct AppendParams {
    const void *c;
    __nv_bfloat16 *pool;
    const int *slots;
    long long ld_c, ld_pool, pool_rows, pieces;
    int per_row;
    int *err;
};

// A stream bound by HBM: neighbouring lanes take neighbouring pieces of 8 elements.
template <typename T, int N>
__global__ void __launch_bounds__(kAppendThreads) append_latent_paged_kernel(const AppendParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const T *const c = static_cast<const T *>(p.c);
    const long long i0 = static_cast<long long>(blockIdx.x) * (N * kAppendThreads) + threadIdx.x;
    uint4 v[N];
    int slot[N], piece[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const long long i = i0 + j * kAppendThreads;
        slot[j] = -1;
        if (i >= p.pieces) continue;
        const long long row = i / p.per_row;
        piece[j] = static_cast<int>(i - row * p.per_row);
        slot[j] = __ldg(p.slots + row);
        const T *const src = c + row * p.ld_c + piece[j] * 8;
        if constexpr (sizeof(T) == 2) {
            v[j] = __ldcs(reinterpret_cast<const uint4 *>(src));
        } else {
            const float4 a = __ldcs(reinterpret_cast<const float4 *>(src));
            const float4 b = __ldcs(reinterpret_cast<const float4 *>(src) + 1);
            v[j] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (slot[j] < 0 || slot[j] >= p.pool_rows) {
            if (slot[j] != -1) record_error(p.err, kDevErrBounds);
            continue;
        }
        *reinterpret_cast<uint4 *>(p.pool + slot[j] * p.ld_pool + piece[j] * 8) = v[j];
    }
}

}  // namespace

cudaError_t launch_reserve_latent_blocks(const ReserveArgs &a, cudaStream_t s) {
    const ReserveParams p{a.lens, a.counts, a.table, a.held, a.free_blocks, a.free_count, a.T > 0 ? a.slots : nullptr,
                          a.ld_table, a.B, a.T, a.max_blocks, a.capacity, a.bs, a.dev_err};
    const size_t smem = 2 * (static_cast<size_t>(a.B) + 1) * sizeof(int);
    // one CTA up to 8192 slots; above, a cluster of 8
    const bool many = static_cast<long long>(a.B) * a.T > 8192;
    auto *kernel = many ? reserve_latent_blocks_kernel<true> : reserve_latent_blocks_kernel<false>;
    if (smem > 40000) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    note_launch();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(many ? 8 : 1);
    cfg.blockDim = dim3(kReserveThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 8;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = many ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_append_latent_paged(const AppendPagedArgs &a, cudaStream_t s) {
    AppendParams p{a.c, static_cast<__nv_bfloat16 *>(a.pool), a.slots, a.ld_c, a.ld_pool, a.pool_rows, 0, a.r / 8, a.dev_err};
    p.pieces = a.rows * p.per_row;
    // four pieces per thread from a wave of the GPU's threads on, one below
    const bool many = p.pieces >= 152ll * 2048;
    const long long blocks = (p.pieces + kAppendThreads * (many ? kMany : 1) - 1) / (kAppendThreads * (many ? kMany : 1));
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    const auto go = [&](auto kernel) {
        note_launch();
        return launch_dependent(kernel, dim3(static_cast<unsigned>(blocks)), kAppendThreads, 0, s, p);
    };
    if (a.f32) return many ? go(append_latent_paged_kernel<float, kMany>) : go(append_latent_paged_kernel<float, 1>);
    return many ? go(append_latent_paged_kernel<__nv_bfloat16, kMany>) : go(append_latent_paged_kernel<__nv_bfloat16, 1>);
}

}  // namespace mla
