// The paged latent cache: block tables and slot maps kept on the GPU, and latent rows written through them.
//
// Only the latent c is cached (page "Gated MLA（矩阵吸收版）", KV-cache table in section "形状与参数对比": r values
// per token).  Here its rows live in a pool of blocks of `bs` rows, and sequence b's row u is row u % bs of block
// table[b][u / bs], so that sequences of any length share the pool.
//
//   reserve  need_b = ceil((lens_b + counts_b) / bs) blocks.  Sequences that hold more give the rest up, numbered
//            k = 0 .. R - 1 in order of (sequence, index); those that need more take, in the same order, number k of what
//            was given up for k < R and then free[F - 1 - (k - R)], the top of the free stack.  What nobody took goes to
//            free[F + R - 1 - k], the first one given up on top, so that a growth and the same shrinking leave the
//            stack as it was.
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

constexpr int kBatch = 4;   // blocks that a thread moves at a time, their searches and loads in flight together
constexpr long long kMostMoved = 0x7FFFFFFFll - kBatch * kReserveThreads;   // their numbers, and a turn of the CTA's more, fit int

// Of each k the sequence whose part of [0, pre[B]) holds it.  `top`: the largest power of two up to B.
__device__ __forceinline__ void owners(const int *pre, int B, int top, const int (&k)[kBatch], int (&b)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) b[i] = 0;
    for (int s = top; s > 0; s >>= 1)
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (b[i] + s < B && pre[b[i] + s] <= k[i]) b[i] += s;
}

// The slots of four tokens from t0 on.
__device__ __forceinline__ void write_slots(const ReserveParams &p, int b, int t0, int len, int count) {
    const int *const table = p.table + b * p.ld_table;
    int s[4], j = (len + t0) / p.bs, off = len + t0 - j * p.bs;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        s[k] = -1;
        if (t0 + k < count) {
            const long long row = static_cast<long long>(table[j]) * p.bs + off;
            if (row >= 0 && row <= 0x7FFFFFFF)
                s[k] = static_cast<int>(row);
            else
                record_error(p.err, kDevErrBounds);
        }
        if (++off == p.bs) off = 0, ++j;
    }
    int *const dst = p.slots + static_cast<long long>(b) * p.T + t0;
    if (p.T % 4 == 0) {
        *reinterpret_cast<int4 *>(dst) = make_int4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (t0 + k < p.T) dst[k] = s[k];
    }
}

// One CTA adds up all sequences' needs and, once no thread reads the old state any more, changes it, each thread a block at
// a time.  With kAll it maps the slots too; otherwise it maps each sequence's first one (-1 where there is none, or where
// nothing fits) and map_slots_kernel the others.
template <bool kAll>
__global__ void __launch_bounds__(kReserveThreads) reserve_latent_blocks_kernel(const ReserveParams p) {
    extern __shared__ int pre[];   // [B + 1] blocks taken, [B + 1] blocks given up by the sequences before; [B] needs
    __shared__ long long warp_sum[2][32];
    __shared__ long long all_sum[2];
    int *const take = pre, *const give = pre + p.B + 1, *const need = give + p.B + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int F = *p.free_count;
    const int per = (p.B + kReserveThreads - 1) / kReserveThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    const auto blocks = [&](int len, int count) {   // neither below 0
        const unsigned n = static_cast<unsigned>(len) + static_cast<unsigned>(count), q = n / static_cast<unsigned>(p.bs);
        return q + (n != q * p.bs ? 1 : 0);
    };
    long long sum[2] = {0, 0};
    bool bad = F < 0 || F > p.capacity;
    for (int b = b0; b < b1; ++b) {
        const int len = p.lens[b], count = p.counts[b], h = p.held[b];
        const long long n = len < 0 || count < 0 ? 0 : blocks(len, count);
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
    bad |= max(A, R) > kMostMoved;
    if (!bad) {
        long long t = warp_sum[0][warp] + before[0] - sum[0], g = warp_sum[1][warp] + before[1] - sum[1];
        for (int b = b0; b < b1; ++b) {
            const int n = static_cast<int>(blocks(p.lens[b], p.counts[b])), h = p.held[b];
            take[b] = static_cast<int>(t), give[b] = static_cast<int>(g), need[b] = n;
            t += max(n - h, 0), g += max(h - n, 0);
        }
        if (tid == 0) take[p.B] = static_cast<int>(A), give[p.B] = static_cast<int>(R);
    }
    const bool slots = p.slots != nullptr;
    const auto refuse = [&] {
        if (tid == 0) record_error(p.err, kDevErrBounds);
        const long long every = kAll ? 1 : p.T, n = slots ? static_cast<long long>(p.B) * p.T : 0;
        for (long long i = tid * every; i < n; i += kReserveThreads * every) p.slots[i] = -1;
    };
    if (bad) return refuse();
    __syncthreads();   // the prefix sums are there; held and free_count have been read
    const int a_all = static_cast<int>(A), r_all = static_cast<int>(R);
    // Only sequences that keep no more than they need take blocks, and only the others give some up: the entries read
    // here and those written are of different sequences, as are the stack's places below F and from F on.
    const int top = p.B > 0 ? 1 << (31 - __clz(p.B)) : 0;
    for (int k0 = tid; k0 < max(a_all, r_all); k0 += kBatch * kReserveThreads) {
        int k[kBatch], b[kBatch], block[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) k[i] = k0 + i * kReserveThreads;
        if (k0 < r_all) {   // number k of what was given up
            owners(give, p.B, top, k, b);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (k[i] < r_all) block[i] = p.table[b[i] * p.ld_table + need[b[i]] + (k[i] - give[b[i]])];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (k[i] >= r_all && k[i] < a_all) block[i] = p.free_blocks[F - 1 - (k[i] - r_all)];
        if (k0 < a_all) {
            owners(take, p.B, top, k, b);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (k[i] < a_all) p.table[b[i] * p.ld_table + need[b[i]] + k[i] - take[b[i] + 1]] = block[i];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (k[i] >= a_all && k[i] < r_all) p.free_blocks[F + r_all - 1 - k[i]] = block[i];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) bad |= k[i] < max(a_all, r_all) && block[i] < 0;
    }
    // A number below 0 is no block, and as one would serve another sequence.  What has been written lies behind what each
    // sequence holds and behind the stack's top: without the new held and free_count nothing has moved.
    if (__syncthreads_or(bad)) return refuse();
    for (int b = tid; b < p.B; b += kReserveThreads) p.held[b] = need[b];
    if (tid == 0) *p.free_count = F + r_all - a_all;
    if (!slots) return;
    __syncthreads();   // the tables are whole
    if constexpr (kAll) {
        const int quads = (p.T + 3) / 4, n = p.B * quads;
        for (int i = tid; i < n; i += kReserveThreads) {
            const int b = i / quads;
            write_slots(p, b, (i - b * quads) * 4, p.lens[b], p.counts[b]);
        }
    } else {
        for (int b = tid; b < p.B; b += kReserveThreads) {
            const int len = p.lens[b], j = len / p.bs;
            long long row = -1;
            if (p.counts[b] > 0) {
                row = static_cast<long long>(p.table[b * p.ld_table + j]) * p.bs + (len - j * p.bs);
                if (row < 0 || row > 0x7FFFFFFF) record_error(p.err, kDevErrBounds), row = -1;
            }
            p.slots[static_cast<long long>(b) * p.T] = static_cast<int>(row);
        }
    }
}

// The slots of 1024 tokens of a sequence.  Its first slot is there already: -1 where the sequence has none.
constexpr int kMapThreads = 256;
__global__ void __launch_bounds__(kMapThreads) map_slots_kernel(const ReserveParams p, unsigned per_seq) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int b = static_cast<int>(blockIdx.x / per_seq);
    const int t0 = static_cast<int>((blockIdx.x - b * per_seq) * kMapThreads + threadIdx.x) * 4;
    if (t0 >= p.T) return;
    const int first = *static_cast<const volatile int *>(p.slots + static_cast<long long>(b) * p.T);
    write_slots(p, b, t0, p.lens[b], first < 0 ? 0 : p.counts[b]);
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
    const size_t smem = (3 * static_cast<size_t>(a.B) + 2) * sizeof(int);
    // the one CTA maps up to 8192 slots itself
    const bool all = static_cast<long long>(a.B) * a.T <= 8192;
    auto *const kernel = all ? reserve_latent_blocks_kernel<true> : reserve_latent_blocks_kernel<false>;
    if (smem > 40000) {
        // The limit is the kernel's, not the call's: always that of the most sequences, so that a call of another thread does
        // not lower it between here and the launch.
        constexpr int kMost = (3 * kReserveMaxB + 2) * static_cast<int>(sizeof(int));
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
    }
    note_launch();
    const cudaError_t e = launch_dependent(kernel, dim3(1), kReserveThreads, smem, s, p);
    if (e != cudaSuccess || all) return e;
    const unsigned per_seq = (static_cast<unsigned>(a.T) + 4 * kMapThreads - 1) / (4 * kMapThreads);
    const long long blocks = static_cast<long long>(per_seq) * a.B;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    note_launch();
    return launch_dependent(map_slots_kernel, dim3(static_cast<unsigned>(blocks)), kMapThreads, 0, s, p, per_seq);
}

cudaError_t launch_append_latent_paged(const AppendPagedArgs &a, cudaStream_t s) {
    AppendParams p{a.c, static_cast<__nv_bfloat16 *>(a.pool), a.slots, a.ld_c, a.ld_pool, a.pool_rows, 0, a.r / 8, a.dev_err};
    p.pieces = a.rows * p.per_row;
    // four pieces per thread from a wave of the GPU's threads on, one below
    const bool many = p.pieces >= a.num_sms * 2048ll;
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
