// Attention of each sequence's new tokens (one, a chunk or a drafted tree) over the paged latent cache on the sm_103a
// tensor cores: r = 512, d_v = 128, 1 <= H <= 128.
//
// Steps 2-4 of section "完整计算流（四步）" on the page "Gated MLA（矩阵吸收版）", over the cache of latents alone (KV-cache
// table, section "形状与参数对比"): token t's head h scores the visible rows u, a = softmax(scale q_abs . c_u),
// o_lat = sum a_u c_u, out = sigmoid(gate) * W_UV[h] o_lat.  All heads of all tokens of a sequence read the same rows, so
// a sequence's (token, head) pairs, in the order of q_abs, are cut into tiles of M = 128 rows of one product.
//
// Pair kernel (persistent, one cluster of two CTAs per SM pair).  A tile walks the cache in units of 128 rows that any of
// its tokens sees: the first few (sinks), then from the window's start to the last token's own row.  All tiles' units, each
// tile's preceded by the cost of starting it, are cut into equal shares, so that one long sequence and many ragged ones
// keep every SM busy: one share per cluster, or a few rounds of one per cluster where a sequence has several tiles and all
// sequences' rows together do not fit L2: the clusters of a round are at the same sequences, and their tiles read a row
// from DRAM once.
//   rank 0, the score CTA: the tile's q_abs sits in TMEM as packed bf16 (columns 0-255) and is the A operand of
//     S = q_abs . c^T, N = 128 cache rows, into one of two buffers (columns 256-511).  Two warpgroups take the units in
//     turn (thread = row of the tile) and hand each other the running maximum, so that a unit's product runs while the
//     one before is exponentiated; P (bf16) with each row's rescaling factor and sum goes to the value CTA by a bulk copy.
//   rank 1, the value CTA: o_lat += P . c, N = 2 x 256 latent columns, fp32 in all 512 TMEM columns, rescaled lazily when
//     a row's maximum grew by more than 2^16.
// Each CTA loads the rows it needs: boxes of 64 (score) or 32 rows, which lie inside one block of the pool.
//
// Masks are bit sets of 128 rows per row of the tile, used only in units that some of the tile's tokens do not see whole.
// A NaN or an infinity in a row of such a unit would reach the tokens that do not see it, as 0 * NaN.  It shows in the
// row's scores with any query: then the value CTA's math warps replace what is not finite in the unit by zeros before the
// product, and a token that does see it gets its NaN through the sum of its weights.
//
// A part (what a share has of a tile) leaves o_lat / l, and where the tile was cut between shares its maxima and sums of
// weights, at most twice per share.  The values go as f16 with an exponent for each 32 of a row: off by 2^-11, an eighth of
// what rounding the output costs, in half of fp32's bytes, which is what a part's end takes (an SM stores 27 bytes a cycle:
// 256 KB of fp32 took as long as four units).  For few tokens and heads one kernel joins the parts, applies W_UV^T on
// the tensor cores and the gate; otherwise one joins them and a product per head follows.  Both take
// the values to the product as two bf16 parts, off by 2^-16 at most.  So the roundings to 16 bits that count are the softmax
// weights' (2^-8 of each, as in the prefill and the other decodes; two parts would double the value CTA's products), that of
// a part (2^-11, and 2^-11 again where joined rows go through memory) and the output's.  Over 9,000 rows in two parts they
// are 0.0008, 0.0003 and 0.0017 of the outputs' norm.
//
// What bounds it.  A unit's products are 2,048 tensor cycles on either CTA, and both work at once.  8 chunks of 512 tokens of 96
// heads under a window of 4096 take 2.06 to 2.14 ms, 1.5 PFLOP/s: 1,289 units per pair, 1.38 ms of products at 1.92 GHz, 40
// parts of 1.2 to 3 us (drain, refill), and W_UV's kernel, 0.13 ms.  The rest lies between the products, and no one thing is
// known to be it.  In copies of the kernel made for timing, cache rows that are loaded once and used again save 0.15 ms,
// softmaxes that are left out 0.08 ms, both together 0.27 ms.  The counters show the tensor pipe 70 % active, L2's way to the
// SMs 56 %, shared memory's banks 25 % read and 23 % written; the score CTA moves 320 KB per unit through shared memory (rows
// written by TMA and read, P written and copied), the value CTA 350 KB (P read for either latent half).
// With one token of 96 heads per sequence HBM is the bound, 1.5 to 1.7 us per unit of all clusters; 64 of them over 1.08 million
// rows take 216 to 225 us, 4.9 to 5.1 TB/s, and 166 with rows used again.  Besides, a call takes 19 to 31 us before its first unit
// and after its last one: instructions come from L2 or DRAM then, a cold unit's softmax takes twice as long.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "attend_shares.h"
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kR = 512, kDV = 128;
constexpr int kM = 128;         // (token, head) rows of a tile
constexpr int kUnit = 128;      // cache rows of a unit
constexpr int kThreads = 384;   // warps 0 and 3 TMA, 1 MMA, 4-7 and 8-11: two warpgroups
constexpr uint32_t kRegsCtl = 80, kRegsMath = 208, kRegsLaunch = 168;
static_assert(128 * kRegsCtl + 256 * kRegsMath <= kThreads * kRegsLaunch, "register split exceeds the launch");
constexpr float kLog2e = 1.4426950408889634f;
// A stale maximum is kept until the new one exceeds it by this (log2 units): p <= 2^16, far inside fp32's range.
constexpr float kRescaleLog2 = 16.0f;
// Units that starting a tile counts for in the shares: its queries' load, its accumulator's drain, the pipeline's refill.
constexpr int kStart = 2;
// Rounds of shares: as many as bring the rows of a round's sequences down to this, but no more than one for every 6 tiles of a
// sequence, each of them of at least 16 units per cluster.  (16 sequences of 64 drafts of 96 heads over up to 16000 rows, 48
// tiles each: 1164 us in one round, 1087 in four; 64 sequences of 4, 3 tiles each: 210 and 222.)  Both go by sequences of T
// tokens each, all with as many tiles: the rows are taken to be the axis' part for one tile, starts included.  Where counts
// differ they are underestimated, by up to the number of tiles where most sequences have one, and fewer rounds are made than
// would bring the rows down to this: a matter of time alone.
constexpr int kRounds = 4, kRoundTiles = 6, kRoundMin = 16;
constexpr long long kRoundBytes = 96ll << 20;

constexpr uint32_t kSlab = 16384;                  // [128 rows x 64 columns] bf16, 128-byte swizzle
constexpr uint32_t kInfo = kM * 8;                 // {rescaling factor, negative to ask for cleaning, sum} per row of the tile
constexpr uint32_t kPUnit = 2 * kSlab + kInfo;     // P [128 x 128] and its info
constexpr uint32_t kStage = 16384;                 // of either ring
// score CTA: stages of [128 cache rows x 64 latent columns], P staging per warpgroup, running maxima per warpgroup
constexpr int kSStages = 9;
constexpr uint32_t S_PST = kSStages * kStage;
constexpr uint32_t S_MAX = S_PST + 2 * kPUnit;
constexpr uint32_t S_END = S_MAX + 2 * kM * 4;
// value CTA: P buffers, stages of [32 cache rows x 256 latent columns] (four slabs of 64 columns)
constexpr int kPBufs = 3, kVStages = 7, kVRows = 32;
constexpr uint32_t kVSlab = kVRows * 128;
constexpr uint32_t V_RING = kPBufs * kPUnit;
constexpr uint32_t V_END = V_RING + kVStages * kStage;
constexpr uint32_t BARS = (S_END > V_END ? S_END : V_END);
constexpr uint32_t kSmemPair = BARS + 768 + 1024;  // + alignment slack
static_assert(kPUnit % 1024 == 0 && BARS % 16 == 0 && kSmemPair <= 232448, "shared memory");
constexpr uint64_t kLandNs = 50000000;             // a load that was issued lands long before this
constexpr uint32_t S_COL = 256;                    // S buffers in the score CTA's TMEM

constexpr uint32_t kIdescS = make_idesc_bf16(128, 128, 0, 0);   // q_abs (TMEM) x c (K-major)
constexpr uint32_t kIdescO = make_idesc_bf16(128, 256, 0, 1);   // P (K-major) x c (MN-major)

struct PairBars {
    uint64_t q_ready, s_full[2], s_free[2], m_ready[2];
    uint64_t sc_full[kSStages], sc_empty[kSStages];
    uint64_t p_free[kPBufs];                             // arrivals from the value CTA
    uint64_t v_full[kVStages], v_empty[kVStages], v_clean[kVStages];
    uint64_t p_full[kPBufs];                             // the score CTA's copies
    uint64_t pv_done[kPBufs], rescaled, drained;
    uint32_t tmem_base;
    int abort;
    // the axis of units, and where the cluster's shares start on it
    long long total;
    int shares, rounds;
    struct Start {
        long long lo, hi, pre;
        int b, j, len, count;
    } start[kRounds];
    long long warp_sum[kThreads / 32];
};
static_assert(sizeof(PairBars) <= 768, "barrier block too large");

// Division of 0 <= n < 2^31 by a d of the launch: n / d = n * mul >> (31 + s) with 2^(s - 1) < d <= 2^s and mul =
// floor(2^(31 + s) / d) + 1, as n (mul d - 2^(31 + s)) <= n 2^s < 2^(31 + s).  (Each division takes some forty instructions,
// and a part's start is a chain of them.)
struct Divisor {
    unsigned mul, shift;
    Divisor() = default;
    explicit Divisor(int d) {
        unsigned s = 0;
        while ((1ull << s) < static_cast<unsigned long long>(d)) ++s;
        mul = d == 1 ? 0 : static_cast<unsigned>((1ull << (31 + s)) / d + 1);
        shift = d == 1 ? 0 : s - 1;
    }
    __device__ __forceinline__ int operator()(int n) const {
        return mul ? static_cast<int>(__umulhi(static_cast<unsigned>(n), mul) >> shift) : n;
    }
};

struct PairParams {
    const int *table, *lens, *counts, *parents;
    long long ld_table;
    __half *ws_rows;                     // [B * T * H + 2 shares * 128][r]: o_lat / l of (token, head) rows, then of parts' rows
    uint8_t *ws_exp;                     // [.][16]: their exponents
    float *ws_m, *ws_l;                  // [2 shares][128]: parts' maxima (log2 units) and sums of weights
    int2 *ws_tile;                       // [B * tiles]: first and last share of each tile
    int4 *ws_cut;                        // [rounds][G]: first row, rows, first and last share of the tile that a share starts
                                         // and leaves unfinished; {., 0, ., .}: none
    long long all_rows;                  // B * T * H
    int *err;
    int max_rounds;
    int B, T, H, tiles, num_blocks, bs, max_blocks, window, sinks;
    float scale_log2;
    Divisor by_H, by_tiles, by_bs;
};

// New tokens of sequence b and its cached rows; none when its numbers are out of range.
template <typename P>
__device__ __forceinline__ int tokens(const P &p, int b, int &len, bool report) {
    len = __ldg(p.lens + b);
    const int count = p.counts ? __ldg(p.counts + b) : p.T;
    if (len < 0 || count < 0 || count > p.T || static_cast<long long>(len) + count > static_cast<long long>(p.max_blocks) * p.bs) {
        if (report) record_error(p.err, kDevErrBounds);
        return 0;
    }
    return count;
}

// Tile j of a sequence: its tokens, and the units of the cache that any of them sees.
struct Tile {
    int rows, t0, t1;      // (token, head) rows; first and last token
    int head, main, n;     // units from the cache's start on, first unit after those, units in all
    int low, end;          // of the rows behind the sinks [low, end) are seen
    __device__ __forceinline__ Tile() {}
    __device__ __forceinline__ Tile(const PairParams &p, int j, int len, int count) {
        const int m0 = j * kM;
        rows = min(count * p.H - m0, kM);
        t0 = p.by_H(m0), t1 = p.by_H(m0 + rows - 1);
        end = len + t1 + 1;
        main = head = low = 0;
        if (p.window > 0) {   // a draft stands at least at the first new position
            low = max(len + (p.parents ? 0 : t0) - p.window + 1, 0);
            main = low / kUnit;
            head = min((min(p.sinks, end) + kUnit - 1) / kUnit, main);
        }
        n = head + (end + kUnit - 1) / kUnit - main;
    }
    __device__ __forceinline__ int row0(int i) const { return (i < head ? i : main + i - head) * kUnit; }
    // Whether some token of the tile does not see all rows of the unit at u0.
    __device__ __forceinline__ bool mixed(const PairParams &p, int len, int u0) const {
        const bool low = p.window > 0 && u0 < len + t1 - p.window + 1 && u0 + kUnit > p.sinks;
        return low || u0 + kUnit > (p.parents ? len : len + t0 + 1);
    }
};

// Every role of both CTAs walks the cluster's shares, tile by tile.
struct Walk {
    long long lo, hi, pre;   // pre: the axis position of tile j of sequence b
    int b, j, len, count;
    int round, share;        // of the current part
    int seq, i0, i1;         // its sequence and units [i0, i1) of the tile
    int index;               // the tile's number in the sequence
    Tile t;
    __device__ __forceinline__ explicit Walk(const PairBars *s) : round(0) { enter(s); }
    __device__ __forceinline__ void enter(const PairBars *s) {
        const auto &x = s->start[round];
        lo = x.lo, hi = x.hi, pre = x.pre, b = x.b, j = x.j, len = x.len, count = x.count;
    }
    __device__ __forceinline__ bool next(const PairParams &p, const PairBars *s, int cl) {
        for (;;) {
            if (pre >= hi || b >= p.B) {
                if (round + 1 >= s->rounds) return false;
                ++round;
                enter(s);
                continue;
            }
            if (static_cast<long long>(j) * kM >= static_cast<long long>(count) * p.H) {
                j = 0;
                if (++b < p.B) count = tokens(p, b, len, false);
                continue;
            }
            t = Tile(p, j, len, count);
            const long long base = pre + kStart;
            const long long s0 = max(base, lo), s1 = min(base + t.n, hi);
            seq = b, index = j;
            pre = base + t.n;
            ++j;
            if (s1 > s0) {
                i0 = static_cast<int>(s0 - base), i1 = static_cast<int>(s1 - base);
                share = round * s->shares + cl;
                return true;
            }
        }
    }
    __device__ __forceinline__ int seq_len(const PairParams &p) const { return __ldg(p.lens + seq); }
    __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == t.n; }
    __device__ __forceinline__ int slot() const { return static_cast<int>(part_number(share, i0 == 0)); }
};

// The cache rows that a token sees: [0, head), [lo, hi), and of the 64 from `hi` on those whose bit is set.
struct Sight {
    int head, lo, hi;
    unsigned long long bits;
    __device__ __forceinline__ Sight() {}
    // Of token t; a whole warp calls it.  Drafts: lane i holds what is known of drafts i and i + 32, the set of their next
    // 2^k ancestors and the one after those, and doubles it.
    __device__ __forceinline__ Sight(const PairParams &p, int b, int t, int len, int count, int lane) {
        bits = 0;
        int position = len + t;
        hi = position + 1;
        if (p.parents) {
            const int *const up = p.parents + static_cast<long long>(b) * p.T;
            unsigned long long set[2];
            int next[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int a = lane + 32 * i, q = a < count ? __ldg(up + a) : -1;
                const bool good = q >= -1 && q < a;
                if (a < count && !good) record_error(p.err, kDevErrBounds);
                next[i] = good ? q : -1;   // below a, so that every line ends
                set[i] = 1ull << a;
            }
            for (int k = 0; k < 6; ++k) {
                unsigned long long more[2];
                int far[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = next[i] & 31;
                    const unsigned long long s0 = __shfl_sync(0xffffffffu, set[0], at), s1 = __shfl_sync(0xffffffffu, set[1], at);
                    const int n0 = __shfl_sync(0xffffffffu, next[0], at), n1 = __shfl_sync(0xffffffffu, next[1], at);
                    more[i] = next[i] < 0 ? 0 : next[i] < 32 ? s0 : s1;
                    far[i] = next[i] < 0 ? -1 : next[i] < 32 ? n0 : n1;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) set[i] |= more[i], next[i] = far[i];
            }
            const unsigned long long s0 = __shfl_sync(0xffffffffu, set[0], t & 31), s1 = __shfl_sync(0xffffffffu, set[1], t & 31);
            bits = t < 32 ? s0 : s1;
            const int depth = __popcll(bits) - 1;
            hi = len, position = len + depth;
            if (p.window > 0) {
                // ancestors come in the order of their depths: those before the window and past the sinks go
                unsigned long long rest = bits, sinks = 0;
                for (int d = 0; d <= depth - p.window; ++d) {
                    const unsigned long long first = rest & (0 - rest);
                    rest ^= first;
                    if (len + d < p.sinks) sinks |= first;
                }
                bits = rest | sinks;
            }
        }
        lo = p.window > 0 ? max(position - p.window + 1, 0) : 0;
        head = min(min(p.sinks, lo), hi);
    }
    // Rows u0 + 32 w .. + 31 as bits.
    __device__ __forceinline__ uint32_t word(int u0, int w) const {
        const int at = u0 + 32 * w;
        const auto below = [&](int x) { return x <= at ? 0u : x - at >= 32 ? ~0u : (1u << (x - at)) - 1; };
        uint32_t m = below(head) | (below(hi) & ~below(lo));
        const int off = at - hi;
        if (off >= 0) {
            if (off < 64) m |= static_cast<uint32_t>(bits >> off);
        } else if (off > -32) {
            m |= static_cast<uint32_t>(bits << -off);
        }
        return m;
    }
};

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_shared_v2f(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_v2f(uint32_t addr, float a, float b) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// Rows of o_lat: [r] f16, and 16 bytes: the biased exponent E of each 32 values' largest.  A value is f16 * 2^(E - 141), so
// that the largest is below 2^15 and what is 2^28 times smaller keeps its 11 bits.
__device__ __forceinline__ int row_exponent(float largest) {
    return max(static_cast<int>(__float_as_uint(largest) >> 23) & 0xFF, 20);   // below 2^-107: as if it were that
}
__device__ __forceinline__ float row_up(int E) { return __uint_as_float(static_cast<uint32_t>(268 - E) << 23); }     // 2^(141 - E)
__device__ __forceinline__ float row_down(int E) { return __uint_as_float(static_cast<uint32_t>(E - 14) << 23); }   // 2^(E - 141)
__device__ __forceinline__ float2 row_values(uint32_t w, float down) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(v.x * down, v.y * down);
}

// Two values as bf16 and what the rounding leaves, as bf16 again.
__device__ __forceinline__ uint32_t split_bf16x2(float a, float b, uint32_t &lo) {
    const uint32_t hi = pack_bf16x2(a, b);
    lo = pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
    return hi;
}

// Not finite bf16 halves of a word to zero.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
    return w;
}

// A place in a ring of barriers and stages.
template <int N>
struct Ring {
    uint32_t st = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++st == N) st = 0, phase ^= 1;
    }
};

// What kernels before this one wrote becomes visible to this thread's TMA loads.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// True in one lane of a warp that is here together.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attend_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_s,
                       const __grid_constant__ CUtensorMap tm_v, const PairParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    PairBars *const bars = reinterpret_cast<PairBars *>(smem_raw + (base - raw) + BARS);
    volatile int *const abort_flag = &bars->abort;
    const auto B_ = [](uint64_t &b) { return smem_u32(&b); };
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // known to be one per warp
    const uint32_t rank = cluster_ctarank();
    const int G = static_cast<int>(gridDim.x >> 1), cl = static_cast<int>(blockIdx.x >> 1);

    if (threadIdx.x == 0) {
        mbar_init(B_(bars->q_ready), 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(B_(bars->s_full[i]), 1);
            mbar_init(B_(bars->s_free[i]), 128);
            mbar_init(B_(bars->m_ready[i]), 128);
        }
        for (int i = 0; i < kSStages; ++i) {
            mbar_init(B_(bars->sc_full[i]), 2);
            mbar_init(B_(bars->sc_empty[i]), 1);
        }
        for (int i = 0; i < kPBufs; ++i) {
            mbar_init(B_(bars->p_free[i]), 1);
            mbar_init(B_(bars->p_full[i]), 1);
            mbar_init(B_(bars->pv_done[i]), 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(B_(bars->v_full[i]), 1);
            mbar_init(B_(bars->v_empty[i]), 1);
            mbar_init(B_(bars->v_clean[i]), 256);
        }
        mbar_init(B_(bars->rescaled), 256);
        mbar_init(B_(bars->drained), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == 0 || warp == 3) {   // the producers
        tma_prefetch_desc(rank == 0 ? &tm_s : &tm_v);
        if (rank == 0) tma_prefetch_desc(&tm_q);
    }
    tc_fence_before();
    cluster_sync_all();   // both CTAs' barriers exist before any remote arrival or copy
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    grid_dependency_wait();
    if (warp == 0 || warp == 3) fence_proxy_async_all();
    grid_launch_dependents();   // the second kernel may take SMs as clusters finish; it waits for the whole grid

    // The axis: thread i adds up its part of the tiles; the one that holds the share's start finds the tile there.
    {
        const int all = p.B * p.tiles, per = (all + kThreads - 1) / kThreads;
        const int g0 = min(static_cast<int>(threadIdx.x) * per, all), g1 = min(g0 + per, all);
        int len = 0, count = 0;
        const auto units = [&](int g, bool report) {
            const int b = p.by_tiles(g), j = g - b * p.tiles;
            count = tokens(p, b, len, report);
            return static_cast<long long>(j) * kM < static_cast<long long>(count) * p.H
                       ? kStart + Tile(p, j, len, count).n : 0;
        };
        long long sum = 0;
        for (int g = g0; g < g1; ++g) sum += units(g, cl == 0 && rank == 0);
        long long incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) bars->warp_sum[warp] = incl;
        __syncthreads();
        long long pre = incl - sum, total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const long long v = bars->warp_sum[w];
            if (w < warp) pre += v;
            total += v;
        }
        // No share is empty but those of the clusters that are too many: a tile's parts lie in successive shares.
        const int n = total < G ? static_cast<int>(total) : G;
        int rounds = 1;
        if (p.max_rounds > 1) {
            const long long bytes = total * (kUnit * kR * 2) / p.tiles, units = total / (max(n, 1) * kRoundMin);
            rounds = max(1, static_cast<int>(min(min((bytes + kRoundBytes - 1) / kRoundBytes, units),
                                                 static_cast<long long>(p.max_rounds))));
        }
        const int shares = n * rounds;
        const auto start = [&](int c) {   // 64-bit divisions take a few hundred cycles
            return total < (1 << 22) ? static_cast<long long>(static_cast<unsigned>(total) * static_cast<unsigned>(c) /
                                                              static_cast<unsigned>(shares))
                                     : total * c / shares;
        };
        if (threadIdx.x == 0) bars->total = total, bars->shares = n, bars->rounds = cl < n ? rounds : 0;
        if (cl >= n && threadIdx.x == 0) bars->start[0] = {0, 0, 0, p.B, 0, 0, 0};
        for (int r = 0; cl < n && r < rounds; ++r) {
            const long long lo = start(r * n + cl), hi = start(r * n + cl + 1);
            if (pre > lo || lo >= pre + sum) continue;
            long long at = pre;
            for (int g = g0; g < g1; ++g) {
                const long long k = per == 1 ? sum : units(g, false);
                if (lo < at + k) {
                    const int b = p.by_tiles(g);
                    bars->start[r] = {lo, hi, at, b, g - b * p.tiles, len, count};
                    break;
                }
                at += k;
            }
        }
        __syncthreads();
    }

    // The pool row of cache row u (u % 64 == 0) of a sequence, or one past the pool, which reads as zeros.  Entries of blocks
    // of which no row is seen are not read and may hold anything.
    const auto pool_row = [&](int seq, int u, const Tile &t) {
        const int none = max(p.num_blocks * p.bs, 1);
        if (u >= t.end || (u + 64 <= t.low && u >= p.sinks)) return none;
        const int j = p.by_bs(u), block = __ldg(p.table + seq * p.ld_table + j);
        if (block < 0 || block >= p.num_blocks) {
            record_error(p.err, kDevErrBounds);
            return none;
        }
        return block * p.bs + (u - j * p.bs);
    };

    if (warp < 4) {
        regs_release<kRegsCtl>();
        Walk w(bars);
        const bool lead = elect_one();
        // a whole warp leaves a wait together and of one mind
        const auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.err, abort_flag));
        };
        if (rank == 0) {
            // =========================================================== score CTA
            if (warp == 0 || warp == 3) {
                // ---- TMA producers: rows [64 half, 64 half + 64) of each stage; a part's queries, then its units
                const int half = warp == 0 ? 0 : 1;
                const uint32_t full0 = B_(bars->sc_full[0]), empty0 = B_(bars->sc_empty[0]);
                Ring<kSStages> at;
                uint32_t it = 0;
                bool ok = true;
                while (ok && w.next(p, bars, cl)) {
                    for (int i = w.i0 - 1; ok && i < w.i1; ++i) {
                        const bool units = i >= w.i0;
                        const int u = units ? w.t.row0(i) + half * 64 : 0;
                        // rows past the tile's, of the next one or past the tensor's end (zeros), are not used
                        const int row = units ? pool_row(w.seq, u, w.t) : w.seq * p.T * p.H + w.index * kM + half * 64;
#pragma unroll 1
                        for (int kc = 0; kc < 8; ++kc, ++it, at.next()) {
                            // a barrier that no one has arrived at counts as past phase 1
                            if (!(ok = wait(empty0 + at.st * 8, at.phase ^ 1))) break;
                            if (!lead) continue;
                            const uint32_t full = full0 + at.st * 8;
                            mbar_arrive_expect_tx(full, kStage / 2);
                            tma_load_2d(base + at.st * kStage + half * (kStage / 2), units ? &tm_s : &tm_q, full, kc * 64,
                                        row);
                        }
                    }
                }
                if (!ok) *abort_flag = 1;
                // no load may still be landing when the CTA exits
                for (uint32_t k = it > kSStages ? it - kSStages : 0; k < it; ++k)
                    mbar_wait(B_(bars->sc_full[k % kSStages]), (k / kSStages) & 1, p.err, nullptr, kLandNs);
            } else if (warp == 1) {
                // ---- MMA issuer
                const uint64_t ring = make_smem_desc(base, 16, 1024);
                const uint32_t full0 = B_(bars->sc_full[0]), empty0 = B_(bars->sc_empty[0]), s_full0 = B_(bars->s_full[0]),
                               s_free0 = B_(bars->s_free[0]), q_ready = B_(bars->q_ready);
                Ring<kSStages> at;
                Ring<2> sb;
                uint32_t q_phase = 0;
                bool ok = true;
                while (ok && w.next(p, bars, cl)) {
                    for (int k = 0; k < 8; ++k) at.next();   // the queries' stages
                    if (!(ok = wait(q_ready, q_phase))) break;
                    q_phase ^= 1;
#pragma unroll 1
                    for (int i = w.i0; ok && i < w.i1; ++i, sb.next()) {
                        if (!(ok = wait(s_free0 + sb.st * 8, sb.phase ^ 1))) break;
                        const uint32_t d = tmem + S_COL + sb.st * 128;
#pragma unroll 1
                        for (int kc = 0; kc < 8; ++kc, at.next()) {
                            if (!(ok = wait(full0 + at.st * 8, at.phase))) break;
                            tc_fence_after();
                            if (lead) {
                                const uint64_t b = desc_add(ring, at.st * kStage);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    umma_bf16_tmem_a(d, tmem + kc * 32 + kk * 8, desc_add(b, kk * 32), kIdescS, (kc | kk) != 0);
                                umma_commit(empty0 + at.st * 8);
                            }
                        }
                        if (ok && lead) umma_commit(s_full0 + sb.st * 8);
                    }
                }
                if (!ok) *abort_flag = 1;
            }
        } else {
            // =========================================================== value CTA
            if (warp == 0 || warp == 3) {
                // ---- TMA producers: a unit is 8 stages, latent half i >> 2, row quarter i & 3; each takes one half of
                // the rows
                const int half = warp == 0 ? 0 : 1;
                const uint32_t full0 = B_(bars->v_full[0]), empty0 = B_(bars->v_empty[0]);
                Ring<kVStages> at;
                uint32_t it = 0;
                bool ok = true;
                while (ok && w.next(p, bars, cl)) {
                    for (int i = w.i0; ok && i < w.i1; ++i, it += 8) {
                        const int u = w.t.row0(i) + half * 64;
                        const int row = pool_row(w.seq, u, w.t);
#pragma unroll 1
                        for (int k = 0; ok && k < 8; ++k, at.next()) {
                            if (((k >> 1) & 1) != half) continue;
                            if (!(ok = wait(empty0 + at.st * 8, at.phase ^ 1))) break;
                            if (!lead) continue;
                            const uint32_t full = full0 + at.st * 8;
                            mbar_arrive_expect_tx(full, kStage);
                            tma_load_3d(base + V_RING + at.st * kStage, &tm_v, full, 0, row + (k & 1) * kVRows, (k >> 2) * 4);
                        }
                    }
                }
                if (!ok) *abort_flag = 1;
                for (uint32_t k = it > kVStages ? it - kVStages : 0; k < it; ++k)
                    mbar_wait(B_(bars->v_full[k % kVStages]), (k / kVStages) & 1, p.err, nullptr, kLandNs);
            } else if (warp == 1) {
                // ---- MMA issuer
                const uint64_t pdesc = make_smem_desc(base, 16, 1024), ring = make_smem_desc(base + V_RING, kVSlab, 1024);
                const uint32_t full0 = B_(bars->v_full[0]), empty0 = B_(bars->v_empty[0]), clean0 = B_(bars->v_clean[0]),
                               p_full0 = B_(bars->p_full[0]), pv_done0 = B_(bars->pv_done[0]);
                Ring<kVStages> at;
                Ring<kPBufs> pb;
                uint32_t fix_phase = 0, drain_phase = 1, cleaned = 0;   // cleaned: a phase bit per stage
                bool ok = true;
                while (ok && w.next(p, bars, cl)) {
                    const uint32_t bytes = 2u * ((w.t.rows + 7) & ~7) * 128u + kInfo;
#pragma unroll 1
                    for (int i = w.i0; ok && i < w.i1; ++i, pb.next()) {
                        const bool first = i == w.i0;
                        const uint32_t p_full = p_full0 + pb.st * 8;
                        if (lead) mbar_arrive_expect_tx(p_full, bytes);
                        if (!(ok = __all_sync(0xffffffffu, mbar_wait<true>(p_full, pb.phase, p.err, abort_flag)))) break;
                        const uint32_t info = base + pb.st * kPUnit + 2 * kSlab;
                        bool grew = false, dirty = false;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float f = ld_shared_f32(info + (lane + 32 * k) * 8);
                            grew |= fabsf(f) != 1.f, dirty |= signbit(f);
                        }
                        dirty = __any_sync(0xffffffffu, dirty);
                        if (first) {   // the accumulator of the part before has been drained
                            if (!(ok = wait(B_(bars->drained), drain_phase))) break;
                            drain_phase ^= 1;
                        } else if (__any_sync(0xffffffffu, grew)) {
                            // rows whose maximum grew need their accumulator rescaled before this unit's product
                            if (!(ok = wait(B_(bars->rescaled), fix_phase))) break;
                            fix_phase ^= 1;
                        }
                        uint64_t a = desc_add(pdesc, pb.st * kPUnit);
#pragma unroll 1
                        for (int k = 0; k < 8; ++k, at.next()) {   // latent half k >> 2, row quarter k & 3
                            if (!(ok = wait(full0 + at.st * 8, at.phase))) break;
                            if (dirty) {
                                if (!(ok = wait(clean0 + at.st * 8, (cleaned >> at.st) & 1))) break;
                                cleaned ^= 1u << at.st;
                            }
                            tc_fence_after();
                            if (lead) {
                                const uint64_t b = desc_add(ring, at.st * kStage);
                                const uint64_t ak = desc_add(a, ((k >> 1) & 1) * kSlab + (k & 1) * 64);
                                const uint32_t d = tmem + (k >> 2) * 256;
                                umma_bf16(d, ak, b, kIdescO, !first || (k & 3) != 0);
                                umma_bf16(d, desc_add(ak, 32), desc_add(b, 2048), kIdescO, 1);
                                umma_commit(empty0 + at.st * 8);
                            }
                        }
                        if (ok && lead) umma_commit(pv_done0 + pb.st * 8);
                    }
                }
                if (!ok && lead) *abort_flag = 1;
            }
        }
    } else {
        regs_acquire<kRegsMath>();
        Walk w(bars);
        const int wg = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;   // row of the tile, TMEM lane
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const bool first_thread = (threadIdx.x & 127) == 0;
        if (rank == 0) {
            // ---- softmax: warpgroup wg takes every other unit
            const uint32_t ptile = base + S_PST + wg * kPUnit, info = ptile + 2 * kSlab;
            uint32_t jb = 0, it = 0;   // units; places in the ring
            bool ok = true;
            // A failed wait is voted on at the next barrier of the warpgroup, which no warp leaves alone.
            bool fail = false;
            const auto wait_warp = [&](uint64_t &bar, uint32_t parity) {
                return __any_sync(0xffffffffu, fail || !mbar_wait(B_(bar), parity, p.err, abort_flag));
            };
            // A part's queries into TMEM: a row's packed bf16 pairs are its 32-bit words in memory order.  Warpgroup wg
            // moves latent columns [256 wg, 256 wg + 256), four stages of 64.
            const auto load_q = [&](bool active) {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    const uint32_t at = it + wg * 4 + k, st = at % kSStages;
                    fail = wait_warp(bars->sc_full[st], (at / kSStages) & 1);
                    if (active) {
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint4 x = ld_shared_v4(base + st * kStage + sw128_offset(row, i));
                            v[4 * i] = __uint_as_float(x.x), v[4 * i + 1] = __uint_as_float(x.y);
                            v[4 * i + 2] = __uint_as_float(x.z), v[4 * i + 3] = __uint_as_float(x.w);
                        }
                        tmem_st32(trow + (wg * 4 + k) * 32, v);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(B_(bars->q_ready));
                fence_proxy_async_smem();   // TMA writes to these stages again
                named_bar_sync(2 + wg, 128);
                if (first_thread)
                    for (int k = 0; k < 4; ++k) mbar_arrive(B_(bars->sc_empty[(it + wg * 4 + k) % kSStages]));
            };
            const auto has_rows = [&](const Walk &v) { return (warp & 3) * 32 < v.t.rows; };
            bool more = w.next(p, bars, cl);
            if (more) load_q(has_rows(w));
            while (ok && more) {
                const int len = w.seq_len(p);
                const Sight sight(p, w.seq, min(p.by_H(w.index * kM + row), w.t.t1), len, w.count, lane);
                const int i0 = w.i0, i1 = w.i1, slot = w.slot(), rows = w.t.rows;
                const Tile tile = w.t;
                const bool whole = w.whole(), active = has_rows(w);
                it += 8 * (1 + i1 - i0);   // where the next part's queries are
                more = w.next(p, bars, cl);          // they go into TMEM after this one's last product
                float m_mine = -INFINITY, l = 0.f;
                for (int i = i0; ok && i < i1; ++i, ++jb) {
                    const bool mine = (jb & 1) == static_cast<uint32_t>(wg), last = i == i1 - 1;
                    if (!mine && !(last && more)) continue;
                    fail = wait_warp(bars->s_full[jb & 1], (jb >> 1) & 1);
                    tc_fence_after();
                    if (mine && !active) {   // none of the tile's rows are this warp's
                        mbar_arrive(B_(bars->s_free[jb & 1]));
                        mbar_arrive(B_(bars->m_ready[wg]));
                        if (first_thread) bulk_wait_read_all();
                        if (named_bar_or(2 + wg, 128, fail)) { ok = false; break; }
                        st_shared_v2f(info + row * 8, 1.f, 0.f);
                        fence_proxy_async_smem();
                        named_bar_sync(2 + wg, 128);
                    } else if (mine) {
                        // Two passes over S, 32 columns at a time in rolled loops, the first one another in a mixed unit, where
                        // it masks S too: short code is faster, in a long call (all roles' loops share the instruction caches:
                        // 8 chunks of 512 under a window take 2.27 ms with the two loops unrolled, 2.16 so) and at a call's
                        // start, when it comes from L2 or DRAM.  The scale multiplies inside the exponent: the largest of
                        // c s is c max(s) for c >= 0, c min(s) otherwise.  A masked unit's scores are multiplied first.
                        const int u0 = tile.row0(i);
                        const uint32_t scol = trow + S_COL + (jb & 1) * 128;
                        float mul = p.scale_log2, mx = -INFINITY;
                        bool dirty = false;
                        if (tile.mixed(p, len, u0)) {
                            mul = 1.f;
                            float zeros[4] = {0.f, 0.f, 0.f, 0.f};   // NaN once a score is not finite
                            float top[4] = {mx, mx, mx, mx};
#pragma unroll 1
                            for (int c4 = 0; c4 < 4; ++c4) {
                                float s[32];
                                tmem_ld32(scol + c4 * 32, s);
                                tmem_wait_ld();
                                const uint32_t seen = sight.word(u0, c4);
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    // an infinite score's row gives NaN, as its product with the weight 0 would
                                    const float zero = s[k] - s[k];
                                    zeros[k & 3] += zero;
                                    s[k] = (seen >> k) & 1 ? fmaf(s[k], p.scale_log2, zero) : -INFINITY;
                                    top[k & 3] = fmaxf(top[k & 3], s[k]);
                                }
                                tmem_st32(scol + c4 * 32, s);
                            }
                            mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                            tmem_wait_st();
                            dirty = (zeros[0] + zeros[1]) + (zeros[2] + zeros[3]) != 0.f && row < rows;
                        } else {
                            float mn = INFINITY;
#pragma unroll 1
                            for (int c4 = 0; c4 < 4; ++c4) {
                                float s[32];
                                tmem_ld32(scol + c4 * 32, s);
                                tmem_wait_ld();
                                if (mul >= 0.f) {
                                    float t[4] = {mx, s[0], s[1], s[2]};
#pragma unroll
                                    for (int k = 3; k < 32; ++k) t[k & 3] = fmaxf(t[k & 3], s[k]);
                                    mx = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                                } else {
#pragma unroll
                                    for (int k = 0; k < 32; ++k) mn = fminf(mn, s[k]);
                                }
                            }
                            mx = mul * (mul >= 0.f ? mx : mn);
                        }
                        // the running maximum of the unit before, from the other warpgroup
                        if (jb > 0) fail = wait_warp(bars->m_ready[wg ^ 1], ((jb - 1) >> 1) & 1);
                        const float m_old = i == i0 ? -INFINITY : ld_shared_f32(base + S_MAX + (wg ^ 1) * kM * 4 + row * 4);
                        float m = m_old, factor = 1.f;
                        if (mx > m_old + kRescaleLog2) {
                            factor = fast_exp2(m_old - mx);
                            m = mx;
                        }
                        st_shared_f32(base + S_MAX + wg * kM * 4 + row * 4, m);
                        mbar_arrive(B_(bars->m_ready[wg]));
                        const float neg_m = m == -INFINITY ? 0.f : -m;
                        if (m != m_mine) l *= fast_exp2(m_mine - m);
                        m_mine = m;
                        if (last && !whole && row < rows) p.ws_m[static_cast<size_t>(slot) * kM + row] = m;

                        // the staging unit is free once this warpgroup's copy before has read it
                        if (first_thread) bulk_wait_read_all();
                        if (named_bar_or(2 + wg, 128, fail)) { ok = false; break; }
#pragma unroll 1
                        for (int c4 = 0; c4 < 4; ++c4) {
                            float s[32];
                            tmem_ld32(scol + c4 * 32, s);
                            tmem_wait_ld();
                            float t[4] = {l, 0.f, 0.f, 0.f};
                            const uint32_t slab = ptile + (c4 >> 1) * kSlab;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float *v = &s[8 * k];
#pragma unroll
                                for (int q = 0; q < 8; ++q) {
                                    v[q] = fast_exp2(fmaf(v[q], mul, neg_m));
                                    t[q & 3] += v[q];
                                }
                                st_shared_v4(slab + sw128_offset(row, (c4 & 1) * 4 + k), pack_bf16x2(v[0], v[1]),
                                             pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                            }
                            l = (t[0] + t[1]) + (t[2] + t[3]);
                        }
                        tc_fence_before();
                        mbar_arrive(B_(bars->s_free[jb & 1]));
                        st_shared_v2f(info + row * 8, dirty ? -factor : factor, l);
                        fence_proxy_async_smem();
                        named_bar_sync(2 + wg, 128);
                        if (first_thread) {
                            const uint32_t pb = jb % kPBufs;
                            if (jb >= kPBufs)
                                fail = !mbar_wait<true>(B_(bars->p_free[pb]), (jb / kPBufs - 1) & 1, p.err, abort_flag);
                            if (!fail) {
                                const uint32_t bar = mapa_shared(B_(bars->p_full[pb]), 1);
                                const uint32_t dst = mapa_shared(base + pb * kPUnit, 1);
                                if (rows == kM) {
                                    bulk_copy_s2cluster(dst, ptile, kPUnit, bar);
                                } else {   // whole groups of 8 rows: the others' products are not read
                                    const uint32_t n = static_cast<uint32_t>((rows + 7) & ~7) * 128;
                                    bulk_copy_s2cluster(dst, ptile, n, bar);
                                    bulk_copy_s2cluster(dst + kSlab, ptile + kSlab, n, bar);
                                    bulk_copy_s2cluster(dst + 2 * kSlab, info, kInfo, bar);
                                }
                                bulk_commit_group();
                            }
                        }
                    }
                    __syncwarp();
                    if (last && more) load_q(has_rows(w));
                }
            }
            if (first_thread) bulk_wait_all();
            if (!ok || fail) *abort_flag = 1;
        } else {
            // ---- rescaling, cleaning and drain: thread = TMEM lane, warpgroup wg has latent columns [256 wg, 256 wg + 256)
            uint32_t jj = 0, it = 0;
            uint32_t uncut = (1u << kRounds) - 1;   // rounds whose share leaves no tile unfinished
            bool ok = true, fail = false;
            while (ok && w.next(p, bars, cl)) {
                float l_old = 0.f, l_new = 0.f;   // the sums of the two warpgroups of the score CTA
                for (int i = w.i0; i < w.i1; ++i, ++jj, it += 8) {
                    const uint32_t pb = jj % kPBufs;
                    fail = !mbar_wait<true>(B_(bars->p_full[pb]), (jj / kPBufs) & 1, p.err, abort_flag) || fail;
                    if (named_bar_or(4, 256, fail)) { ok = false; break; }
                    float2 fl = ld_shared_v2f(base + pb * kPUnit + 2 * kSlab + row * 8);
                    const bool dirty = signbit(fl.x);
                    fl.x = fabsf(fl.x);
                    l_old = i == w.i0 ? 0.f : l_new * fl.x;
                    l_new = fl.y;
                    const bool grew = i > w.i0 && fl.x != 1.f;
                    const bool any_dirty = named_bar_or(4, 256, dirty), any_grew = named_bar_or(5, 256, grew);
                    const uint32_t prev = jj - 1;
                    if (any_grew) {
                        fail = !mbar_wait(B_(bars->pv_done[prev % kPBufs]), (prev / kPBufs) & 1, p.err, abort_flag);
                        if (named_bar_or(4, 256, fail)) { ok = false; break; }
                        tc_fence_after();
                        if (__any_sync(0xffffffffu, fl.x != 1.f)) {
#pragma unroll 1
                            for (int cc = 0; cc < 8; ++cc) {
                                float v[32];
                                const uint32_t ta = trow + wg * 256 + cc * 32;
                                tmem_ld32(ta, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) v[k] *= fl.x;
                                tmem_st32(ta, v);
                            }
                            tmem_wait_st();
                        }
                        tc_fence_before();
                        mbar_arrive(B_(bars->rescaled));
                    }
                    if (any_dirty) {
                        // the ring has come to this unit once the product of the one before is done
                        fail = i > w.i0 && !mbar_wait(B_(bars->pv_done[prev % kPBufs]), (prev / kPBufs) & 1, p.err, abort_flag);
                        for (int k = 0; !fail && k < 8; ++k) {
                            const uint32_t s = it + k, st = s % kVStages;
                            fail = !mbar_wait(B_(bars->v_full[st]), (s / kVStages) & 1, p.err, abort_flag);
                            if (fail) break;
                            const uint32_t at = base + V_RING + st * kStage + (threadIdx.x - 128) * 16;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint4 v = ld_shared_v4(at + q * 4096);
                                const uint4 c = make_uint4(finite_halves(v.x), finite_halves(v.y), finite_halves(v.z),
                                                           finite_halves(v.w));
                                if (c.x != v.x || c.y != v.y || c.z != v.z || c.w != v.w)
                                    st_shared_v4(at + q * 4096, c.x, c.y, c.z, c.w);
                            }
                            fence_proxy_async_smem();
                            mbar_arrive(B_(bars->v_clean[st]));
                        }
                        if (named_bar_or(4, 256, fail)) { ok = false; break; }
                    }
                    // All have read the info of the unit before: its P buffer is free once its product is done.  (A part's
                    // last one is freed by the drain.)
                    if (threadIdx.x == 128 && i > w.i0) {
                        fail = !mbar_wait(B_(bars->pv_done[prev % kPBufs]), (prev / kPBufs) & 1, p.err, abort_flag);
                        if (!fail) mbar_arrive_remote(B_(bars->p_free[prev % kPBufs]), 0);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                // the part's end
                const uint32_t prev = jj - 1;
                fail = !mbar_wait(B_(bars->pv_done[prev % kPBufs]), (prev / kPBufs) & 1, p.err, abort_flag) || fail;
                if (named_bar_or(4, 256, fail)) { ok = false; break; }
                tc_fence_after();
                const bool whole = w.whole();
                const float sum = l_old + l_new, inv = 1.f / sum;
                const int quad = (warp & 3) * 32, rows = min(w.t.rows - quad, 32);   // of the tile's, this warp's
                const long long part = static_cast<long long>(w.slot()) * kM + quad;
                const long long r0 = whole ? static_cast<long long>(w.seq) * p.T * p.H + static_cast<long long>(w.index) * kM + quad
                                           : p.all_rows + part;
                if (rows > 0) {
                    // A lane has a row; a warp's 4 KB of the buffer turn 64 columns of 32 rows, so that stores fill whole
                    // lines
                    const uint32_t turn = base + (prev % kPBufs) * kPUnit + (warp - 4) * 4096;
                    const int piece = lane & 7;   // 16 bytes of a row; four rows at a time
                    uint4 *dst = reinterpret_cast<uint4 *>(p.ws_rows + (r0 + (lane >> 3)) * kR + wg * 256) + piece;
                    uint32_t exps[2] = {0, 0};
#pragma unroll 1
                    for (int cc = 0; cc < 4; ++cc, dst += 8) {
                        float v[2][32];
                        tmem_ld32(trow + wg * 256 + cc * 64, v[0]);
                        tmem_ld32(trow + wg * 256 + cc * 64 + 32, v[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            float top = 0.f;
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[g][k] *= inv, top = fmaxf(top, fabsf(v[g][k]));
                            const int E = row_exponent(top);
                            const float up = row_up(E);
                            exps[1] = __funnelshift_r(exps[1], static_cast<uint32_t>(E), 8);   // bytes enter at the top
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                st_shared_v4(turn + lane * 128 + (((g * 4 + k) ^ (lane & 7)) << 4),
                                             pack_f16x2(v[g][8 * k] * up, v[g][8 * k + 1] * up),
                                             pack_f16x2(v[g][8 * k + 2] * up, v[g][8 * k + 3] * up),
                                             pack_f16x2(v[g][8 * k + 4] * up, v[g][8 * k + 5] * up),
                                             pack_f16x2(v[g][8 * k + 6] * up, v[g][8 * k + 7] * up));
                        }
                        if (cc == 1) exps[0] = exps[1];
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = k * 4 + (lane >> 3);
                            if (r < rows) dst[k * 4 * (kR / 8)] = ld_shared_v4(turn + r * 128 + ((piece ^ (r & 7)) << 4));
                        }
                        __syncwarp();
                    }
                    if (lane < rows) {
                        *reinterpret_cast<uint2 *>(p.ws_exp + (r0 + lane) * 16 + wg * 8) = make_uint2(exps[0], exps[1]);
                        if (wg == 0 && !whole) p.ws_l[part + lane] = sum;
                    }
                }
                if (threadIdx.x == 128) {
                    int2 *const tile = p.ws_tile + static_cast<long long>(w.seq) * p.tiles + w.index;
                    if (w.i0 == 0) tile->x = w.share;
                    if (w.i1 == w.t.n) tile->y = w.share;
                    if (w.i0 == 0 && w.i1 < w.t.n) {   // the share that holds the tile's last unit: start(c) < w.pre
                        const int last = static_cast<int>((w.pre * (bars->shares * bars->rounds) - 1) / bars->total);
                        p.ws_cut[w.round * G + cl] = make_int4(w.seq * p.T * p.H + w.index * kM, w.t.rows, w.share, last);
                        uncut &= ~(1u << w.round);
                    }
                }
                fence_proxy_async_smem();   // the next P's copy follows
                tc_fence_before();
                named_bar_sync(4, 256);
                if (threadIdx.x == 128) {
                    mbar_arrive(B_(bars->drained));
                    mbar_arrive_remote(B_(bars->p_free[prev % kPBufs]), 0);
                }
            }
            for (int r = 0; threadIdx.x == 128 && r < p.max_rounds; ++r)
                if ((uncut >> r) & 1) p.ws_cut[r * G + cl] = make_int4(0, 0, 0, 0);
            if (!ok) *abort_flag = 1;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
    cluster_sync_all();   // the partner no longer touches this CTA's shared memory or barriers
}

// ----------------------------------------------------------------------------- join, W_UV, gate
struct UpParams {
    const int *lens, *counts;
    __half *ws_rows;
    uint8_t *ws_exp;
    const float *ws_m, *ws_l;
    const int2 *ws_tile;
    const int4 *ws_cut;
    long long all_rows;
    const __nv_bfloat16 *gate;
    __nv_bfloat16 *out;
    int *err;
    int max_rounds, G;
    int B, T, H, tiles, bs, max_blocks;
};

// 16 columns of a row by each lane of a warp, as they are stored: f16 and the exponent of the 32 that they are half of.
struct RowPiece {
    uint4 v[2];
    int E;
    __device__ __forceinline__ void load(const UpParams &p, long long row, int lane) {
        ld_global_32B(p.ws_rows + row * kR + lane * 16, v[0], v[1]);
        E = __ldg(p.ws_exp + row * 16 + (lane >> 1));
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        const float down = row_down(E);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 y = row_values(w[k], down);
            x[2 * k] = y.x, x[2 * k + 1] = y.y;
        }
    }
};

// Parts c0, c0 + step, ... of a tile's row r by one warp: the running maximum M (log2 units), the sum of the weights and,
// 16 latent columns per lane, the weighted sum.  Share `first` started the tile; those up to `last` went on with it.
__device__ __forceinline__ void join_parts(const UpParams &p, int first, int last, int r, int c0, int step, int lane,
                                           float (&o)[16], float &M, float &sum) {
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
    M = -INFINITY, sum = 0.f;
    const auto part = [&](int c) { return part_number(c, c == first) * kM + r; };
    for (int c = first + c0; c <= last; c += 32 * step) {   // a lane per part: maxima and weights, 32 at a time
        const int mine = c + lane * step;
        const bool has = mine <= last;
        const float m = has ? __ldg(p.ws_m + part(mine)) : -INFINITY, l = has ? __ldg(p.ws_l + part(mine)) : 0.f;
        float top = m;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        top = fmaxf(top, M);
        // a part that the row sees nothing of has weight 0 and is not read (0 / 0 = NaN)
        const float f = M == top ? 1.f : fast_exp2(M - top), g = !has || l == 0.f ? 0.f : m == top ? l : fast_exp2(m - top) * l;
        float w_all = g;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) w_all += __shfl_xor_sync(0xffffffffu, w_all, off);
        M = top;
        sum = sum * f + w_all;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] *= f;
        const int n = min(32, (last - c) / step + 1);
#pragma unroll 1
        for (int i = 0; i < n; i += 4) {   // four parts' loads in flight
            RowPiece x[4];
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = i + k < n ? __shfl_sync(0xffffffffu, g, i + k) : 0.f;
                if (w[k] != 0.f) x[k].load(p, p.all_rows + part(c + (i + k) * step), lane);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (w[k] != 0.f) {
                    float y[16];
                    x[k].get(y);
#pragma unroll
                    for (int q = 0; q < 16; ++q) o[q] = fmaf(y[q], w[k], o[q]);
                }
        }
    }
}

// The token of [B, T] numbered m: whether it is one of its sequence's new ones.
__device__ __forceinline__ bool is_token(const UpParams &p, long long m, int &b, int &t) {
    b = static_cast<int>(m / p.T), t = static_cast<int>(m - static_cast<long long>(b) * p.T);
    int len;
    return b < p.B && t < tokens(p, b, len, false);
}

// Few tokens and heads: one CTA per (head, 32 tokens).  Rows into swizzled slabs, hi over lo, from ws_rows or joined from parts, as
// many warps to a row as there are.  W_UV[h] is the M side and the rows, hi and lo, the N = 64 of one product: 32
// instructions of 53 cycles where the rows as M = 128 would take 64 of 64, and outputs that lie side by side in a warp.  All
// of W_UV's eight slabs of 64 latent columns are loaded before the pair kernel ends where every CTA has an SM to itself
// (kW = 8); otherwise two CTAs share one and two stages take the slabs in turn.
constexpr int kFewRows = 32;
constexpr int few_threads(int kW) { return kW == 8 ? 512 : 256; }   // at most
constexpr uint32_t kFewSlab = 2 * kFewRows * 128;         // [32 rows x 64 latent columns] hi, then lo
constexpr uint32_t kFewW = 8 * kFewSlab;
constexpr uint32_t few_bars(int kW) { return kFewW + kW * kSlab; }
constexpr uint32_t few_smem(int kW) { return few_bars(kW) + 192 + 1024; }
static_assert(few_threads(8) / 32 * kR * 4 <= 8 * kFewSlab, "the warps' sums fit where the rows go");

template <int kW>
__global__ void __launch_bounds__(few_threads(kW), kW == 8 ? 1 : 2)
    attend_few_kernel(const __grid_constant__ CUtensorMap tm_w, const UpParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint64_t *const w_full = reinterpret_cast<uint64_t *>(smem_raw + (base - raw) + few_bars(kW));   // [kW]
    uint64_t *const w_empty = w_full + kW;                                                            // [kW]
    uint64_t *const done = w_full + 2 * kW;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(w_full + 2 * kW + 1);
    __shared__ int2 s_tile[kFewRows];   // first and last share of each row's tile; {-1, .}: not a token, or nothing there
    __shared__ int s_row[kFewRows];     // the row's place in its tile
    __shared__ float s_m[few_threads(kW) / 32], s_sum[few_threads(kW) / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int h = blockIdx.x % p.H;
    const long long m0 = static_cast<long long>(blockIdx.x / p.H) * kFewRows;
    const int rows = static_cast<int>(min(static_cast<long long>(kFewRows), static_cast<long long>(p.B) * p.T - m0));

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kW + 1; ++i) mbar_init(smem_u32(w_full + i), 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), 64);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const auto load_w = [&](int k) {   // latent columns [64 k, 64 k + 64) of W_UV[h] into stage k % kW
        const uint32_t bar = smem_u32(w_full + k % kW);
        mbar_arrive_expect_tx(bar, kSlab);
        tma_load_2d(base + kFewW + (k % kW) * kSlab, &tm_w, bar, k * 64, h * kDV);
    };
    // the pair kernel launches this one after its own wait: what the call was given may be read already
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_w);
#pragma unroll 1
        for (int k = 0; k < kW; ++k) load_w(k);
        for (int k = kW; k < 8; ++k) tma_prefetch_l2_2d(&tm_w, k * 64, h * kDV);
    }
    if (p.gate && threadIdx.x < 2 * rows)   // the gate's rows, of two lines each, into L2
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.gate + ((m0 + (threadIdx.x >> 1)) * p.H + h) * kDV + (threadIdx.x & 1) * 64));
    int b = 0, t = 0;
    const bool token = threadIdx.x < rows && is_token(p, m0 + threadIdx.x, b, t);
    grid_dependency_wait();
    grid_launch_dependents();
    if (threadIdx.x < kFewRows) {
        const long long r = static_cast<long long>(t) * p.H + h;
        int2 tile = token ? p.ws_tile[static_cast<long long>(b) * p.tiles + r / kM] : make_int2(-1, -1);
        if (token && !shares_written(tile.x, tile.y, p.max_rounds * p.G)) {   // a wait ran out before the tile was done
            record_error(p.err, kDevErrTimeout);
            tile = make_int2(-1, -1);
        }
        s_tile[threadIdx.x] = tile;
        s_row[threadIdx.x] = static_cast<int>(r % kM);
    }
    __syncthreads();
    int per_row = 1;   // warps
    while (rows * per_row * 2 <= warps) per_row *= 2;
    const auto store_row = [&](int i, const float (&o)[16], float mul) {
        const uint32_t slab = base + (lane >> 2) * kFewSlab;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) hi[q] = split_bf16x2(o[8 * k + 2 * q] * mul, o[8 * k + 2 * q + 1] * mul, lo[q]);
            const uint32_t at = slab + sw128_offset(i, (lane & 3) * 2 + k);
            st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(at + kFewSlab / 2, lo[0], lo[1], lo[2], lo[3]);
        }
    };
    for (int i0 = 0; i0 < rows; i0 += warps / per_row) {
        const int i = i0 + warp / per_row, c0 = warp % per_row;
        const int2 tile = i < rows ? s_tile[i] : make_int2(-1, -1);
        const bool cut = tile.x >= 0 && tile.x != tile.y;
        float o[16], M = -INFINITY, sum = 1.f;
        if (cut) {
            join_parts(p, tile.x, tile.y, s_row[i], c0, per_row, lane, o, M, sum);
        } else if (tile.x >= 0 && c0 == 0) {
            RowPiece x;
            x.load(p, (m0 + i) * p.H + h, lane);
            x.get(o);
        }
        if (per_row > 1) {   // once: the row's first warp adds up the others' sums, in their order
            if (cut && c0 > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    st_shared_v4(base + warp * (kR * 4) + k * 512 + lane * 16, __float_as_uint(o[4 * k]),
                                 __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
                if (lane == 0) s_m[warp] = M, s_sum[warp] = sum;
            }
            __syncthreads();
            if (cut && c0 == 0) {
                float top = M;
                for (int k = 1; k < per_row; ++k) top = fmaxf(top, s_m[warp + k]);
                const float f = M == top ? 1.f : fast_exp2(M - top);
                sum *= f;
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= f;
#pragma unroll 1
                for (int k = 1; k < per_row; ++k) {
                    if (s_sum[warp + k] == 0.f) continue;
                    const float g = s_m[warp + k] == top ? 1.f : fast_exp2(s_m[warp + k] - top);
                    sum = fmaf(s_sum[warp + k], g, sum);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 x = ld_shared_v4(base + (warp + k) * (kR * 4) + q * 512 + lane * 16);
                        o[4 * q] = fmaf(__uint_as_float(x.x), g, o[4 * q]);
                        o[4 * q + 1] = fmaf(__uint_as_float(x.y), g, o[4 * q + 1]);
                        o[4 * q + 2] = fmaf(__uint_as_float(x.z), g, o[4 * q + 2]);
                        o[4 * q + 3] = fmaf(__uint_as_float(x.w), g, o[4 * q + 3]);
                    }
                }
            }
            __syncthreads();
        }
        if (tile.x >= 0 && c0 == 0) store_row(i, o, 1.f / sum);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t idesc = make_idesc_bf16(kDV, 2 * kFewRows, 0, 0);
        const uint64_t rows0 = make_smem_desc(base, 16, 1024), w0 = make_smem_desc(base + kFewW, 16, 1024);
        bool ok = true;
        int loaded = kW;
#pragma unroll 1
        for (int k = 0; ok && k < 8; ++k) {
            const int st = k % kW;
            if (!(ok = mbar_wait(smem_u32(w_full + st), (k / kW) & 1, p.err))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                umma_bf16(tmem, desc_add(w0, st * kSlab + kk * 32), desc_add(rows0, k * kFewSlab + kk * 32), idesc, (k | kk) != 0);
            if (k + kW < 8) {   // the stage is refilled once its products completed
                umma_commit(smem_u32(w_empty + st));
                if (!(ok = mbar_wait(smem_u32(w_empty + st), (k / kW) & 1, p.err))) break;
                load_w(k + kW);
                ++loaded;
            }
        }
        if (ok) umma_commit(smem_u32(done));
        if (!ok)   // no load may still be landing when the CTA exits
            for (int k = loaded - kW; k < loaded; ++k)
                mbar_wait(smem_u32(w_full + k % kW), (k / kW) & 1, p.err, nullptr, kLandNs);
    }
    __syncwarp();
    if (warp < kDV / 32) {   // thread = output column, TMEM column = token
        // kN tokens at a time, so many gates' loads in flight: 8 in short calls, whose code is short too (18.4 us against 19.2
        // with 32 for 4 tokens of 8 heads), else 32 (64 tokens of 96 heads: 90 us against 97)
        constexpr int kN = kW == 8 ? 8 : kFewRows;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        bool good = true;
#pragma unroll 1
        for (int i0 = 0; good && i0 < rows; i0 += kN) {
            const long long off = ((m0 + i0) * p.H + h) * kDV + threadIdx.x, step = static_cast<long long>(p.H) * kDV;
            __nv_bfloat16 g[kN];
            if (p.gate)
#pragma unroll
                for (int k = 0; k < kN; ++k)
                    if (i0 + k < rows && s_tile[i0 + k].x >= 0) g[k] = p.gate[off + k * step];
            good = __all_sync(0xffffffffu, mbar_wait(smem_u32(done), 0, p.err));
            if (!good) break;
            tc_fence_after();
            float hi[kN], lo[kN];
            if constexpr (kN == 8) {
                tmem_ld8(lanes + i0, hi);
                tmem_ld8(lanes + kFewRows + i0, lo);
            } else {
                tmem_ld32(lanes, hi);
                tmem_ld32(lanes + kFewRows, lo);
            }
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                float y = hi[k] + lo[k];
                if (p.gate) y *= __fdividef(1.f, 1.f + fast_exp2(-__bfloat162float(g[k]) * kLog2e));
                if (i0 + k < rows && s_tile[i0 + k].x >= 0) p.out[off + k * step] = __float2bfloat16(y);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 64);
}

// Many tokens, first: the cut tiles' parts into rows.  Eight CTAs per cluster, for its shares that left a tile unfinished; a
// warp per row.
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const UpParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, r = (blockIdx.x & 7) * 16 + (threadIdx.x >> 5);
    for (int round = 0; round < p.max_rounds; ++round) {
        const int4 cut = p.ws_cut[round * p.G + (blockIdx.x >> 3)];
        if (r >= cut.y) continue;
        float o[16], M, sum;
        join_parts(p, cut.z, cut.w, r, 0, 1, lane, o, M, sum);
        const float inv = 1.f / sum;
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] *= inv, top = fmaxf(top, fabsf(o[k]));
        const int E = row_exponent(fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1)));   // of 32 columns
        const float up = row_up(E);
        uint32_t x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = pack_f16x2(o[2 * k] * up, o[2 * k + 1] * up);
        const long long row = cut.x + r;
        st_global_32B(p.ws_rows + row * kR + lane * 16, make_uint4(x[0], x[1], x[2], x[3]), make_uint4(x[4], x[5], x[6], x[7]));
        if ((lane & 1) == 0) p.ws_exp[row * 16 + (lane >> 1)] = static_cast<uint8_t>(E);
    }
}

// Many tokens, then: out = gate * (hi + lo) . W_UV[h]^T, 128 tokens of a head at a time.  Persistent: a CTA takes a run of
// items, the blocks of one head after the other, with W_UV[h] in shared memory while the head stays.  A stage takes 64
// latent columns of f16 rows; two warpgroups (thread = row) turn every other one into hi and lo in TMEM, the A operands of
// the products, so that shared memory has room for four loads in flight.  Two accumulators: four more warps gate and store
// one item while the next one's products run.
// 393,216 rows (8 x 512 tokens of 96 heads, 516 MB with W_UV and out) take 110 us, 4.7 TB/s, gated (617 MB) 137; with hi
// and lo in shared memory, three stages and every lane loading and storing a row of its own 153 and 181.
constexpr int kUpThreads = 448;   // warps 0 TMA, 1 MMA, 2-9 split, 10-13 store
constexpr int kUpStages = 4;   // of the loads' ring in shared memory and of the split ones' in TMEM: two turns per item
constexpr uint32_t kUpA = 8 * kSlab;
constexpr uint32_t kUpOut = kUpA + kUpStages * kSlab;   // [128 tokens x 128] bf16
constexpr uint32_t kUpBars = kUpOut + kM * kDV * 2;
struct UpBars {
    uint64_t w_full[8], w_empty[8], full[kUpStages], empty[kUpStages], split[kUpStages], done[kUpStages], acc_full[2], acc_empty[2];
    uint32_t tmem_base;
};
constexpr uint32_t kUpSmem = kUpBars + 384 + 1024;
static_assert(sizeof(UpBars) <= 384 && kUpSmem <= 232448, "shared memory");
constexpr uint32_t kUpSplit = 256;   // TMEM: two accumulators of 128 columns, then stages of 32 columns of hi and 32 of lo

__global__ void __launch_bounds__(kUpThreads, 1)
    attend_up_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w, const UpParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    UpBars *const bars = reinterpret_cast<UpBars *>(smem_raw + (base - raw) + kUpBars);
    const auto B_ = [](uint64_t &b) { return smem_u32(&b); };
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const long long m_all = static_cast<long long>(p.B) * p.T;
    const int blocks = static_cast<int>((m_all + kM - 1) / kM);
    const long long items = static_cast<long long>(blocks) * p.H;
    const int i0 = static_cast<int>(items * blockIdx.x / gridDim.x), i1 = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(B_(bars->w_full[i]), 1), mbar_init(B_(bars->w_empty[i]), 1);
        for (int i = 0; i < kUpStages; ++i) {
            mbar_init(B_(bars->full[i]), 1);
            mbar_init(B_(bars->empty[i]), 128);
            mbar_init(B_(bars->split[i]), 128);
            mbar_init(B_(bars->done[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(B_(bars->acc_full[i]), 1);
            mbar_init(B_(bars->acc_empty[i]), 128);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    const auto wait = [&](uint64_t &bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(B_(bar), parity, p.err));
    };
    if (warp == 0) {
        const bool lead = elect_one();
        Ring<kUpStages> at;
        uint32_t it = 0, w_phase = 0;
        int head = -1;
        bool ok = true;
        for (int i = i0; ok && i < i1; ++i) {
            const int h = i / blocks, m0 = (i - h * blocks) * kM;
            const bool new_head = h != head;
#pragma unroll 1
            for (int k = 0; k < 8; ++k, ++it, at.next()) {
                if (new_head) {   // a slab of the next head's W_UV as soon as this one's last products with it are done
                    if (!(ok = wait(bars->w_empty[k], w_phase ^ 1))) break;
                    if (lead) {
                        mbar_arrive_expect_tx(B_(bars->w_full[k]), kSlab);
                        tma_load_2d(base + k * kSlab, &tm_w, B_(bars->w_full[k]), k * 64, h * kDV);
                    }
                }
                if (it == 0) {   // W_UV was there before the kernels that this one waits for
                    grid_dependency_wait();
                    fence_proxy_async_all();
                }
                if (!(ok = wait(bars->empty[at.st], at.phase ^ 1))) break;
                if (lead) {
                    mbar_arrive_expect_tx(B_(bars->full[at.st]), kSlab);
                    tma_load_3d(base + kUpA + at.st * kSlab, &tm_a, B_(bars->full[at.st]), k * 64, h, m0);
                }
            }
            w_phase ^= new_head;
            head = h;
        }
        // no load may still be landing when the CTA exits
        for (uint32_t k = it > kUpStages ? it - kUpStages : 0; k < it; ++k)
            mbar_wait(B_(bars->full[k % kUpStages]), (k / kUpStages) & 1, p.err, nullptr, kLandNs);
        for (int k = 0; ok && head >= 0 && k < 8; ++k) mbar_wait(B_(bars->w_full[k]), w_phase ^ 1, p.err, nullptr, kLandNs);
    } else if (warp == 1) {
        const bool lead = elect_one();
        const uint32_t idesc = make_idesc_bf16(128, kDV, 0, 0);
        const uint64_t w0 = make_smem_desc(base, 16, 1024);
        Ring<kUpStages> at;
        Ring<2> acc;
        uint32_t w_phase = 1;   // of the head that is there
        int head = -1;
        bool ok = true;
        for (int i = i0; ok && i < i1; ++i, acc.next()) {
            const int h = i / blocks;
            w_phase ^= h != head;
            head = h;
            const bool last = i + 1 == i1 || (i + 1) / blocks != h;   // of the head's items here
            if (!(ok = wait(bars->acc_empty[acc.st], acc.phase ^ 1))) break;
            const uint32_t d = tmem + acc.st * 128;
#pragma unroll 1
            for (int k = 0; k < 8; ++k, at.next()) {
                if (!(ok = wait(bars->w_full[k], w_phase)) || !(ok = wait(bars->split[at.st], at.phase))) break;
                tc_fence_after();
                if (lead) {
                    const uint32_t a = tmem + kUpSplit + at.st * 64;
                    const uint64_t w = desc_add(w0, k * kSlab);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        umma_bf16_tmem_a(d, a + kk * 8, desc_add(w, kk * 32), idesc, (k | kk) != 0);
                        umma_bf16_tmem_a(d, a + 32 + kk * 8, desc_add(w, kk * 32), idesc, 1);
                    }
                    umma_commit(B_(bars->done[at.st]));
                    if (last) umma_commit(B_(bars->w_empty[k]));
                }
            }
            if (ok && lead) umma_commit(B_(bars->acc_full[acc.st]));
        }
    } else if (warp < 10) {
        grid_dependency_wait();
        const int r = (warp & 3) * 32 + lane, group = (warp - 2) >> 2;   // every other slab
        const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kUpSplit;
        const auto exponents = [&](int i) {
            const int h = i / blocks;
            const long long m = static_cast<long long>(i - h * blocks) * kM + r;
            return i < i1 && m < m_all ? __ldg(reinterpret_cast<const uint4 *>(p.ws_exp) + m * p.H + h) : uint4();
        };
        uint4 next = exponents(i0);
        bool ok = true;
        for (int i = i0; ok && i < i1; ++i) {
            const uint4 E = next;
            next = exponents(i + 1);
#pragma unroll 1
            for (int k = group; k < 8; k += 2) {
                const int st = k & 3, phase = k >> 2;
                if (!(ok = wait(bars->full[st], phase))) break;
                const uint32_t slab = base + kUpA + st * kSlab;
                const uint32_t e = (k < 4 ? k < 2 ? E.x : E.y : k < 6 ? E.z : E.w) >> (group * 16);
                float hi[32], lo[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    // (no token's row may hold anything)
                    const float down = row_down(max(static_cast<int>(e >> (c < 4 ? 0 : 8) & 0xFF), 20));
                    const uint4 v = ld_shared_v4(slab + sw128_offset(r, c));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 x = row_values(w[q], down);
                        uint32_t rest;
                        hi[4 * c + q] = __uint_as_float(split_bf16x2(x.x, x.y, rest));
                        lo[4 * c + q] = __uint_as_float(rest);
                    }
                }
                fence_proxy_async_smem();   // TMA writes there again
                mbar_arrive(B_(bars->empty[st]));
                if (!(ok = wait(bars->done[st], phase ^ 1))) break;
                tc_fence_after();
                tmem_st32(to + st * 64, hi);
                tmem_st32(to + st * 64 + 32, lo);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(B_(bars->split[st]));
            }
        }
    } else {
        grid_dependency_wait();
        grid_launch_dependents();
        // A lane has a row of the accumulator, but memory wants a row from 16 lanes: gates come and outputs go through shared
        // memory, 16 bytes c of row q at c ^ (q & 7), each warp for its own 32 rows.
        const int w0 = (warp & 3) * 32;
        const uint32_t row = tmem + (static_cast<uint32_t>(w0) << 16), stage = base + kUpOut + w0 * 256;
        const auto cell = [&](int q, int c) { return stage + q * 256 + ((c ^ (q & 7)) << 4); };
        uint4 g[16];
        uint32_t tokens = 0;
        // which of the item's 32 tokens there are, and their gates
        const auto ask = [&](int i) {
            if (i >= i1) return;
            const int h = i / blocks;
            const long long m0 = static_cast<long long>(i - h * blocks) * kM + w0;
            int b, t;
            tokens = __ballot_sync(0xffffffffu, is_token(p, m0 + lane, b, t));
            if (!p.gate) return;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int q = 2 * k + (lane >> 4);
                if ((tokens >> q) & 1)
                    g[k] = __ldg(reinterpret_cast<const uint4 *>(p.gate + ((m0 + q) * p.H + h) * kDV) + (lane & 15));
            }
        };
        ask(i0);
        Ring<2> acc;
        bool ok = true;
        for (int i = i0; ok && i < i1; ++i, acc.next()) {
            const int h = i / blocks;
            const long long m0 = static_cast<long long>(i - h * blocks) * kM + w0;
            const uint32_t here = tokens;
            if (p.gate) {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    st_shared_v4(cell(2 * k + (lane >> 4), lane & 15), g[k].x, g[k].y, g[k].z, g[k].w);
                __syncwarp();
            }
            ask(i + 1);
            if (!(ok = wait(bars->acc_full[acc.st], acc.phase))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float o[32];
                tmem_ld32(row + acc.st * 128 + c * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t to = cell(lane, c * 4 + k);
                    if (p.gate) {
                        const uint4 g = ld_shared_v4(to);
                        const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            o[8 * k + 2 * n] *= __fdividef(1.f, 1.f + fast_exp2(-__uint_as_float(gw[n] << 16) * kLog2e));
                            o[8 * k + 2 * n + 1] *= __fdividef(1.f, 1.f + fast_exp2(-__uint_as_float(gw[n] & 0xFFFF0000u) * kLog2e));
                        }
                    }
                    st_shared_v4(to, pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                 pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
                }
            }
            tc_fence_before();
            mbar_arrive(B_(bars->acc_empty[acc.st]));
            __syncwarp();
#pragma unroll 4
            for (int k = 0; k < 16; ++k) {
                const int q = 2 * k + (lane >> 4);
                if ((here >> q) & 1)
                    reinterpret_cast<uint4 *>(p.out + ((m0 + q) * p.H + h) * kDV)[lane & 15] = ld_shared_v4(cell(q, lane & 15));
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

CUresult encode_map(CUtensorMap *m, const void *ptr, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                    const cuuint32_t *box) {
    auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
    if (!fn) return CUDA_ERROR_NOT_SUPPORTED;
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(ptr), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// What is asked of a device once: the kernels' attributes, and how many clusters of the pair kernel run at once.
cudaError_t prepare(int num_sms, int &clusters) {
    constexpr int kMaxDev = 64;
    static std::atomic<int> cached[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDev && (clusters = cached[dev].load()) > 0) return cudaSuccess;
    const auto smem = [](auto *kernel, uint32_t bytes) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    };
    if ((e = smem(attend_pair_kernel, kSmemPair)) != cudaSuccess) return e;
    if ((e = smem(attend_few_kernel<2>, few_smem(2))) != cudaSuccess) return e;
    if ((e = smem(attend_few_kernel<8>, few_smem(8))) != cudaSuccess) return e;
    if ((e = smem(attend_up_kernel, kUpSmem)) != cudaSuccess) return e;
    cudaFuncAttributes fa;   // the register split assumes this launch budget
    if ((e = cudaFuncGetAttributes(&fa, attend_pair_kernel)) != cudaSuccess) return e;
    if (fa.numRegs != static_cast<int>(kRegsLaunch)) return cudaErrorInvalidConfiguration;
    const int cap = num_sms / 2 > 0 ? num_sms / 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * cap);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemPair;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, attend_pair_kernel, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = cap;
    }
    clusters = n < cap ? n : cap;
    if (dev < kMaxDev) cached[dev].store(clusters);
    return cudaSuccess;
}

// The workspace: rows, parts, tiles' shares, shares' unfinished tiles.
struct Space {
    size_t exp, m, l, tile, cut, end;
    int tiles, rounds;
    Space(long long B, long long T, int H, int num_sms) {
        tiles = static_cast<int>((T * H + kM - 1) / kM);
        rounds = B > 1 ? std::max(1, std::min(tiles / kRoundTiles, kRounds)) : 1;
        const size_t shares = static_cast<size_t>(num_sms / 2 > 0 ? num_sms / 2 : 1) * rounds, parts = shares * 2 * kM;
        const size_t rows = static_cast<size_t>(B) * T * H + parts;
        exp = rows * kR * 2;
        m = exp + rows * 16;
        l = m + parts * 4;
        tile = l + parts * 4;
        cut = (tile + static_cast<size_t>(B) * tiles * sizeof(int2) + 15) / 16 * 16;
        end = cut + shares * sizeof(int4) + 16;   // the base goes up to 32 bytes
    }
};

}  // namespace

bool attend_paged_supports(int H, int d_v, int r) { return r == kR && d_v == kDV && H >= 1 && H <= 128; }

size_t attend_paged_workspace_bytes(long long B, long long T, int H, int num_sms) { return Space(B, T, H, num_sms).end; }

cudaError_t launch_attend_paged(const AttendPagedArgs &a, cudaStream_t s) {
    const Space sp(a.B, a.T, a.H, a.num_sms);
    if (sp.end > a.workspace_bytes) return cudaErrorInvalidValue;
    int G = 0;
    cudaError_t e = prepare(a.num_sms, G);
    if (e != cudaSuccess) return e;
    CUtensorMap tm_q, tm_s, tm_v, tm_w;
    {
        const long long rows = static_cast<long long>(a.num_blocks) * a.bs;
        const void *const pool = rows > 0 ? a.pool : a.q_abs;   // no row of an empty pool is inside its map
        const cuuint64_t n = static_cast<cuuint64_t>(rows > 0 ? rows : 1), ld = static_cast<cuuint64_t>(a.ld_pool) * 2;
        const cuuint64_t dims_s[2] = {kR, n}, dims_v[3] = {64, n, kR / 64};
        const cuuint64_t strides_s[1] = {ld}, strides_v[2] = {ld, 128};
        const cuuint32_t box_s[2] = {64, 64}, box_v[3] = {64, kVRows, 4};
        const cuuint64_t dims_w[2] = {kR, static_cast<cuuint64_t>(a.H) * kDV}, strides_w[1] = {kR * 2};
        const cuuint32_t box_w[2] = {64, kDV};
        const cuuint64_t dims_q[2] = {kR, static_cast<cuuint64_t>(a.B) * a.T * a.H};
        if (encode_map(&tm_q, a.q_abs, 2, dims_q, strides_w, box_s) != CUDA_SUCCESS ||
            encode_map(&tm_s, pool, 2, dims_s, strides_s, box_s) != CUDA_SUCCESS ||
            encode_map(&tm_v, pool, 3, dims_v, strides_v, box_v) != CUDA_SUCCESS ||
            encode_map(&tm_w, a.w_uv, 2, dims_w, strides_w, box_w) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    char *const ws = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(a.workspace) + 31) & ~static_cast<uintptr_t>(31));
    auto *const ws_rows = reinterpret_cast<__half *>(ws);
    auto *const ws_exp = reinterpret_cast<uint8_t *>(ws + sp.exp);
    float *const ws_m = reinterpret_cast<float *>(ws + sp.m), *const ws_l = reinterpret_cast<float *>(ws + sp.l);
    int2 *const ws_tile = reinterpret_cast<int2 *>(ws + sp.tile);
    int4 *const ws_cut = reinterpret_cast<int4 *>(ws + sp.cut);
    const long long m = static_cast<long long>(a.B) * a.T;
    const long long all_rows = m * a.H;
    const PairParams pp{a.table, a.lens, a.counts, a.parents, a.ld_table,
                        ws_rows, ws_exp, ws_m, ws_l, ws_tile, ws_cut, all_rows, a.dev_err, sp.rounds, a.B, a.T, a.H, sp.tiles,
                        a.num_blocks, a.bs, a.max_blocks, a.window, a.sinks, a.scale * kLog2e, Divisor(a.H), Divisor(sp.tiles), Divisor(a.bs)};
    note_launch();
    e = launch_dependent(attend_pair_kernel, dim3(2 * G), kThreads, kSmemPair, s, tm_q, tm_s, tm_v, pp);
    if (e != cudaSuccess) return e;
    const UpParams up{a.lens, a.counts, ws_rows, ws_exp, ws_m, ws_l, ws_tile, ws_cut, all_rows,
                      static_cast<const __nv_bfloat16 *>(a.gate), static_cast<__nv_bfloat16 *>(a.out), a.dev_err, sp.rounds,
                      G, a.B, a.T, a.H, sp.tiles, a.bs, a.max_blocks};
    // Where all its CTAs run at once (two of kW = 2 to an SM), the join, W_UV and the gate are one kernel of short CTAs; two
    // kernels otherwise.  One token of 96 heads over 30000 rows takes 26.8 us with the one and 51.1 with the two, 64 tokens of
    // 64 heads 81 and 88, 512 of 8 heads 40 and 44, 128 of 64 heads 86.8 and 87.2, 128 of 96 heads (384 CTAs) 125 and 113.
    const long long ctas = (m + kFewRows - 1) / kFewRows * a.H;
    if (ctas <= 2 * a.num_sms) {
        note_launch();
        const dim3 grid(static_cast<unsigned>(ctas));
        // Twice the warps for more than 8 rows: 32 tokens of 8 heads 29.5 -> 27.1 us, of 96 heads 89.0 -> 85.7; 4 tokens of 8
        // heads 17.7 with few and 18.1 with many.
        const int kW = ctas <= a.num_sms ? 8 : 2, threads = m > 8 ? few_threads(kW) : 256;
        return kW == 8 ? launch_dependent(attend_few_kernel<8>, grid, threads, few_smem(8), s, tm_w, up)
                       : launch_dependent(attend_few_kernel<2>, grid, threads, few_smem(2), s, tm_w, up);
    }
    CUtensorMap tm_a;
    {
        const cuuint64_t row = kR * 2, dims[3] = {kR, static_cast<cuuint64_t>(a.H), static_cast<cuuint64_t>(m)};
        const cuuint64_t strides[2] = {row, row * a.H};
        const cuuint32_t box[3] = {64, 1, kM};
        if (encode_map(&tm_a, ws_rows, 3, dims, strides, box) != CUDA_SUCCESS) return cudaErrorInvalidValue;
    }
    note_launch();
    e = launch_dependent(attend_join_kernel, dim3(8 * G), kJoinThreads, 0, s, up);
    if (e != cudaSuccess) return e;
    note_launch();
    const long long items = (m + kM - 1) / kM * a.H;
    return launch_dependent(attend_up_kernel, dim3(static_cast<unsigned>(items < a.num_sms ? items : a.num_sms)), kUpThreads,
                            kUpSmem, s, tm_a, tm_w, up);
}

}  // namespace mla
