// Cached-latent decode over the fp4 latent cache (latent_fp4.cu) on the sm_103a tensor cores: r = 512, d_v = 128,
// 1 <= H <= 96.
//
// Sequence b's absorbed query q_abs[b] (all H heads) attends to its cache rows [0, lens[b]); steps 2-4 of section
// "完整计算流（四步）" of the page "Gated MLA（矩阵吸收版）" follow: scores against c itself, softmax, the latent
// weighting by c itself, W_UV^T, gate.
//
// Attention kernel (persistent, one CTA per SM).  A CTA takes all heads and a contiguous share of all sequences' rows, in
// units of 128 rows, and computes both products with the rows' side as M:
//   S^T [128 rows x heads]       = c . q_abs^T     A = c as stored, K-major       (K = r)
//   O^T [128 latent x heads] x 4 += c^T . P^T      A = the same tile, MN-major    (K = rows)
// so a unit is expanded once, to e4m3 in shared memory, for both, heads are not padded to 128, and O^T (fp32) leaves room
// in tensor memory for S^T.  An e2m1 value times its group's power of two is exact in e4m3 relative to its row's largest
// scale, 14 binades down, so the tile is the row divided by a power of two, `ref`, that goes into the softmax's exponent.
// Where a group of other values than zeros lies further down, e4m3 would round it or lose it: the expanding warps mark the
// CTA's share, and the merge does the share's segments again in fp32 from the codes (no real latent does that; 64 x 16384
// such rows take 6.0 ms at 16 heads).  q_abs and P are split into two 8-bit parts:
//   up to 48 heads   e4m3 hi and lo = e4m3(16 x rest), side by side as 2 x heads columns of the N side: one pass over the
//                    tile serves both parts, which the fp32 epilogues join
//   above            the two parts' products go into the same accumulators, as 2 x heads columns would not fit tensor
//                    memory: unscaled, q_abs's lo in e4m3, P's in e5m2 for its range
// Of a bf16 query, whose head's largest element is brought to [128, 256), both hold everything but what lies below lo's
// last step: elements below 2^-9 of the largest are off by at most 2^-14 (above 48 heads 2^-10).
//
// Softmax of one unit: thread = row, so every head's statistics lie across lanes.  With a = score * log2 e + ref,
//   P = 2^(a - M + 8), l += P * 2^-ref,   M[head] >= running max of a - 0.75
// M moves when some row exceeds it by more than 0.75 (P <= 2^8.75 = 430, inside e4m3's 448), to kHead above that row: a
// barrier with an OR tells whether any does, and only then are the maxima taken across lanes and the moved heads' columns
// of O^T rescaled.  The two 8-bit parts of P are off by 2^-8 of it (above 48 heads 2^-7), or by 2^-14 where hi is subnormal
// (half a step of lo up to 48 heads; above, e5m2's 2^-4 of a rest of 2^-10), while l takes all of it.  2^-14 is 2^-21 of
// the largest P when M was set.  So that thousands of light rows behind one heavy row are not lost, M is set anew, higher
// or up to kDrop lower, every kWindow units: rows behind the heavy one lose at most 2^-21 of its P each in its window, 2^-24
// in the next and so on, 4096 * 2^-21 * 8/7 = 1.15 * 2^-9 of it in all (and over a segment's eight windows O^T and l grow by
// 2^21 at most, well inside fp32).  64 x 16384 rows, scores of a deviation of 5, with M never lowered / a drop of 3 / to
// any depth: 48 heads 170 / 172 / 174 us, 96 heads 256 / 257 / 260.
//
// Warps: 0 loads scale bytes (TMA) and turns them into table numbers, 1 issues S, 2 issues O, 3 loads codes (TMA); two
// (above 48 heads: four) softmax warpgroups, each with its share of the heads, that never wait for one another (also
// q_abs, rescale and drain); two warpgroups expand, every other slab of 128 latent columns each.  The expansion is a byte
// permute per four codes: the group's exponent selects an 8-byte table of e4m3 magnitudes, the codes' three magnitude
// bits are the selector.
//
// What bounds it (64 x 16384 rows, scores of a deviation of 5, 1.85 GHz): at 96 heads 242 us and 17 of the merge, 8400 cycles
// a unit, of which the tensor pipe is busy 46 % (64 products of about 56 cycles: shared memory feeds it 128 bytes a cycle).
// The queries' 96 KB leave room for one unit of expanded slabs and one slab more, so a unit's expansion, S, softmax and O
// mostly follow one another, each slab of the next unit expanded as O leaves one.  At 48 heads 171 us with the merge (144
// for scores of a deviation of 0.5, where the maxima seldom move), at 16 heads 106 (3300 cycles a unit; tensor pipe 46 %,
// ALUs 55 %: the expansion's byte permutes and logic; nothing is full).  HBM is at 0.16 to 0.38 of its
// peak.  All roles' loops share an instruction cache that they overflow easily: waits that carry their error path and
// issue loops unrolled fourfold cost 193 us instead of 127 at 16 heads, which is why loops here are kept rolled, issuing
// warps converged and cold code short.
//
// Merge kernels: the segments of a sequence are joined with the log-sum-exp rule and multiplied by W_UV^T, then the gate.
// Few (head, sequence) pairs: a CTA per head and up to four sequences, the product in fp32 from W_UV[h] in shared memory.
// Many: a CTA per head and 32 sequences, o_lat as bf16 hi + lo (2^-17 of a value off, far below the output's own rounding),
// on the tensor cores (W_UV as the M side).
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kR = 512;
constexpr int kDV = 128;
constexpr int kRows = 128;                 // cache rows per unit
constexpr int kChunkUnits = 256;           // units of a sequence that share one running maximum per segment
constexpr int kChunkRows = kChunkUnits * kRows;
// A segment's start and end in units: 64 ragged sequences up to 32768 rows at 96 heads 270 / 266 / 266 / 267 us with 1 / 2 /
// 3 / 4, up to 8192 rows at 64 heads 86 / 86 / 86 / 89, at 48 heads 73 / 73 / 73 / 75, at 16 heads 46 / 47 / 47 / 48.
constexpr int kOver = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kBias = 8.f;               // P = 2^(a - M + kBias)
constexpr float kSlack = 0.75f;            // how far a row may exceed M before M moves
constexpr float kHead = 1.f;               // M is set this far above the row that forces it
constexpr int kWindow = 32;                // units after which M is set anew
constexpr float kDrop = 3.f;               // how far it may then fall
constexpr uint32_t kSlab = 16384;          // [128 rows x 128 latent] e4m3, 128-byte swizzle
constexpr uint32_t kPicks = 2048;          // [128 rows x 16 groups] table numbers of a unit
constexpr uint32_t kStage = 8192;          // codes of one slab: [128 rows x 64 bytes]
constexpr int kMaxPickBufs = 4;
// Tables of a group's magnitudes, by its exponent below the row's largest (kTop); below kExact e4m3 rounds some of them.
constexpr int kTop = 20, kExact = 6, kNanTable = 21, kPastTable = 22, kTables = 23;   // (rows past the end: zeros)
constexpr int kMaxSoftWarps = 16, kMaxHW = 24;

struct Fp4Shared {
    uint64_t stage_full[4], stage_empty[4];
    uint64_t scale_full[kMaxPickBufs], pick_full[kMaxPickBufs], pick_empty[kMaxPickBufs];
    uint64_t slab_full[8], slab_free[8];
    uint64_t s_full[2], s_free[2], q_ready;
    uint64_t p_full[2], p_free[2];
    uint32_t tmem_base;
    uint2 table[kTables];
    int16_t ref[8][kRows];                 // per row of the last eight units: the power of two its tile is divided by
    alignas(16) float mul[96];             // per head: score factor
    // per softmax warpgroup and head: kBias - M, and the last change of it with its power of two
    alignas(16) float bias[kMaxSoftWarps / 4][kMaxHW], step[kMaxSoftWarps / 4][kMaxHW], fac[kMaxSoftWarps / 4][kMaxHW];
    // per softmax warp: maxima, and parts of l while a segment is drained
    float part[kMaxSoftWarps][kMaxHW];
    bool low[8];                           // of the last eight units: whether any group takes a table below kExact
};

// Heads are padded to HP and shared by the softmax warpgroups, HW each.  kJoin: hi and lo parts have columns of their own,
// per pair of heads the two hi parts, then the two lo parts; else head h is column h of both.
template <int HP>
struct Fp4Layout {
    static constexpr bool kJoin = HP <= 48;
    static constexpr int kSoftGroups = kJoin ? 2 : 4, kExpGroups = 2, kGroups = 1 + kSoftGroups + kExpGroups;
    static constexpr int kThreads = 128 * kGroups, HW = HP / kSoftGroups, N = kJoin ? 2 * HP : HP;   // N: columns of an MMA
    static constexpr int WC = N / kSoftGroups;                          // columns of a warpgroup
    // Expanded slabs in flight (four per unit), stages of codes and buffers of table numbers, as the queries leave room:
    // 64 x 16384 rows, us with slabs + stages and scores of a deviation of 5 / 0.5: 16 heads 106 / 106 with 8 + 4, 117 / 105
    // with 7 + 4; 32 heads 131 / 128 with 8 + 2, 144 / 125 with 7 + 4; 48 heads 171 / 144 with 7 + 2, 177 / 152 with 6 + 4;
    // 64 heads 211 / 186 with 6 + 2, 221 / 198 with 5 + 4; 96 heads 258 / 237 with 5 + 1, 265 / 231 with 4 + 2.
    static constexpr int kSlabs = HP == 96 ? 5 : (HP == 64 ? 6 : (HP == 48 ? 7 : 8)),
                         kStages = HP == 96 ? 1 : (HP == 16 ? 4 : 2), kPickBufs = HP == 96 ? 2 : 4;
    static constexpr int kPBufs = kJoin ? 2 : 1, kSBufs = 2 * N <= 128 ? 2 : 1;
    static constexpr uint32_t kQPart = HP * 128, kQSlab = 2 * kQPart;   // [hi | lo rows x 128 latent]; kJoin: interleaved
    static constexpr uint32_t kPPart = kRows * 128, kPBuf = kJoin ? kPPart : 2 * kPPart;
    static constexpr uint32_t Q = 0, C = Q + 4 * kQSlab, P = C + kSlabs * kSlab, STAGE = P + kPBufs * kPBuf,
                              PICK = STAGE + kStages * kStage, END = PICK + kPickBufs * kPicks;
    static constexpr uint32_t kSmem = END + sizeof(Fp4Shared) + 1024;   // + alignment slack
    static constexpr uint32_t S_COL = 0, O_COL = 128;                   // TMEM columns
    // Register split of the warpgroups: control, softmax, expansion.
    static constexpr uint32_t kRegsLaunch = kJoin ? 96 : 72, kRegsCtl = kJoin ? 80 : 56, kRegsSoft = kJoin ? 104 : 88,
                              kRegsExp = kJoin ? 96 : 48;
    static_assert(kRegsCtl + kSoftGroups * kRegsSoft + kExpGroups * kRegsExp <= kGroups * kRegsLaunch,
                  "register split exceeds the launch");
    static_assert(kQPart % 1024 == 0 && O_COL + 4 * N <= 512 && kSBufs * N <= O_COL && N <= 128, "layout");
    // barriers of full stages: each is waited on by one warpgroup alone, which so sees every one of its phases
    static constexpr int kFull = kStages == 1 ? 2 : kStages;
    static_assert(kExpGroups == 2 && kFull % 2 == 0, "layout");
    static_assert(HW % 8 == 0 && HW <= kMaxHW && 4 * kSoftGroups <= kMaxSoftWarps, "layout");
    static_assert(kSlabs <= 8 && kSlabs >= 4 && END % 16 == 0 && kSmem <= 232448, "shared memory");
};

struct Fp4Params {
    const __nv_bfloat16 *q_abs;
    const int *lens;
    float *ws_o, *ws_m, *ws_l;   // [slots][H] (x r): sum of P c, M - kBias, l
    int2 *ws_seq;                // [B] per sequence: its first virtual unit and first chunk number
    int *ws_share;               // [G + 1] the shares' first virtual units
    int *ws_far;                 // [G] whether a share has rows that e4m3 cannot hold: the merge does it again
    const __nv_bfloat16 *w_uv;   // asked into L2 for the merge
    int *err;
    int B, H, max_len, G;
    float scale_log2;
};

// ------------------------------------------------------------------ the work axis
// Virtual units: a sequence is a run of chunks of up to kChunkUnits units, each preceded by kOver (what starting a segment
// costs: its queries, the first fill, the drain).  Share c of G
// owns [share_lo(c), share_lo(c + 1)); its part of chunk number v (over all sequences) is segment slot c + v: both
// only grow along the axis and one of them does between two segments.
__host__ __device__ __forceinline__ int chunks_of(int len) {
    return static_cast<int>((static_cast<unsigned>(len) + kChunkRows - 1u) / kChunkRows);
}
__device__ __forceinline__ long long units_of(int len) {   // virtual units of a sequence
    const int full = len / kChunkRows, rest = len - full * kChunkRows;
    return static_cast<long long>(full) * (kOver + kChunkUnits) + (rest > 0 ? kOver + (rest + kRows - 1) / kRows : 0);
}
// floor(total * c / G) without a 64-bit division: total = G a + b, b c < 2^18.
__device__ __forceinline__ int share_lo(int total, int c, int G) {
    const int a = total / G, b = total - a * G;
    return a * c + b * c / G;
}
__device__ __forceinline__ int read_len(const int *lens, int b, int max_len, int *err) {
    const int x = __ldg(lens + b);
    if (err && (x < 0 || x > max_len)) record_error(err, kDevErrBounds);
    return min(max(x, 0), max_len);
}
template <typename T>
__device__ __forceinline__ T warp_scan(T v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    return v;
}

struct Segment {
    int seq, row0, units, len;   // rows row0 .. row0 + 128 * units - 1, those below len
    int slot;
};

// (Positions on the axis fit 32 bits: 2^31 units are 75 TB of cache.)
struct Walk {
    const int *lens;
    int B, max_len, c, b, j;   // chunk j of sequence b is next
    int lo, hi, pre, v;          // its first virtual unit and its number
    // Every lane of a warp calls this; all get the same walk.
    __device__ void start(const Fp4Params &p, int share, int lane, int *err) {
        lens = p.lens, B = p.B, max_len = p.max_len, c = share;
        // (the first 32 sequences are often all there are: loaded once)
        const int len0 = lane < B ? read_len(lens, lane, max_len, err) : 0;
        int total = static_cast<int>(units_of(len0));
#pragma unroll 1
        for (int i = lane + 32; i < B; i += 32) total += static_cast<int>(units_of(read_len(lens, i, max_len, err)));
        total = __reduce_add_sync(0xffffffffu, total);
        lo = share_lo(total, share, p.G), hi = share_lo(total, share + 1, p.G);
        b = B, j = 0, pre = hi, v = 0;
        int run = 0, chunks = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < B && lo < hi; i0 += 32) {
            const int len = i0 == 0 ? len0 : (i0 + lane < B ? read_len(lens, i0 + lane, max_len, nullptr) : 0);
            const int u = static_cast<int>(units_of(len)), incl = warp_scan(u, lane);
            const int n = len > 0 ? chunks_of(len) : 0, nincl = warp_scan(n, lane);
            const unsigned past = __ballot_sync(0xffffffffu, run + incl > lo);
            if (past) {
                const int first = __ffs(past) - 1;
                b = i0 + first;
                pre = run + __shfl_sync(0xffffffffu, incl - u, first);
                v = chunks + __shfl_sync(0xffffffffu, nincl - n, first);
                j = (lo - pre) / (kOver + kChunkUnits);
                pre += j * (kOver + kChunkUnits);
                v += j;
                break;
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
            chunks += __shfl_sync(0xffffffffu, nincl, 31);
        }
    }
    __device__ bool next(Segment &s) {
#pragma unroll 1
        while (b < B && pre < hi) {
            const int len = read_len(lens, b, max_len, nullptr);
            if (len <= 0) {
                ++b;
                continue;
            }
            const int left = len - j * kChunkRows;   // > 0: the walk leaves a sequence with its last chunk
            const int units = left >= kChunkRows ? kChunkUnits : (left + kRows - 1) / kRows;
            const int base = pre + kOver, s0 = max(base, lo), s1 = min(base + units, hi);
            s.seq = b, s.len = len, s.slot = c + v;
            s.row0 = j * kChunkRows + (s0 - base) * kRows;
            s.units = s1 - s0;
            pre = base + units, ++v;
            if (left > kChunkRows) ++j; else ++b, j = 0;
            if (s1 > s0) return true;
        }
        return false;
    }
};

// Where each sequence and each share lies on the axis, for the merge.
__device__ __forceinline__ void write_seq(const Fp4Params &p, int lane) {
    int run = 0, chunks = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < p.B; i0 += 32) {
        const int len = i0 + lane < p.B ? read_len(p.lens, i0 + lane, p.max_len, nullptr) : 0;
        const int u = static_cast<int>(units_of(len)), n = len > 0 ? chunks_of(len) : 0;
        const int incl = warp_scan(u, lane), nincl = warp_scan(n, lane);
        if (i0 + lane < p.B) p.ws_seq[i0 + lane] = make_int2(run + incl - u, chunks + nincl - n);
        run += __shfl_sync(0xffffffffu, incl, 31);
        chunks += __shfl_sync(0xffffffffu, nincl, 31);
    }
#pragma unroll 1
    for (int c = lane; c <= p.G; c += 32) p.ws_share[c] = share_lo(run, c, p.G);
}

// The units of a walk, one after the other; rows = 0 at the end.
struct Units {
    int u, rows;
    __device__ void start(Walk &walk, Segment &seg) {
        u = -1, rows = 0, seg.units = 0;
        next(walk, seg);
    }
    __device__ void next(Walk &walk, Segment &seg) {
        rows = 0;
        if (++u >= seg.units) {
            if (!walk.next(seg)) return;
            u = 0;
        }
        rows = min(kRows, seg.len - seg.row0 - u * kRows);
    }
    __device__ int row(const Segment &seg) const { return seg.row0 + u * kRows; }
};

// ------------------------------------------------------------------ small pieces
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// (a, b) as e4m3 hi (bits 0-15) and lo (bits 16-31): hi = e4m3(x), lo = e4m3(16 (x - hi)), the difference exact in f16.
__device__ __forceinline__ uint32_t split16_e4m3x2(float a, float b) {
    const uint32_t hi = cvt_e4m3x2(a, b);
    const uint32_t rest = sub_f16x2(pack_f16x2(a, b), e4m3x2_to_f16x2(hi));
    return hi | (f16x2_to_e4m3x2(mul_f16x2(rest, 0x4C004C00u)) << 16);   // f16 16.0
}
constexpr float kLoPart = 0.0625f;
// (a, b) as e4m3 hi (bits 0-15) and e5m2 lo (bits 16-31): lo = e5m2(x - hi).
__device__ __forceinline__ uint32_t split_e4m3_e5m2x2(float a, float b) {
    const uint32_t hi = cvt_e4m3x2(a, b);
    uint16_t lo;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(lo) : "r"(sub_f16x2(pack_f16x2(a, b), e4m3x2_to_f16x2(hi))));
    return hi | static_cast<uint32_t>(lo) << 16;
}
__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
// Eight codes as e4m3 bytes by the group's table of magnitudes: three bits of each code select one of its bytes; the
// codes' fourth bits are the top bits of the bytes of w (odd codes) and of w << 4 (even ones).
__device__ __forceinline__ void expand8(uint32_t w, uint2 table, uint32_t &o0, uint32_t &o1) {
    const uint32_t m = w & 0x77777777u, w4 = w * 16u, m_hi = static_cast<uint32_t>(static_cast<uint64_t>(m) * 65536u >> 32);
    o0 = byte_perm(table.x, table.y, m) | (byte_perm(w, w4, 0x1504) & 0x80808080u);
    o1 = byte_perm(table.x, table.y, m_hi) | (byte_perm(w, w4, 0x3726) & 0x80808080u);
}
// A store whose line stays in L2.
__device__ __forceinline__ void st_keep(float *p, float v, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.f32 [%0], %1, %2;" ::"l"(p), "f"(v), "l"(policy) : "memory");
}
// A row's 16 scale bytes to the numbers of their tables; returns the largest of them, NaN bytes aside, in the range that
// the format allows: what becomes e4m3's 2^6.  Sets `low` if some table may be one below kExact.
__device__ __forceinline__ int row_picks(uint32_t (&w)[4], bool &low) {
    uint32_t hi = 0, lo = 0x00FF00FFu;   // two 16-bit maxima and minima
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t even = w[i] & 0x00FF00FFu, odd = byte_perm(w[i], 0u, 0x4341);
        hi = __vmaxu2(hi, __vmaxu2(even, odd));
        lo = __vminu2(lo, __vminu2(even, odd));
    }
    int top = max(hi & 0xFFFFu, hi >> 16);
    const int least = min(lo & 0xFFFFu, lo >> 16);
    low = least < top - (kTop - kExact);
    if (top <= kFp4ScaleMax && least >= max(kFp4ScaleMin, top - kTop)) {   // every group within the tables
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] -= static_cast<uint32_t>(top - kTop) * 0x01010101u;   // no byte borrows
        return top;
    }
    if (top == kFp4ScaleNan) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int X = w[i >> 2] >> (8 * (i & 3)) & 0xFF;
            if (X != kFp4ScaleNan) top = max(top, X);
        }
    }
    top = min(max(top, kFp4ScaleMin), kFp4ScaleMax);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t at = 0;
#pragma unroll 1
        for (int k = 0; k < 32; k += 8) {
            const int X = w[i] >> k & 0xFF, in = min(max(X, kFp4ScaleMin), kFp4ScaleMax);
            at |= static_cast<uint32_t>(X == kFp4ScaleNan ? kNanTable : max(in - top + kTop, 0)) << k;
        }
        w[i] = at;
    }
    return top;
}
// Two fp32 operations in one instruction (sm_100 family).
__device__ __forceinline__ unsigned long long bits2(float2 v) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 floats2(unsigned long long v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return floats2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return floats2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return floats2(r);
}
// Maximum over the warp, NaN aside (-infinity when there is nothing else).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float4 lds4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// One head's query into the N side of S, lane j the latent elements 16j .. 16j + 15.
// Scaled by a power of two that brings its largest magnitude into [128, 256); returns the factor that undoes it (NaN
// for a query that holds a NaN or an infinity).
template <int HP>
__device__ __forceinline__ float store_query(uint32_t q_base, int h, int lane, const uint4 (&v)[2]) {
    using L = Fp4Layout<HP>;
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, max(w[i] << 16 & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
    top = __reduce_max_sync(0xffffffffu, top);
    const int e = f16_range_exponent(__uint_as_float(top)) - 6;
    const float up = exp2_int(e);
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float x0 = __uint_as_float(w[2 * k] << 16) * up, x1 = __uint_as_float(w[2 * k] & 0xFFFF0000u) * up;
        const float x2 = __uint_as_float(w[2 * k + 1] << 16) * up, x3 = __uint_as_float(w[2 * k + 1] & 0xFFFF0000u) * up;
        const uint32_t a = L::kJoin ? split16_e4m3x2(x0, x1) : split_e4m3x2(x0, x1);
        const uint32_t b = L::kJoin ? split16_e4m3x2(x2, x3) : split_e4m3x2(x2, x3);
        hw[k] = byte_perm(a, b, 0x5410);
        lw[k] = byte_perm(a, b, 0x7632);
    }
    const uint32_t slab = q_base + (lane >> 3) * L::kQSlab;
    const int row = L::kJoin ? 2 * (h & ~1) + (h & 1) : h;
    st_shared_v4(slab + sw128_offset(row, lane & 7), hw[0], hw[1], hw[2], hw[3]);
    st_shared_v4(slab + sw128_offset(row + (L::kJoin ? 2 : HP), lane & 7), lw[0], lw[1], lw[2], lw[3]);
    return top >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu) : exp2_int(-e);
}

// mbar_wait that looks at the clock only every 256 tries and leaves the error to the caller: there are many of these, and
// the kernel's loops have to share the instruction cache.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    uint32_t tries = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if ((++tries & 255u) != 0) continue;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > MLA_WAIT_LIMIT_NS) return false;
    }
    return true;
}

// The same for a whole warp, which leaves it together and of one mind (a lane that fell two phases behind the others would
// mistake the barrier's parity).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity));
}
// True in one lane of a warp that is here together: the issuing warps stay converged around their waits and loops, as
// code that the compiler knows to be one lane's takes more instructions (319 -> 305 us at 96 heads, 64 x 16384 rows).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}
// ------------------------------------------------------------------ attention
template <int HP>
__global__ void __launch_bounds__(Fp4Layout<HP>::kThreads, 1)
    fp4_attention_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_scales,
                         const Fp4Params p) {
    using L = Fp4Layout<HP>;
    constexpr bool kJoin = L::kJoin;
    constexpr int HW = L::HW, N = L::N, WC = L::WC, kSlabs = L::kSlabs, kStages = L::kStages, kPBufs = L::kPBufs,
                  kSBufs = L::kSBufs, kPickBufs = L::kPickBufs, kFull = L::kFull;
    constexpr int kSoftWarps = 4 * L::kSoftGroups, kExpWarps = 4 * L::kExpGroups;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - raw);
    Fp4Shared &sh = *reinterpret_cast<Fp4Shared *>(smem + L::END);
    auto bar = [](uint64_t &b) { return smem_u32(&b); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_scales);
        tma_prefetch_desc(&tm_codes);
        for (int i = 0; i < kFull; ++i) mbar_init(bar(sh.stage_full[i]), 1);
        for (int i = 0; i < kStages; ++i) mbar_init(bar(sh.stage_empty[i]), 4);
        for (int i = 0; i < kPickBufs; ++i) {
            mbar_init(bar(sh.scale_full[i]), 1);
            mbar_init(bar(sh.pick_full[i]), 1);
            mbar_init(bar(sh.pick_empty[i]), kExpWarps);
        }
        for (int i = 0; i < kSlabs; ++i) mbar_init(bar(sh.slab_full[i]), 4), mbar_init(bar(sh.slab_free[i]), 1);
        for (int i = 0; i < kSBufs; ++i) mbar_init(bar(sh.s_full[i]), 1), mbar_init(bar(sh.s_free[i]), kSoftWarps);
        for (int i = 0; i < kPBufs; ++i) mbar_init(bar(sh.p_full[i]), kSoftWarps), mbar_init(bar(sh.p_free[i]), 1);
        mbar_init(bar(sh.q_ready), kSoftWarps);
        fence_mbar_init();
    }
    if (threadIdx.x >= 64 && threadIdx.x < 64 + kTables) {   // magnitudes times 2^k as e4m3 bytes
        const int i = threadIdx.x - 64;
        const float f = i == kNanTable ? __uint_as_float(0x7FFFFFFFu)
                                       : (i == 0 || i == kPastTable ? 0.f : exp2_int(i - kTop + 6));
        uint32_t b[4];
        const float m[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = cvt_e4m3x2(m[2 * k] * f, m[2 * k + 1] * f);
        sh.table[i] = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&sh.tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    grid_dependency_wait();     // launched as a programmatic dependent too: nothing before this reads or writes memory
    grid_launch_dependents();   // the merge takes SMs as CTAs finish; it waits for the whole grid

    Walk walk;
    walk.start(p, blockIdx.x, lane, blockIdx.x == 0 && warp == 0 ? p.err : nullptr);
    Segment seg;

    if (warp < 4) {
        regs_release<L::kRegsCtl>();
        if (warp == 0) {
            // ---- a unit's scale bytes to table numbers, in place, and refs; the bytes are asked for three units ahead
            if (lane == 0) p.ws_far[blockIdx.x] = 0;
            Walk far = walk;
            Segment far_seg;
            Units unit, next;
            unit.start(walk, seg);
            next.start(far, far_seg);
            bool ok = true;
            uint32_t asked = 0;
            auto ask = [&] {
                const uint32_t pb = asked % kPickBufs;
                if (asked >= kPickBufs) ok = ok && wait_bar(bar(sh.pick_empty[pb]), (asked / kPickBufs - 1) & 1);
                if (lane == 0) {
                    fence_proxy_async_smem();   // this warp's table numbers were written through the generic proxy
                    mbar_arrive_expect_tx(bar(sh.scale_full[pb]), kPicks);
                    tma_load_3d(base + L::PICK + pb * kPicks, &tm_scales, bar(sh.scale_full[pb]), kR / 2, next.row(far_seg),
                                far_seg.seq);
                }
                ++asked;
                next.next(far, far_seg);
            };
#pragma unroll 1
            for (int i = 0; i < kPickBufs - 1 && next.rows > 0; ++i) ask();
#pragma unroll 1
            for (uint32_t un = 0; unit.rows > 0; ++un) {
                const uint32_t pb = un % kPickBufs;
                ok = ok && wait_bar(bar(sh.scale_full[pb]), (un / kPickBufs) & 1);
                // (the expansion is done with the unit four back, so O is with the unit six back, and the softmax: the
                // ref slot, last used eight back, is free)
                uint4 *const at = reinterpret_cast<uint4 *>(smem + L::PICK + pb * kPicks) + lane;
                bool low = false;
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {   // a lane takes rows lane + 32 i
                    const uint4 v = at[32 * i];
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    bool row_low;
                    const int top = row_picks(w, row_low);
                    const bool real = lane + 32 * i < unit.rows;   // rows past the end: zeros
                    constexpr uint32_t past = kPastTable * 0x01010101u;
                    at[32 * i] = real ? make_uint4(w[0], w[1], w[2], w[3]) : make_uint4(past, past, past, past);
                    sh.ref[un & 7][lane + 32 * i] = static_cast<int16_t>(top - 127 - 6);
                    low |= real && row_low;
                }
                low = __any_sync(0xffffffffu, low);
                if (lane == 0) sh.low[un & 7] = low;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sh.pick_full[pb]));
                unit.next(walk, seg);
                if (next.rows > 0) ask();
            }
            if (!ok) {
                record_error(p.err, kDevErrTimeout);
                // no load may still be landing when the CTA exits
                for (uint32_t k = asked > kPickBufs ? asked - kPickBufs : 0; k < asked; ++k)
                    wait_bar(bar(sh.scale_full[k % kPickBufs]), (k / kPickBufs) & 1);
            }
        } else if (warp == 3) {
            const bool lead = elect_one();
            // ---- TMA: a unit's codes, slab by slab
            const uint64_t once = l2_policy_evict_first();
            uint32_t it = 0;
            bool ok = true;
#pragma unroll 1
            while (ok && walk.next(seg)) {
#pragma unroll 1
                for (int u = 0; ok && u < seg.units; ++u) {
#pragma unroll 1
                    for (int k = 0; k < 4; ++k, ++it) {
                        const uint32_t st = it % kStages;
                        if (it >= kStages &&
                            !(ok = wait_warp(bar(sh.stage_empty[st]), (it / kStages - 1) & 1)))
                            break;
                        if (lead) {
                            const uint32_t full = bar(sh.stage_full[it % kFull]);
                            mbar_arrive_expect_tx(full, kStage);
                            tma_load_3d_hint(base + L::STAGE + st * kStage, &tm_codes, full, k * 64,
                                             seg.row0 + u * kRows, seg.seq, once);
                        }
                    }
                }
            }
            if (!ok && lane == 0) record_error(p.err, kDevErrTimeout);
            {   // this CTA's part of W_UV into L2: the cache's rows have pushed it out
                const uint32_t lines = static_cast<uint32_t>(p.H) * (kDV * kR * 2 / 128);   // of 128 bytes
                const uint32_t from = lines * blockIdx.x / gridDim.x, to = lines * (blockIdx.x + 1) / gridDim.x;
                if (lead && to > from)
                    bulk_prefetch_l2(reinterpret_cast<const uint8_t *>(p.w_uv) + from * 128ull, (to - from) * 128);
            }
            // no load may still be landing when the CTA exits
#pragma unroll 1
            for (uint32_t k = it > kStages ? it - kStages : 0; k < it; ++k)
                wait_bar(bar(sh.stage_full[k % kFull]), (k / kFull) & 1);
        } else if (warp == 1) {
            const bool lead = elect_one();
            // ---- S^T = c . q^T: four slabs of K = 128
            constexpr uint32_t idesc = make_idesc_e4m3(128, N, 0, 0);
            const uint64_t q0 = make_smem_desc(base + L::Q, 16, 1024), c0 = make_smem_desc(base + L::C, 16, 1024);
            uint32_t it = 0, un = 0, ns = 0;
            bool ok = true;
#pragma unroll 1
            while (ok && walk.next(seg)) {
                if (!(ok = wait_warp(bar(sh.q_ready), ns++ & 1))) break;
#pragma unroll 1
                for (int u = 0; ok && u < seg.units; ++u, ++un) {
                    const uint32_t sb = un % kSBufs, d = tmem + L::S_COL + sb * N;
                    if (un >= kSBufs && !(ok = wait_warp(bar(sh.s_free[sb]), (un / kSBufs - 1) & 1)))
                        break;
#pragma unroll 1
                    for (int k = 0; k < 4; ++k, ++it) {
                        const uint32_t sl = it % kSlabs;
                        if (!(ok = wait_warp(bar(sh.slab_full[sl]), (it / kSlabs) & 1))) break;
                        tc_fence_after();
                        const uint64_t a = desc_add(c0, sl * kSlab), b = desc_add(q0, k * L::kQSlab);
                        if (lead) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                umma_f8(d, desc_add(a, kk * 32), desc_add(b, kk * 32), idesc, (k | kk) != 0);
                                if (!kJoin) umma_f8(d, desc_add(a, kk * 32), desc_add(b, L::kQPart + kk * 32), idesc, 1);
                            }
                        }
                    }
                    if (ok && lead) umma_commit(bar(sh.s_full[sb]));
                }
            }
            if (!ok && lane == 0) record_error(p.err, kDevErrTimeout);
        } else if (warp == 2) {
            if (blockIdx.x == 0) write_seq(p, lane);   // its first product is far off
            const bool lead = elect_one();
            // ---- O^T += c^T . P^T: slab t holds latent columns [128 t, 128 t + 128)
            constexpr uint32_t idesc = make_idesc_e4m3(128, N, 1, 1), idesc_lo = idesc | 1u << 10;   // B: e5m2
            const uint64_t p0 = make_smem_desc(base + L::P, kSlab, 1024), c0 = make_smem_desc(base + L::C, kSlab, 1024);
            uint32_t it = 0, un = 0;
            bool ok = true;
#pragma unroll 1
            while (ok && walk.next(seg)) {
#pragma unroll 1
                for (int u = 0; ok && u < seg.units; ++u, ++un) {
                    const uint32_t pb = un % kPBufs;
                    if (!(ok = wait_warp(bar(sh.p_full[pb]), (un / kPBufs) & 1))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int t = 0; t < 4; ++t, ++it) {
                        const uint32_t sl = it % kSlabs, d = tmem + L::O_COL + t * N;
                        if (!(ok = wait_warp(bar(sh.slab_full[sl]), (it / kSlabs) & 1))) break;
                        const uint64_t a = desc_add(c0, sl * kSlab), b = desc_add(p0, pb * L::kPBuf);
                        if (lead) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                umma_f8(d, desc_add(a, kk * 4096), desc_add(b, kk * 4096), idesc, (u | kk) != 0);
                                if (!kJoin)
                                    umma_f8(d, desc_add(a, kk * 4096), desc_add(b, L::kPPart + kk * 4096), idesc_lo, 1);
                            }
                            umma_commit(bar(sh.slab_free[sl]));
                        }
                    }
                    if (ok && lead) umma_commit(bar(sh.p_free[pb]));
                }
            }
            if (!ok && lane == 0) record_error(p.err, kDevErrTimeout);
        }
    } else if (warp < 4 + kSoftWarps) {
        regs_acquire<L::kRegsSoft>();
        // ---- softmax: thread = row `t` of the unit (TMEM lane t), warpgroup `wg` the heads [HW wg, HW wg + HW).  After a
        // failed wait every warp runs its loops to their end, without waiting
        const int sw = warp - 4, wg = sw >> 2, quad = warp & 3, t = quad * 32 + lane, id = 1 + wg;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + wg * WC;
        float *const mul = sh.mul + wg * HW, *const bias = sh.bias[wg], *const step = sh.step[wg], *const fac = sh.fac[wg],
                     *const part = sh.part[sw];
        const float(*const all)[kMaxHW] = sh.part + 4 * wg;
        const int mine = min(HW, p.H - wg * HW);   // real heads of this warpgroup (may be <= 0)
        uint32_t un = 0;
        bool ok = true, more = walk.next(seg);
        size_t done = 0;   // the slot (first row of this warpgroup's heads) of the segment before, to be drained
        float l[HW];
#pragma unroll 1
        for (;;) {
            if (more) {
                // the segment's queries: S of the last unit before this has been read, so the buffer is free, and S of the
                // first one can run while O^T of the segment before is drained
#pragma unroll 1
                for (int i0 = quad; i0 < HW; i0 += 8) {
                    uint4 v[2][2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int h = i0 + 4 * i;
                        const size_t row = static_cast<size_t>(seg.seq) * p.H + (h < mine ? wg * HW + h : 0);
                        const uint4 *src = reinterpret_cast<const uint4 *>(p.q_abs + row * kR) + lane * 2;
                        v[i][0] = h < mine ? __ldg(src) : make_uint4(0, 0, 0, 0);
                        v[i][1] = h < mine ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int h = i0 + 4 * i;
                        const float undo = store_query<HP>(base + L::Q, wg * HW + h, lane, v[i]);
                        if (lane == 0) mul[h] = h < mine ? undo * p.scale_log2 : 0.f;
                    }
                }
                if (quad == 0 && lane < HW)
                    bias[lane] = lane < mine ? kBias : -INFINITY;   // padding heads: P = 0, never a new maximum
                fence_proxy_async_smem();
                named_bar_sync(id, 128);
                if (lane == 0) mbar_arrive(bar(sh.q_ready));
            }
            if (un > 0) {
                // ---- O^T of the segment before (lane = latent column of its tile)
                const uint32_t last = un - 1;
                ok = ok && wait_bar(bar(sh.p_free[last % kPBufs]), (last / kPBufs) & 1);
                __syncwarp();
                tc_fence_after();
                const uint64_t keep = l2_policy_evict_last();   // the merge reads it soon
#pragma unroll 1
                for (int c = 0; c < 4 * (HW / 8); ++c) {
                    const int tile = c / (HW / 8), g = c % (HW / 8) * 8;
                    float *const dst = p.ws_o + (done + g) * kR + tile * 128 + t;
                    float o[kJoin ? 16 : 8];
#pragma unroll
                    for (int i = 0; i < (kJoin ? 16 : 8); i += 8)
                        tmem_ld8(lanes + L::O_COL + tile * N + (kJoin ? 2 * g : g) + i,
                                 *reinterpret_cast<float (*)[8]>(o + i));
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int at = kJoin ? 2 * (k & ~1) + (k & 1) : k;
                        if (g + k < mine)
                            st_keep(dst + static_cast<size_t>(k) * kR,
                                    kJoin ? fmaf(o[(at + 2) % 16], kLoPart, o[at]) : o[at], keep);
                    }
                }
                tc_fence_before();
            }
            if (!more) break;
#pragma unroll
            for (int h = 0; h < HW; ++h) l[h] = 0.f;

#pragma unroll 1
            for (int u = 0; u < seg.units; ++u, ++un) {
                const uint32_t sb = un % kSBufs, pb = un % kPBufs;
                float x[HW], s[WC];
                // one warp asks: tries cost the others their shared-memory accesses
                if (quad == 0) {
                    ok = ok && wait_bar(bar(sh.s_full[sb]), (un / kSBufs) & 1);
                    if (un >= kPBufs) ok = ok && wait_bar(bar(sh.p_free[pb]), (un / kPBufs - 1) & 1);
                    __syncwarp();   // its lanes leave the waits one by one; the barrier takes a whole warp
                }
                named_bar_sync(id, 128);
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < WC; g += 8)
                    tmem_ld8(lanes + L::S_COL + sb * N + g, *reinterpret_cast<float (*)[8]>(s + g));
                const int ref = sh.ref[un & 7][t];
                // a row past the end has an all-zero tile row: its exponents are -infinity
                const float row_scale = exp2_int(ref),
                            row_exp = t < seg.len - seg.row0 - u * kRows ? static_cast<float>(ref) : -INFINITY;
                tmem_wait_ld();
                // x = score * log2 e + ref + kBias - M
                float top = -INFINITY;
                const float2 rs = make_float2(row_scale, row_scale), re = make_float2(row_exp, row_exp);
#pragma unroll
                for (int h = 0; h < HW; h += 4) {
                    const float4 m = lds4(mul + h), bi = lds4(bias + h);
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const float2 mk = k ? make_float2(m.z, m.w) : make_float2(m.x, m.y);
                        const float2 bk = k ? make_float2(bi.z, bi.w) : make_float2(bi.x, bi.y);
                        float2 sc;
                        if constexpr (kJoin) {
                            const int c = 2 * (h + k);
                            sc = fma2(make_float2(s[c + 2], s[c + 3]), make_float2(kLoPart, kLoPart),
                                      make_float2(s[c], s[c + 1]));
                        } else {
                            sc = make_float2(s[h + k], s[h + k + 1]);
                        }
                        const float2 v = fma2(sc, mul2(mk, rs), add2(bk, re));
                        x[h + k] = v.x, x[h + k + 1] = v.y;
                        top = fmaxf(fmaxf(top, v.x), v.y);
                    }
                }
                uint32_t moved = 0;   // heads whose columns of O^T are to be rescaled
                const bool fresh = u % kWindow == 0;   // M is set anew, higher or lower
                if (fresh || named_bar_or(id, 128, top > kBias + kSlack)) {
                    // the maxima over the rows of the heads that a row of this warp pushes past (of all, in a fresh unit):
                    // lane h gets head h's, first of its warp, then of all four
                    // (a short loop that reads S again: this code is seldom in the instruction cache)
                    float most = -INFINITY;
                    if (fresh) {
#pragma unroll 1
                        for (int h0 = 0; h0 < HW; h0 += 8) {
                            constexpr int W = kJoin ? 16 : 8;
                            float y[W];
#pragma unroll
                            for (int i = 0; i < W; i += 8)
                                tmem_ld8(lanes + L::S_COL + sb * N + h0 * (W / 8) + i,
                                         *reinterpret_cast<float (*)[8]>(y + i));
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int c = kJoin ? 2 * (k & ~1) + (k & 1) : k;
                                const float sc = kJoin ? fmaf(y[(c + 2) % W], kLoPart, y[c]) : y[c];
                                const float v = warp_max(fmaf(sc, mul[h0 + k] * row_scale, bias[h0 + k] + row_exp));
                                if (lane == h0 + k) most = v;
                            }
                        }
                    } else {
                        uint32_t past = 0;   // bit HW - 1 - h: head h (the sign of threshold - x)
#pragma unroll
                        for (int h = 0; h < HW; ++h)
                            past = __funnelshift_l(__float_as_uint(kBias + kSlack - x[h]), past, 1);
#pragma unroll 1
                        for (past = __reduce_or_sync(0xffffffffu, past); past; past &= past - 1) {
                            const int h = HW - __ffs(past);
                            float v;
                            if constexpr (kJoin) {
                                float lo;
                                tmem_ld1(lanes + L::S_COL + sb * N + 2 * (h & ~1) + (h & 1), v);
                                tmem_ld1(lanes + L::S_COL + sb * N + 2 * (h & ~1) + (h & 1) + 2, lo);
                                tmem_wait_ld();
                                v = fmaf(lo, kLoPart, v);
                            } else {
                                tmem_ld1(lanes + L::S_COL + sb * N + h, v);
                                tmem_wait_ld();
                            }
                            v = warp_max(fmaf(v, mul[h] * row_scale, bias[h] + row_exp));
                            if (lane == h) most = v;
                        }
                    }
                    if (lane < HW) part[lane] = most;
                    named_bar_sync(id, 128);
                    bool moves = false;
                    if (lane < HW) {
                        most = fmaxf(fmaxf(all[0][lane], all[1][lane]), fmaxf(all[2][lane], all[3][lane]));
                        moves = (most > kBias + kSlack || fresh) && most > -INFINITY;
                        if (quad == 0) {
                            float by = moves ? kBias - kHead - most : 0.f;   // M_old - M_new
                            if (u > 0) by = fminf(by, kDrop);
                            step[lane] = by;
                            fac[lane] = fast_exp2(by);
                            bias[lane] += by;
                        }
                    }
                    moved = u > 0 ? __ballot_sync(0xffffffffu, moves) : 0u;
                    named_bar_sync(id, 128);
#pragma unroll
                    for (int h = 0; h < HW; h += 4) {
                        const float4 by = lds4(step + h);
                        const float2 a = add2(make_float2(x[h], x[h + 1]), make_float2(by.x, by.y));
                        const float2 b = add2(make_float2(x[h + 2], x[h + 3]), make_float2(by.z, by.w));
                        x[h] = a.x, x[h + 1] = a.y, x[h + 2] = b.x, x[h + 3] = b.y;
                    }
                    if (u > 0) {
#pragma unroll
                        for (int h = 0; h < HW; h += 4) {
                            const float4 f = lds4(fac + h);
                            const float2 a = mul2(make_float2(l[h], l[h + 1]), make_float2(f.x, f.y));
                            const float2 b = mul2(make_float2(l[h + 2], l[h + 3]), make_float2(f.z, f.w));
                            l[h] = a.x, l[h + 1] = a.y, l[h + 2] = b.x, l[h + 3] = b.y;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sh.s_free[sb]));
                // weights, their sums, and P^T as the MN-major N side: row t, the bytes of this warpgroup's columns
                const float2 unref = make_float2(exp2_int(-ref), exp2_int(-ref));
                uint32_t w[HW / 2];   // kJoin: two heads' hi and lo; else HW / 4 words of hi, then of lo
#pragma unroll
                for (int h = 0; h < HW; h += 4) {
                    const float2 p01 = make_float2(fast_exp2(x[h]), fast_exp2(x[h + 1]));
                    const float2 p23 = make_float2(fast_exp2(x[h + 2]), fast_exp2(x[h + 3]));
                    const float2 l01 = fma2(p01, unref, make_float2(l[h], l[h + 1]));
                    const float2 l23 = fma2(p23, unref, make_float2(l[h + 2], l[h + 3]));
                    l[h] = l01.x, l[h + 1] = l01.y, l[h + 2] = l23.x, l[h + 3] = l23.y;
                    if constexpr (kJoin) {
                        w[h / 2] = split16_e4m3x2(p01.x, p01.y);
                        w[h / 2 + 1] = split16_e4m3x2(p23.x, p23.y);
                    } else {
                        const uint32_t y = split_e4m3_e5m2x2(p01.x, p01.y), z = split_e4m3_e5m2x2(p23.x, p23.y);
                        w[h / 4] = byte_perm(y, z, 0x5410);
                        w[HW / 4 + h / 4] = byte_perm(y, z, 0x7632);
                    }
                }
                const uint32_t prow = base + L::P + pb * L::kPBuf;
                if constexpr (kJoin) {
#pragma unroll
                    for (int i = 0; i < HW / 8; ++i)
                        st_shared_v4(prow + sw128_offset(t, wg * (HW / 8) + i), w[4 * i], w[4 * i + 1], w[4 * i + 2],
                                     w[4 * i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < HW / 8; ++i) {   // HW = 24 leaves 8-byte pieces
                        const int piece = wg * (HW / 8) + i;
                        const uint32_t at = prow + sw128_offset(t, piece >> 1) + 8 * (piece & 1);
                        st_shared_v2(at, w[2 * i], w[2 * i + 1]);
                        st_shared_v2(at + L::kPPart, w[HW / 4 + 2 * i], w[HW / 4 + 2 * i + 1]);
                    }
                }
                if (moved) {   // once the products of the unit before are complete
                    ok = ok && wait_bar(bar(sh.p_free[(un - 1) % kPBufs]), ((un - 1) / kPBufs) & 1);
                    __syncwarp();
                    tc_fence_after();
                    // four columns at a time, of all the heads that they hold (a factor of one for those that did not move):
                    // a head on its own would load columns that its neighbour's store has not reached yet, as only
                    // wait::st orders a store before a later load
                    constexpr int kQuad = kJoin ? 2 : 4;   // heads of four columns
#pragma unroll 1
                    while (moved) {
                        const int h = (__ffs(moved) - 1) & ~(kQuad - 1), col = kJoin ? 2 * h : h;
                        moved &= ~(((1u << kQuad) - 1u) << h);
                        float f[kQuad], o[4][4];   // of the four latent tiles
#pragma unroll
                        for (int i = 0; i < kQuad; ++i) f[i] = fac[h + i];
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld4(lanes + L::O_COL + c * N + col, o[c]);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[c][i] *= f[i % kQuad];
                            tmem_st4(lanes + L::O_COL + c * N + col, o[c]);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sh.p_full[pb]));
            }
            // ---- the segment's maxima, and l over the 128 rows
            // (every step halves the heads that a lane holds, so that lane h ends with head h's sum over the warp)
            {
                constexpr int P = HW <= 8 ? 8 : (HW <= 16 ? 16 : 32);
                float v[P];
#pragma unroll
                for (int h = 0; h < P; ++h) v[h] = h < HW ? l[h] : 0.f;
#pragma unroll
                for (int o = P / 2; o >= 1; o >>= 1) {
                    const bool up = lane & o;
#pragma unroll
                    for (int i = 0; i < o; ++i) {
                        const float send = up ? v[i] : v[i + o];
                        v[i] = (up ? v[i + o] : v[i]) + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                }
#pragma unroll
                for (int o = 16; o >= P; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                if (lane < HW) part[lane] = v[0];
            }
            named_bar_sync(id, 128);   // also: every warp is done with mul and bias
            done = static_cast<size_t>(seg.slot) * p.H + wg * HW;
            if (t < mine) {   // (mine <= 24: the warpgroup's first warp)
                p.ws_m[done + t] = -bias[t];
                p.ws_l[done + t] = (all[0][t] + all[1][t]) + (all[2][t] + all[3][t]);
            }
            more = walk.next(seg);
        }
        if (!ok && lane == 0) record_error(p.err, kDevErrTimeout);
    } else {
        regs_release<L::kRegsExp>();
        // ---- expansion: a warpgroup takes every other slab, a warp 32 of its rows, a lane the groups (32 codes) `g` of
        // rows r + 8 i
        constexpr int kBatch = kJoin ? 4 : 2;   // by the registers there are
        const int first = (warp - 4 - kSoftWarps) >> 2, g = lane & 3, r = (warp & 3) * 32 + (lane >> 2);
        const int x = ((2 * g) ^ (lane >> 2)) * 16;   // row & 7 = lane >> 2: the swizzle of the group's first 16 bytes
        const uint32_t slab_at = L::C + sw128_offset(r, 0) - (lane >> 2) * 16, pick_at = L::PICK + r * 16 + g,
                       stage_at = L::STAGE + r * 64 + g * 16;
        bool ok = true;
        uint32_t un = 0;
#pragma unroll 1
        while (walk.next(seg)) {
#pragma unroll 1
            for (int u = 0; u < seg.units; ++u, ++un) {
                const uint32_t pb = un % kPickBufs;
                ok = ok && wait_bar(bar(sh.pick_full[pb]), (un / kPickBufs) & 1);
                const bool low = sh.low[un & 7];
#pragma unroll 1
                for (int k = first; k < 4; k += L::kExpGroups) {
                    const uint32_t it = 4 * un + k, sl = it % kSlabs, st = it % kStages;
                    ok = ok && wait_bar(bar(sh.stage_full[it % kFull]), (it / kFull) & 1);
                    // the codes wait for their slab in registers: the stage can take the next ones meanwhile
                    uint4 c[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        c[i] = *reinterpret_cast<const uint4 *>(smem + stage_at + st * kStage + i * 512);
                    if (__builtin_expect(low, 0)) {
                        // groups of zeros may lie anywhere below their row's largest, others make the merge do the share again
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(smem + stage_at + st * kStage + i * 512);
                            if (smem[pick_at + pb * kPicks + i * 128 + k * 4] < kExact &&
                                ((w.x | w.y | w.z | w.w) & 0x77777777u))
                                p.ws_far[blockIdx.x] = 1;   // (after warp 0's zero: pick_full lies between)
                        }
                    }
                    fence_proxy_async_smem();   // the reads, before TMA writes there again
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(sh.stage_empty[st]));
                    if (it >= kSlabs) ok = ok && wait_bar(bar(sh.slab_free[sl]), (it / kSlabs - 1) & 1);
                    uint8_t *const slab = smem + slab_at + sl * kSlab;
#pragma unroll
                    for (int h = 0; h < 4; h += kBatch) {
                        uint2 tb[kBatch];   // read before the stores
#pragma unroll
                        for (int i = 0; i < kBatch; ++i)
                            tb[i] = sh.table[smem[pick_at + pb * kPicks + (h + i) * 128 + k * 4]];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const uint4 w = c[h + i];
                            uint32_t o[8];
                            expand8(w.x, tb[i], o[0], o[1]);
                            expand8(w.y, tb[i], o[2], o[3]);
                            expand8(w.z, tb[i], o[4], o[5]);
                            expand8(w.w, tb[i], o[6], o[7]);
                            uint8_t *const to = slab + (h + i) * 1024;
                            *reinterpret_cast<uint4 *>(to + x) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4 *>(to + (x ^ 16)) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(sh.slab_full[sl]));
                        if (k >= 2) mbar_arrive(bar(sh.pick_empty[pb]));
                    }
                }
            }
        }
        if (!ok && lane == 0) record_error(p.err, kDevErrTimeout);
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ merge
struct MergeParams {
    const int *lens;
    const int2 *ws_seq;
    const int *ws_share, *ws_far;
    float *ws_o, *ws_m, *ws_l;
    const __nv_bfloat16 *w_uv, *gate;
    __nv_bfloat16 *out;
    int *err;
    int B, H, max_len, G;
    const __nv_bfloat16 *q_abs;   // for the shares that are done again
    const uint8_t *c4_cache;
    long long ld_cache;
    float scale_log2;
};

constexpr int kMaxShares = 512;   // share boundaries that the merge keeps in shared memory

// A segment with rows that e4m3 cannot hold (groups more than 2^14 below their row's largest), for one head by one warp:
// fp32 from the codes, one row after the other, into ws_o, ws_m and ws_l.
__device__ __forceinline__ void exact_segment(const __nv_bfloat16 *q, const uint8_t *rows, long long ld, int n,
                                              float scale_log2, float *to_o, float *to_m, float *to_l) {
    const int lane = threadIdx.x & 31;   // columns 16 lane .. 16 lane + 15
    const uint4 *src = reinterpret_cast<const uint4 *>(q) + lane * 2;
    const uint4 q0 = __ldg(src), q1 = __ldg(src + 1);
    const uint32_t qw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
    float o[16], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
    uint2 codes = __ldg(reinterpret_cast<const uint2 *>(rows) + lane);
    int X = __ldg(rows + kR / 2 + (lane >> 1));
#pragma unroll 1
    for (int u = 0; u < n; ++u) {
        const float by = fp4_scale(X);
        const uint32_t w[2] = {codes.x, codes.y};
        if (u + 1 < n) {   // the next row, meanwhile
            rows += ld;
            codes = __ldg(reinterpret_cast<const uint2 *>(rows) + lane);
            X = __ldg(rows + kR / 2 + (lane >> 1));
        }
        float c[16], s = 0.f;
        unpack_e2m1x8(w[0], *reinterpret_cast<float (*)[8]>(c));
        unpack_e2m1x8(w[1], *reinterpret_cast<float (*)[8]>(c + 8));
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            c[k] *= by;
            s = fmaf(c[k], __uint_as_float(k & 1 ? qw[k / 2] & 0xFFFF0000u : qw[k / 2] << 16), s);
        }
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= scale_log2;
        const float top = fmaxf(m, s), f = fast_exp2(m - top), p = fast_exp2(s - top);
        m = top;
        l = fmaf(l, f, p);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = fmaf(o[k], f, p * c[k]);
    }
#pragma unroll
    for (int k = 0; k < 16; k += 4)
        *reinterpret_cast<float4 *>(to_o + lane * 16 + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
    if (lane == 0) *to_m = m, *to_l = l;
    __syncwarp();
}

// A sequence whose first unit is r0: where its last one ends, and the share that holds the first.
__device__ __forceinline__ int end_of(int r0, int len) {
    const int more = chunks_of(len) - 1;
    return r0 + more * (kOver + kChunkUnits) + (len - more * kChunkRows + kRows - 1) / kRows;
}
__device__ __forceinline__ int first_share(const MergeParams &p, const int *shares, int r0) {
    // from an estimate on, as shares are equal but for a unit
    int c = min(p.G - 1, static_cast<int>(static_cast<float>(r0) * p.G / shares[p.G]));
    while (c > 0 && shares[c] > r0) --c;
    while (c + 1 < p.G && shares[c + 1] <= r0) ++c;
    return c;
}
// A sequence's segments in shares with such rows, for one head by one warp: of the shares that join_segments takes there.
__device__ __noinline__ void finish_segments(const MergeParams &p, const int *shares, int b, int h, int len, int sub,
                                             int per) {
    if (len <= 0) return;
    const int2 at = p.ws_seq[b];
    const int span = kOver + kChunkUnits, r0 = at.x + kOver, end = end_of(r0, len);
    for (int c = first_share(p, shares, r0) + sub; c < p.G && shares[c] < end; c += per) {
        if (p.ws_far[c] == 0) continue;
        const int lo = max(shares[c], r0), hi = min(shares[c + 1], end);
        for (int j = (lo - at.x) / span, base; (base = r0 + j * span) < hi; ++j) {   // base: the chunk's first unit
            const int u0 = max(lo, base) - base, u1 = min(hi - base, kChunkUnits), row0 = j * kChunkRows + u0 * kRows;
            const size_t slot = static_cast<size_t>(c + at.y + j) * p.H + h;
            if (u1 <= u0) continue;
            exact_segment(p.q_abs + (static_cast<size_t>(b) * p.H + h) * kR,
                          p.c4_cache + (static_cast<long long>(b) * p.max_len + row0) * p.ld_cache, p.ld_cache,
                          min(len - row0, (u1 - u0) * kRows), p.scale_log2, p.ws_o + slot * kR, p.ws_m + slot,
                          p.ws_l + slot);
        }
    }
}

// Log-sum-exp join of a sequence's segments for one head by one warp, which takes every `per`-th share of the axis from
// the `sub`-th on, all chunks' segments together (one chunk after the other waits once for each: 59 against 53 us for one
// sequence of 131000 rows): o = sum of 2^(m - M) ws_o in the lane's columns 4 lane + 128 q, L = sum of 2^(m - M) l.
template <int kFly>   // segments whose rows are in flight at a time
__device__ __forceinline__ void join_segments(const MergeParams &p, const int *shares, int2 at, int h, int len, int sub,
                                              int per, int lane, float (&o)[16], float &M, float &L) {
    M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
    if (len <= 0) return;
    const int span = kOver + kChunkUnits, r0 = at.x + kOver, end = end_of(r0, len), c_first = first_share(p, shares, r0);
    for (int c0 = c_first + sub; c0 < p.G && shares[c0] < end; c0 += 32 * per) {
        // a lane takes a share, and one after the other the chunks j that it has rows of (mostly one or two)
        const int c = c0 + lane * per;
        const bool in = c < p.G && shares[min(c, p.G)] < end;
        const int lo = in ? max(shares[c], r0) : 0, hi = in ? min(shares[c + 1], end) : 0;
        const int j0 = (lo - at.x) / span, turns = hi > lo ? (hi - 1 - at.x) / span - j0 + 1 : 0;
        for (int turn = 0, most = __reduce_max_sync(0xffffffffu, turns); turn < most; ++turn) {
            const int j = j0 + turn;
            const bool has = turn < turns && hi > max(lo, r0 + j * span);   // (between two chunks lie the kOver units)
            const size_t slot = static_cast<size_t>(c + at.y + j) * p.H + h;
            const float m = has ? p.ws_m[slot] : -INFINITY, l = has ? p.ws_l[slot] : 0.f;
            float w = 0.f;
            bool first = true;
            for (unsigned left = __ballot_sync(0xffffffffu, has); left;) {
                float4 v[kFly][4];
                int from[kFly];
#pragma unroll
                for (int i = 0; i < kFly; ++i) {
                    from[i] = left ? __ffs(left) - 1 : -1;
                    left &= left - 1;
                    const size_t row = __shfl_sync(0xffffffffu, slot, max(from[i], 0));
                    const float4 *src = reinterpret_cast<const float4 *>(p.ws_o + row * kR) + lane;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[i][q] = from[i] >= 0 ? src[32 * q] : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (first) {   // the weights, once the rows are on their way
                    first = false;
                    const float top = fmaxf(M, warp_max(m)), f = M == -INFINITY ? 0.f : fast_exp2(M - top);
                    w = has ? fast_exp2(m - top) : 0.f;
                    float s = has ? w * l : 0.f;
#pragma unroll
                    for (int q = 16; q >= 1; q >>= 1) s += __shfl_xor_sync(0xffffffffu, s, q);
                    L = L * f + s;
                    M = top;
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] *= f;
                }
#pragma unroll
                for (int i = 0; i < kFly; ++i) {
                    const float wi = __shfl_sync(0xffffffffu, w, max(from[i], 0));
                    if (from[i] < 0) continue;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[4 * q] = fmaf(wi, v[i][q].x, o[4 * q]);
                        o[4 * q + 1] = fmaf(wi, v[i][q].y, o[4 * q + 1]);
                        o[4 * q + 2] = fmaf(wi, v[i][q].z, o[4 * q + 2]);
                        o[4 * q + 3] = fmaf(wi, v[i][q].w, o[4 * q + 3]);
                    }
                }
            }
        }
    }
}
__device__ __forceinline__ float gated(const __nv_bfloat16 *gate, size_t at, float y) {
    return gate ? y * __fdividef(1.f, 1.f + fast_exp2(-__bfloat162float(gate[at]) * kLog2e)) : y;
}

// Few (head, sequence) pairs: a CTA per head and kSeqs sequences, fp32 products.  W_UV[h] (128 KB, contiguous) is asked
// into shared memory before the attention is done; 16 / kSeqs warps join a sequence's segments, then a warp takes eight
// rows of W_UV, a lane 16 columns of each.
constexpr int kDotThreads = 512;
constexpr uint32_t kDotW = kDV * kR * 2, kDotPart = 16 * kR * 4;
template <int kSeqs>
constexpr uint32_t kDotSmem = kDotW + kDotPart + kSeqs * kR * 4;
template <int kSeqs>
__global__ void __launch_bounds__(kDotThreads, 1) fp4_merge_dot_kernel(const __grid_constant__ MergeParams p) {
    constexpr int kPer = 16 / kSeqs;
    extern __shared__ __align__(128) uint8_t dot_smem[];
    float(*const s_part)[kR] = reinterpret_cast<float(*)[kR]>(dot_smem + kDotW);
    float(*const s_lat)[kR] = reinterpret_cast<float(*)[kR]>(dot_smem + kDotW + kDotPart);
    __shared__ float s_m[16], s_l[16];
    __shared__ int s_shares[kMaxShares + 1];
    __shared__ uint64_t w_full;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x, b0 = static_cast<int>(blockIdx.y) * kSeqs, nb = min(kSeqs, p.B - b0);
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&w_full), 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(smem_u32(&w_full), kDotW);
        bulk_load(smem_u32(dot_smem), p.w_uv + static_cast<size_t>(h) * kDV * kR, kDotW, smem_u32(&w_full));
    }
    const int i = warp / kPer, b = b0 + min(i, nb - 1), len = i < nb ? read_len(p.lens, b, p.max_len, nullptr) : 0;
    grid_dependency_wait();   // the segments are complete and visible after this
    bool far = false;
    for (int c = threadIdx.x; c <= p.G; c += kDotThreads) s_shares[c] = p.ws_share[c], far |= c < p.G && p.ws_far[c];
    const int2 at = p.ws_seq[b];
    if (__syncthreads_or(far)) finish_segments(p, s_shares, b, h, len, warp % kPer, kPer);
    {
        float o[16], M, L;
        join_segments<4>(p, s_shares, at, h, len, warp % kPer, kPer, lane, o, M, L);
        float4 *mine = reinterpret_cast<float4 *>(s_part[warp]) + lane;
#pragma unroll
        for (int q = 0; q < 4; ++q) mine[32 * q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        if (lane == 0) s_m[warp] = M, s_l[warp] = L;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSeqs; ++s) {
        float M = -INFINITY, L = 0.f, x = 0.f;
#pragma unroll
        for (int q = 0; q < kPer; ++q) M = fmaxf(M, s_m[s * kPer + q]);
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const float m = s_m[s * kPer + q], f = m == -INFINITY ? 0.f : fast_exp2(m - M);
            L = fmaf(f, s_l[s * kPer + q], L);
            x = fmaf(f, s_part[s * kPer + q][threadIdx.x], x);   // (a warp without a segment holds zeros)
        }
        s_lat[s][threadIdx.x] = M == -INFINITY ? 0.f : x / L;    // (an empty sequence has none)
    }
    bool ok = mbar_wait(smem_u32(&w_full), 0, p.err);
    __syncthreads();
    float y[kSeqs][8];
    {
        float2 lat[kSeqs][8];
#pragma unroll
        for (int s = 0; s < kSeqs; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k) {   // lane: columns 8 lane .. and 256 + 8 lane ..
                const float4 v = *reinterpret_cast<const float4 *>(&s_lat[s][(k >> 1) * 256 + lane * 8 + (k & 1) * 4]);
                lat[s][2 * k] = make_float2(v.x, v.y), lat[s][2 * k + 1] = make_float2(v.z, v.w);
            }
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            const uint4 *row = reinterpret_cast<const uint4 *>(dot_smem) + (warp * 8 + v) * (kR / 8) + lane;
            const uint4 w0 = row[0], w1 = row[32];
            const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            float2 acc[kSeqs];
#pragma unroll
            for (int s = 0; s < kSeqs; ++s) acc[s] = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 wk = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
#pragma unroll
                for (int s = 0; s < kSeqs; ++s) acc[s] = fma2(wk, lat[s][k], acc[s]);
            }
#pragma unroll
            for (int s = 0; s < kSeqs; ++s) y[s][v] = acc[s].x + acc[s].y;
        }
    }
#pragma unroll
    for (int s = 0; s < kSeqs; ++s) {
        // eight sums over the warp: halve the number of values held with each of the first three exchanges
#pragma unroll
        for (int k = 4; k >= 1; k >>= 1) {
            const bool up = lane & k;
#pragma unroll
            for (int v = 0; v < k; ++v) {
                const float keep = up ? y[s][v + k] : y[s][v], give = up ? y[s][v] : y[s][v + k];
                y[s][v] = keep + __shfl_xor_sync(0xffffffffu, give, k);
            }
        }
        y[s][0] += __shfl_xor_sync(0xffffffffu, y[s][0], 8);
        y[s][0] += __shfl_xor_sync(0xffffffffu, y[s][0], 16);
        if (lane < 8 && s < nb && ok) {   // lane v: output column 8 warp + v
            const size_t to = (static_cast<size_t>(b0 + s) * p.H + h) * kDV + warp * 8 + lane;
            p.out[to] = __float2bfloat16(gated(p.gate, to, y[s][0]));
        }
    }
}

// Many: a CTA per head and 32 sequences; o_lat as bf16 hi + lo, the product on the tensor cores.
constexpr int kMRows = 32;
constexpr int kMergeThreads = 512;
constexpr uint32_t kOSlab = 2 * kMRows * 128;       // o_lat [hi rows | lo rows] x 64 latent columns, bf16
constexpr uint32_t kWSlab = kDV * 128;              // W_UV[h] [128 x 64 latent columns]
constexpr int kWStages = 2;
constexpr uint32_t MW_OFF = 8 * kOSlab, MBAR_OFF = MW_OFF + kWStages * kWSlab;
constexpr uint32_t kSmemMerge = MBAR_OFF + 128 + 1024;

__global__ void __launch_bounds__(kMergeThreads, 2)
    fp4_merge_kernel(const __grid_constant__ CUtensorMap tm_wuv, const __grid_constant__ MergeParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint64_t *w_full = reinterpret_cast<uint64_t *>(smem_raw + (base - raw) + MBAR_OFF), *w_empty = w_full + kWStages,
             *done = w_empty + kWStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    __shared__ int s_shares[kMaxShares + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (sequences along x: the grid's other dimensions end at 65535)
    const int h = blockIdx.y, b0 = static_cast<int>(blockIdx.x) * kMRows, nb = min(kMRows, p.B - b0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kWStages + 1; ++i) mbar_init(smem_u32(w_full + i), 1);
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
    auto load_w = [&](int k) {   // latent columns [64 k, 64 k + 64) of W_UV[h]
        const uint32_t b = smem_u32(w_full + k % kWStages);
        mbar_arrive_expect_tx(b, kWSlab);
        tma_load_2d(base + MW_OFF + (k % kWStages) * kWSlab, &tm_wuv, b, k * 64, h * kDV);
    };
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_wuv);
        for (int k = 0; k < kWStages; ++k) load_w(k);
        for (int k = kWStages; k < 8; ++k) tma_prefetch_l2_2d(&tm_wuv, k * 64, h * kDV);
    }
    // launched as a programmatic dependent: what is above overlaps the attention's tail, its segments are complete
    // and visible after this
    grid_dependency_wait();

    bool far = false;
    for (int c = threadIdx.x; c <= p.G; c += kMergeThreads) s_shares[c] = p.ws_share[c], far |= c < p.G && p.ws_far[c];
    if (__syncthreads_or(far))
        for (int i = warp; i < nb; i += kMergeThreads / 32)
            finish_segments(p, s_shares, b0 + i, h, read_len(p.lens, b0 + i, p.max_len, nullptr), 0, 1);
    for (int i = warp; i < nb; i += kMergeThreads / 32) {
        const int len = read_len(p.lens, b0 + i, p.max_len, nullptr);
        float o[16], M, L;
        join_segments<2>(p, s_shares, p.ws_seq[b0 + i], h, len, 0, 1, lane, o, M, L);
        const float mul = len > 0 ? 1.f / L : 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // row i of the o_lat tile, hi and lo parts
            float y[4], z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[k] = o[4 * q + k] * mul;
                z[k] = y[k] - __bfloat162float(__float2bfloat16(y[k]));
            }
            const uint32_t at = base + (2 * q + (lane >> 4)) * kOSlab + 8 * (lane & 1), ch = (lane & 15) >> 1;
            st_shared_v2(at + sw128_offset(i, ch), pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            st_shared_v2(at + sw128_offset(kMRows + i, ch), pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        // [128 x hi | lo rows] = W_UV[h] . o_lat^T over eight 64-column slabs of the latent
        constexpr uint32_t idesc = make_idesc_bf16(kDV, 2 * kMRows, 0, 0);
        tc_fence_after();
        bool ok = true;
        int loaded = kWStages;
        for (int k = 0; ok && k < 8; ++k) {
            const int st = k % kWStages;
            if (!(ok = mbar_wait(smem_u32(w_full + st), (k / kWStages) & 1, p.err))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                umma_bf16(tmem, make_smem_desc(base + MW_OFF + st * kWSlab + kk * 32, 16, 1024),
                          make_smem_desc(base + k * kOSlab + kk * 32, 16, 1024), idesc, (k | kk) != 0);
            umma_commit(smem_u32(w_empty + st));
            if (k + kWStages < 8) {
                if (!(ok = mbar_wait(smem_u32(w_empty + st), (k / kWStages) & 1, p.err))) break;
                load_w(k + kWStages);
                ++loaded;
            }
        }
        if (ok) umma_commit(smem_u32(done));
        if (!ok)   // no load may still be landing when the CTA exits
            for (int k = 0; k < loaded; ++k) mbar_wait(smem_u32(w_full + k % kWStages), (k / kWStages) & 1, p.err);
    }
    __syncwarp();
    const bool ok = mbar_wait(smem_u32(done), 0, p.err);
    tc_fence_after();
    if (warp < 8 && __all_sync(0xffffffffu, ok)) {   // warp: output column 32 (warp & 3) + lane, rows 16 (warp >> 2) ..
        const int v = (warp & 3) * 32 + lane, i0 = (warp >> 2) * 16;
        const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + i0;
        float hi[16], lo[16];
        tmem_ld16(at, hi);
        tmem_ld16(at + kMRows, lo);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if (i0 + k >= nb) break;
            const size_t off = (static_cast<size_t>(b0 + i0 + k) * p.H + h) * kDV + v;
            p.out[off] = __float2bfloat16(gated(p.gate, off, hi[k] + lo[k]));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 64);
}

// ------------------------------------------------------------------ host
CUresult encode_map(CUtensorMap *m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void *ptr, int rank,
                    const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
    auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
    if (!fn) return CUDA_ERROR_NOT_SUPPORTED;
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, type, rank, const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

size_t slot_count(int B, int max_len, int G) {
    return static_cast<size_t>(G) + static_cast<size_t>(B) * (max_len > 0 ? chunks_of(max_len) : 0);
}

// Runs f, which sets a kernel's attributes, the first time on each device (a call's host time counts in small decodes).
template <typename F>
cudaError_t first_time(std::atomic<unsigned long long> &done, F f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    if ((e = f()) == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <int HP>
cudaError_t launch_attention(const CUtensorMap &codes, const CUtensorMap &scales, const Fp4Params &p, cudaStream_t s) {
    using L = Fp4Layout<HP>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = first_time(done, [] {
        cudaFuncAttributes fa;   // the kernel's register split assumes this launch budget
        const cudaError_t e = cudaFuncGetAttributes(&fa, fp4_attention_kernel<HP>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != static_cast<int>(L::kRegsLaunch)) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(fp4_attention_kernel<HP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(L::kSmem));
    });
    if (e != cudaSuccess) return e;
    note_launch();
    return launch_dependent(fp4_attention_kernel<HP>, dim3(p.G), L::kThreads, L::kSmem, s, codes, scales, p);
}

template <int kSeqs>
cudaError_t launch_dot(const MergeParams &mp, cudaLaunchConfig_t &cfg) {
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = first_time(done, [] {
        return cudaFuncSetAttribute(fp4_merge_dot_kernel<kSeqs>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kDotSmem<kSeqs>));
    });
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(mp.H, (mp.B + kSeqs - 1) / kSeqs);
    cfg.blockDim = dim3(kDotThreads);
    cfg.dynamicSmemBytes = kDotSmem<kSeqs>;
    return cudaLaunchKernelEx(&cfg, fp4_merge_dot_kernel<kSeqs>, mp);
}

}  // namespace

size_t decode_fp4_workspace_bytes(int B, int H, int max_len, int num_sms) {
    return static_cast<size_t>(B) * sizeof(int2) + (2 * num_sms + 1) * sizeof(int) + 8 +
           slot_count(B, max_len, num_sms) * H * (kR + 2) * sizeof(float);
}

cudaError_t launch_decode_fp4(const DecodeArgs &a, cudaStream_t s) {
    if (!decode_bf16_supports(a.H, a.d_v, a.r)) return cudaErrorInvalidValue;
    if (a.num_sms > kMaxShares) return cudaErrorInvalidConfiguration;
    Fp4Params p;
    p.q_abs = static_cast<const __nv_bfloat16 *>(a.q_abs);
    p.lens = a.lens;
    p.B = a.B;
    p.H = a.H;
    p.max_len = a.max_len;
    p.G = a.num_sms;
    const size_t slots = slot_count(a.B, a.max_len, p.G);
    if (decode_fp4_workspace_bytes(a.B, a.H, a.max_len, a.num_sms) > a.workspace_bytes) return cudaErrorInvalidValue;
    p.ws_o = static_cast<float *>(a.workspace);
    p.ws_m = p.ws_o + slots * a.H * kR;
    p.ws_l = p.ws_m + slots * a.H;
    const uintptr_t seq = reinterpret_cast<uintptr_t>(p.ws_l + slots * a.H);
    p.ws_seq = reinterpret_cast<int2 *>((seq + 7) & ~static_cast<uintptr_t>(7));
    p.ws_share = reinterpret_cast<int *>(p.ws_seq + a.B);
    p.ws_far = p.ws_share + p.G + 1;
    p.w_uv = static_cast<const __nv_bfloat16 *>(a.w_uv);
    p.err = a.dev_err;
    p.scale_log2 = a.scale * kLog2e;
    CUtensorMap tm_codes, tm_scales;
    {
        const cuuint64_t rows = static_cast<cuuint64_t>(a.max_len > 0 ? a.max_len : 1);
        const cuuint64_t dims[3] = {kR / 2 + kR / 32, rows, static_cast<cuuint64_t>(a.B)};
        const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.ld_cache), rows * static_cast<cuuint64_t>(a.ld_cache)};
        const cuuint32_t box[3] = {64, kRows, 1}, sbox[3] = {16, kRows, 1};
        const void *rows_at = a.c_cache ? a.c_cache : a.q_abs;   // an empty cache: the maps are not used
        if (encode_map(&tm_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE, rows_at, 3, dims, strides,
                       box) != CUDA_SUCCESS ||
            encode_map(&tm_scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE, rows_at, 3, dims, strides,
                       sbox) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    cudaError_t e = a.H <= 16   ? launch_attention<16>(tm_codes, tm_scales, p, s)
                    : a.H <= 32 ? launch_attention<32>(tm_codes, tm_scales, p, s)
                    : a.H <= 48 ? launch_attention<48>(tm_codes, tm_scales, p, s)
                    : a.H <= 64 ? launch_attention<64>(tm_codes, tm_scales, p, s)
                                : launch_attention<96>(tm_codes, tm_scales, p, s);
    if (e != cudaSuccess) return e;
    const MergeParams mp{a.lens, p.ws_seq, p.ws_share, p.ws_far, p.ws_o, p.ws_m, p.ws_l, p.w_uv,
                         static_cast<const __nv_bfloat16 *>(a.gate), static_cast<__nv_bfloat16 *>(a.out), a.dev_err, a.B,
                         a.H, a.max_len, p.G, p.q_abs, static_cast<const uint8_t *>(a.c_cache), a.ld_cache,
                         p.scale_log2};
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    note_launch();
    // Up to four sequences per CTA, as long as one wave of CTAs (two, of the largest) takes them all.  Whole decodes of 300
    // rows: 16 heads x 16 sequences 17.1 / 14.7 / 15.9 / 18.5 us with one, two, four per CTA and the tensor cores, x 64
    // 37.5 / 30.4 / 25.9 / 27.8, x 96 49.7 / 38.2 / 32.2 / 29.4; 96 heads x 1 20.9 / 21.6 / 23.2 / 24.8 (of 100000 rows,
    // chunk by chunk, 55 / 57 / 59 / 97: there a pair's segments are spread over sixteen warps), x 64 156 / 109 / 87 / 41.
    const auto ctas = [&](int seqs) { return static_cast<long long>(a.H) * ((a.B + seqs - 1) / seqs); };
    if (ctas(1) <= a.num_sms) return launch_dot<1>(mp, cfg);
    if (ctas(2) <= a.num_sms) return launch_dot<2>(mp, cfg);
    if (ctas(4) <= 2 * a.num_sms) return launch_dot<4>(mp, cfg);
    static std::atomic<unsigned long long> done{0};
    if ((e = first_time(done, [] {
             return cudaFuncSetAttribute(fp4_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemMerge));
         })) != cudaSuccess)
        return e;
    CUtensorMap tm_wuv;
    const cuuint64_t wd[2] = {kR, static_cast<cuuint64_t>(a.H) * kDV}, ws[1] = {kR * 2};
    const cuuint32_t wb[2] = {64, kDV};
    if (encode_map(&tm_wuv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, a.w_uv, 2, wd, ws, wb) !=
        CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    cfg.gridDim = dim3((a.B + kMRows - 1) / kMRows, a.H);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = kSmemMerge;
    return cudaLaunchKernelEx(&cfg, fp4_merge_kernel, tm_wuv, mp);
}

}  // namespace mla
