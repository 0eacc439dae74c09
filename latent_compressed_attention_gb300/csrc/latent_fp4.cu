// The 4-bit latent cache: writing rows (whole prompts, chunks, single tokens) and reading them back.
//
// Only the latent c is cached (page "Gated MLA（矩阵吸收版）", KV-cache table in section "形状与参数对比": r values
// per token).  Here a row of r values is held as OCP MX fp4: r / 2 bytes of e2m1 codes (element 2j in the low half of
// byte j), then r / 32 scale bytes, one power of two per 32 consecutive elements.
//
//   write  e = the smallest exponent in [-40, 40] with max|group| <= 7 * 2^e, code = e2m1(x * 2^-e), scale = e + 127.
//          Up to 7 the saturation at 6 is off by no more than the half step between 4 and 6, and one exponent lower
//          keeps twice the resolution for the rest of the group: mean squared error 1.25 % of the mean square on
//          normal data, against 1.33 % when the group's maximum itself must fit.  x * 2^-e is exact, so the
//          conversion's rounding is the only one.
//   read   value = e2m1 * 2^(scale - 127): at most two significant bits, exact in bf16 and fp32.
//
// Both directions are a stream bound by HBM: a thread takes pieces of a few elements, neighbouring lanes a group, so that
// every access of a warp is contiguous.  A thread has four pieces' loads in flight (131072 bf16 rows written in 30 us,
// 5.7 TB/s, and read back in 26, against 42 and 38 with one; 4096 rows 2.1 and 1.8 us against 2.3 and 2.2; 131072 fp32
// rows 47 us, 6.5 TB/s, and 46, against 46 and 70), or one where a sequence has too few rows for that, as the single
// tokens of a decode step.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 8;      // elements that a thread of the write converts at a time
constexpr int kMany = 4;       // pieces per thread of a long run

// The rows of a launch: runs (a sequence's rows) of `run`, each cut into blocks of rows and those into pieces.
struct Pieces {
    long long run;
    int per_row;          // pieces of a row
    unsigned magic;       // ceil(2^32 / per_row): i / per_row = (i * magic) >> 32 for i * per_row < 2^32
    int rows_per_block;
    unsigned blocks_per_run;
};
__device__ __forceinline__ unsigned piece_row(const Pieces &p, unsigned i) { return __umulhi(i, p.magic); }

struct Block {
    long long seq, row0;   // its run, and its first row there
    unsigned n;            // its pieces
    __device__ explicit Block(const Pieces &p) {
        const unsigned b = blockIdx.x / p.blocks_per_run;
        seq = b;
        row0 = static_cast<long long>(blockIdx.x - b * p.blocks_per_run) * p.rows_per_block;
        n = static_cast<unsigned>(min(static_cast<long long>(p.rows_per_block), p.run - row0)) *
            static_cast<unsigned>(p.per_row);
    }
};

struct WriteParams {
    const void *c;
    uint8_t *c4;
    long long ld_c, ld_c4;      // elements, bytes
    const int *lens, *counts;   // append: [B]; NULL: rows go to the same row of c4
    long long max_len;
    int *err;
    Pieces pc;
    int r;
};

template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ void load(const __nv_bfloat16 *src) { v = __ldcs(reinterpret_cast<const uint4 *>(src)); }
    __device__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ void load(const float *src) {
        a = __ldcs(reinterpret_cast<const float4 *>(src)), b = __ldcs(reinterpret_cast<const float4 *>(src) + 1);
    }
    __device__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};

template <typename T, bool kAppend, int N>
__global__ void __launch_bounds__(kThreads) write_latent_fp4_kernel(const WriteParams p) {
    grid_dependency_wait();
    const Block blk(p.pc);
    const T *const src = static_cast<const T *>(p.c) + (blk.seq * p.pc.run + blk.row0) * p.ld_c;
    long long row0 = blk.row0;       // of the block's first row, in its sequence's part of c4
    unsigned first = 0, past = blk.n;   // the block's rows [first, past) are written (append)
    if constexpr (kAppend) {
        long long count = p.pc.run;
        if (p.counts) {
            count = __ldg(p.counts + blk.seq);
            if (count < 0 || count > p.pc.run) record_error(p.err, kDevErrBounds);
        }
        row0 += __ldg(p.lens + blk.seq);
        const long long rows = min(static_cast<long long>(p.pc.rows_per_block), min(count, p.pc.run) - blk.row0);
        const long long lo = min(max(-row0, 0ll), max(rows, 0ll)), hi = max(lo, min(rows, p.max_len - row0));
        if (rows > 0 && (lo > 0 || hi < rows)) record_error(p.err, kDevErrBounds);
        first = static_cast<unsigned>(lo), past = static_cast<unsigned>(hi);
    }
    uint8_t *const dst = p.c4 + ((kAppend ? blk.seq * p.max_len : blk.seq * p.pc.run) + row0) * p.ld_c4;
    for (unsigned i0 = 0; i0 < blk.n; i0 += N * blockDim.x) {
        Raw<T> raw[N];
        unsigned lr[N], piece[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned i = min(i0 + j * blockDim.x + threadIdx.x, blk.n - 1);   // whole warps: the shuffles below
            lr[j] = piece_row(p.pc, i);                                             // want every lane
            piece[j] = i - lr[j] * static_cast<unsigned>(p.pc.per_row);
            raw[j].load(src + lr[j] * p.ld_c + piece[j] * kPiece);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float x[kPiece];
            raw[j].get(x);
            uint32_t top = 0;   // |x| orders like its bits; infinities and NaN lie above every finite value
#pragma unroll
            for (int k = 0; k < kPiece; ++k) top = max(top, __float_as_uint(x[k]) & 0x7FFFFFFFu);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const bool bad = top >= 0x7F800000u;
            // max|x| = 1.f * 2^E <= 7 * 2^e: e = E - 2 up to 1.75 * 2^E, E - 1 beyond
            const int e = min(40, max(-40, static_cast<int>(top >> 23) - 129 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0)));
            const float down = exp2_int(-e);
            uint32_t codes = 0;
            if (!bad) codes = pack_e2m1x8(x, down);
            if (i0 + j * blockDim.x + threadIdx.x >= blk.n || (kAppend && (lr[j] < first || lr[j] >= past))) continue;
            uint8_t *to = dst + lr[j] * p.ld_c4;
            reinterpret_cast<uint32_t *>(to)[piece[j]] = codes;
            if ((piece[j] & 3) == 0) to[p.r / 2 + (piece[j] >> 2)] = static_cast<uint8_t>(bad ? 255 : e + 127);
        }
    }
}

struct ReadParams {
    const uint8_t *c4;
    void *c;
    long long ld_c4, batch_c4, ld_c;   // bytes, bytes, elements
    const int *lens;                   // [B] or NULL: rows at or past lens[b] are not written
    int *err;
    Pieces pc;
    int r;
};

// A piece of the read is 16 bytes of output, so that a warp's stores are contiguous: 8 codes of bf16, 4 of fp32.
__device__ __forceinline__ uint32_t load_codes(const uint8_t *src, unsigned piece, const __nv_bfloat16 *) {
    return __ldg(reinterpret_cast<const uint32_t *>(src) + piece);
}
__device__ __forceinline__ uint32_t load_codes(const uint8_t *src, unsigned piece, const float *) {
    return __ldg(reinterpret_cast<const uint16_t *>(src) + piece);
}
__device__ __forceinline__ void store_piece(__nv_bfloat16 *dst, uint32_t codes, float by) {
    float x[8];
    unpack_e2m1x8(codes, x);
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(x[0] * by, x[1] * by), pack_bf16x2(x[2] * by, x[3] * by),
                                                 pack_bf16x2(x[4] * by, x[5] * by), pack_bf16x2(x[6] * by, x[7] * by));
}
__device__ __forceinline__ void store_piece(float *dst, uint32_t codes, float by) {
    float x[8];
    unpack_e2m1x8(codes, x);
    *reinterpret_cast<float4 *>(dst) = make_float4(x[0] * by, x[1] * by, x[2] * by, x[3] * by);
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads) read_latent_fp4_kernel(const ReadParams p) {
    constexpr int kOut = 16 / sizeof(T);
    grid_dependency_wait();
    const Block blk(p.pc);
    unsigned n = blk.n;
    if (p.lens) {
        const int len = __ldg(p.lens + blk.seq);
        if (len < 0) record_error(p.err, kDevErrBounds);
        const long long rows = min(static_cast<long long>(p.pc.rows_per_block), len - blk.row0);
        n = rows <= 0 ? 0u : min(n, static_cast<unsigned>(rows) * static_cast<unsigned>(p.pc.per_row));
    }
    const uint8_t *const src = p.c4 + blk.seq * p.batch_c4 + blk.row0 * p.ld_c4;
    T *const dst = static_cast<T *>(p.c) + (blk.seq * p.pc.run + blk.row0) * p.ld_c;
    for (unsigned i0 = 0; i0 < n; i0 += N * blockDim.x) {
        uint32_t codes[N];
        uint8_t scale[N];
        unsigned lr[N], piece[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned i = min(i0 + j * blockDim.x + threadIdx.x, n - 1);
            lr[j] = piece_row(p.pc, i);
            piece[j] = i - lr[j] * static_cast<unsigned>(p.pc.per_row);
            const uint8_t *row = src + lr[j] * p.ld_c4;
            codes[j] = load_codes(row, piece[j], static_cast<const T *>(nullptr));
            scale[j] = __ldg(row + p.r / 2 + piece[j] / (32 / kOut));
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (i0 + j * blockDim.x + threadIdx.x < n)
                store_piece(dst + lr[j] * p.ld_c + piece[j] * kOut, codes[j], fp4_scale(scale[j]));
    }
}

// Runs f(pieces, blocks, threads, is_long).
template <typename F>
cudaError_t launch_pieces(long long runs, long long run, int per_row, F f) {
    if (runs <= 0 || run <= 0) return cudaSuccess;
    Pieces pc;
    pc.run = run;
    pc.per_row = per_row;
    pc.magic = static_cast<unsigned>((0x100000000ull + per_row - 1) / per_row);
    const auto cut = [&](int pieces) {
        pc.rows_per_block = std::max(1, pieces * kThreads / per_row);
        const long long blocks = (run + pc.rows_per_block - 1) / pc.rows_per_block;
        pc.blocks_per_run = static_cast<unsigned>(std::min(blocks, 0xFFFFFFFFll));
        return blocks;
    };
    const bool is_long = run * per_row >= kMany * kThreads;
    const long long blocks = cut(is_long ? kMany : 1);
    if (blocks > 0x7FFFFFFFLL / runs) return cudaErrorInvalidValue;
    // a short run takes no more warps than it fills
    const long long pieces = std::min<long long>(run, pc.rows_per_block) * per_row;
    const unsigned threads = static_cast<unsigned>(std::min<long long>(kThreads, (pieces + 31) / 32 * 32));
    note_launch();
    return f(pc, static_cast<unsigned>(blocks * runs), threads, is_long);
}

template <typename T, bool kAppend>
cudaError_t launch_write(const WriteParams &p, unsigned grid, unsigned threads, bool is_long, cudaStream_t s) {
    return is_long ? launch_dependent(write_latent_fp4_kernel<T, kAppend, kMany>, dim3(grid), threads, 0, s, p)
                   : launch_dependent(write_latent_fp4_kernel<T, kAppend, 1>, dim3(grid), threads, 0, s, p);
}
template <typename T>
cudaError_t launch_read(const ReadParams &p, unsigned grid, unsigned threads, bool is_long, cudaStream_t s) {
    return is_long ? launch_dependent(read_latent_fp4_kernel<T, kMany>, dim3(grid), threads, 0, s, p)
                   : launch_dependent(read_latent_fp4_kernel<T, 1>, dim3(grid), threads, 0, s, p);
}

}  // namespace

cudaError_t launch_write_latent_fp4(const LatentFp4Args &a, cudaStream_t s) {
    WriteParams p{a.c,    static_cast<uint8_t *>(a.c4), a.ld_c, a.ld_c4, a.lens, a.counts, a.max_len,
                  a.dev_err, {},                        a.r};
    return launch_pieces(a.B, a.rows, a.r / kPiece, [&](const Pieces &pc, unsigned grid, unsigned threads, bool is_long) {
        p.pc = pc;
        if (a.lens)
            return a.f32 ? launch_write<float, true>(p, grid, threads, is_long, s)
                         : launch_write<__nv_bfloat16, true>(p, grid, threads, is_long, s);
        return a.f32 ? launch_write<float, false>(p, grid, threads, is_long, s)
                     : launch_write<__nv_bfloat16, false>(p, grid, threads, is_long, s);
    });
}

cudaError_t launch_read_latent_fp4(const LatentFp4Args &a, cudaStream_t s) {
    ReadParams p{static_cast<const uint8_t *>(a.c4), const_cast<void *>(a.c), a.ld_c4, a.batch_c4, a.ld_c, a.lens,
                 a.dev_err, {}, a.r};
    const int per_row = a.f32 ? a.r / 4 : a.r / 8;
    return launch_pieces(a.B, a.rows, per_row, [&](const Pieces &pc, unsigned grid, unsigned threads, bool is_long) {
        p.pc = pc;
        return a.f32 ? launch_read<float>(p, grid, threads, is_long, s)
                     : launch_read<__nv_bfloat16>(p, grid, threads, is_long, s);
    });
}

}  // namespace mla
