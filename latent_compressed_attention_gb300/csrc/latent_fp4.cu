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
// Both directions are a stream bound by HBM: a thread takes 8 elements (16 bytes of bf16 or 32 of fp32 against 4 of
// codes), four neighbouring lanes a group, so that every access of a warp is contiguous.
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 8;      // elements a thread converts at a time

// Rows of one launch: `rows` of them in runs of `run` (a sequence's rows), each cut into r / 8 pieces.
struct Pieces {
    long long rows, run;
    int per_row;          // r / 8
    unsigned magic;       // ceil(2^32 / per_row): i / per_row = (i * magic) >> 32 for i * per_row < 2^32
    int rows_per_block;
};

__device__ __forceinline__ unsigned piece_row(const Pieces &p, unsigned i) {
    return __umulhi(i, p.magic);
}

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

__device__ __forceinline__ void load_piece(const __nv_bfloat16 *src, float (&x)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load_piece(const float *src, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(src)), b = __ldg(reinterpret_cast<const float4 *>(src) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <typename T, bool kAppend>
__global__ void __launch_bounds__(kThreads) write_latent_fp4_kernel(const WriteParams p) {
    const long long row0 = static_cast<long long>(blockIdx.x) * p.pc.rows_per_block;
    const unsigned n = static_cast<unsigned>(min(static_cast<long long>(p.pc.rows_per_block), p.pc.rows - row0)) *
                       static_cast<unsigned>(p.pc.per_row);
    for (unsigned i0 = threadIdx.x; i0 - threadIdx.x < n; i0 += kThreads) {   // whole warps: the shuffles below
        const unsigned i = min(i0, n - 1);                                    // want every lane
        const unsigned lr = piece_row(p.pc, i), piece = i - lr * static_cast<unsigned>(p.pc.per_row);
        const long long row = row0 + lr;
        float x[kPiece];
        load_piece(static_cast<const T *>(p.c) + row * p.ld_c + piece * kPiece, x);
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
        if (i0 >= n) continue;
        long long to = row;
        if constexpr (kAppend) {
            const long long b = row / p.pc.run, t = row - b * p.pc.run;
            if (p.counts) {
                const int count = __ldg(p.counts + b);
                if (count < 0 || count > p.pc.run) record_error(p.err, kDevErrBounds);
                if (t >= count) continue;
            }
            const long long pos = __ldg(p.lens + b) + t;
            if (pos < 0 || pos >= p.max_len) {
                record_error(p.err, kDevErrBounds);
                continue;
            }
            to = b * p.max_len + pos;
        }
        uint8_t *dst = p.c4 + to * p.ld_c4;
        reinterpret_cast<uint32_t *>(dst)[piece] = codes;
        if ((piece & 3) == 0) dst[p.r / 2 + (piece >> 2)] = static_cast<uint8_t>(bad ? 255 : e + 127);
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

__device__ __forceinline__ void store_piece(__nv_bfloat16 *dst, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                 pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store_piece(float *dst, const float (&x)[8]) {
    reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) read_latent_fp4_kernel(const ReadParams p) {
    const long long row0 = static_cast<long long>(blockIdx.x) * p.pc.rows_per_block;
    const unsigned n = static_cast<unsigned>(min(static_cast<long long>(p.pc.rows_per_block), p.pc.rows - row0)) *
                       static_cast<unsigned>(p.pc.per_row);
    for (unsigned i = threadIdx.x; i < n; i += kThreads) {
        const unsigned lr = piece_row(p.pc, i), piece = i - lr * static_cast<unsigned>(p.pc.per_row);
        const long long row = row0 + lr;
        const long long b = p.pc.run == p.pc.rows ? 0 : row / p.pc.run, u = row - b * p.pc.run;
        if (p.lens) {
            const int len = __ldg(p.lens + b);
            if (len < 0) record_error(p.err, kDevErrBounds);
            if (u >= len) continue;
        }
        const uint8_t *src = p.c4 + b * p.batch_c4 + u * p.ld_c4;
        const uint32_t codes = __ldg(reinterpret_cast<const uint32_t *>(src) + piece);
        const float scale = fp4_scale(__ldg(src + p.r / 2 + (piece >> 2)));
        float x[kPiece];
        unpack_e2m1x8(codes, x);
#pragma unroll
        for (int k = 0; k < kPiece; ++k) x[k] *= scale;
        store_piece(static_cast<T *>(p.c) + row * p.ld_c + piece * kPiece, x);
    }
}

Pieces pieces_of(long long rows, long long run, int r, long long *blocks) {
    Pieces pc;
    pc.rows = rows;
    pc.run = run;
    pc.per_row = r / kPiece;
    pc.magic = static_cast<unsigned>((0x100000000ull + pc.per_row - 1) / pc.per_row);
    pc.rows_per_block = pc.per_row >= kThreads ? 1 : kThreads / pc.per_row;
    *blocks = (rows + pc.rows_per_block - 1) / pc.rows_per_block;
    return pc;
}

}  // namespace

cudaError_t launch_write_latent_fp4(const LatentFp4Args &a, cudaStream_t s) {
    WriteParams p{a.c,    static_cast<uint8_t *>(a.c4), a.ld_c, a.ld_c4, a.lens, a.counts, a.max_len,
                  a.dev_err, {},                        a.r};
    long long blocks = 0;
    p.pc = pieces_of(a.B * a.rows, a.rows, a.r, &blocks);
    if (blocks <= 0) return cudaSuccess;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(blocks);
    note_launch();
    if (a.lens)
        a.f32 ? write_latent_fp4_kernel<float, true><<<grid, kThreads, 0, s>>>(p)
              : write_latent_fp4_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, s>>>(p);
    else
        a.f32 ? write_latent_fp4_kernel<float, false><<<grid, kThreads, 0, s>>>(p)
              : write_latent_fp4_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_read_latent_fp4(const LatentFp4Args &a, cudaStream_t s) {
    ReadParams p{static_cast<const uint8_t *>(a.c4), const_cast<void *>(a.c), a.ld_c4, a.batch_c4, a.ld_c, a.lens,
                 a.dev_err, {}, a.r};
    long long blocks = 0;
    p.pc = pieces_of(a.B * a.rows, a.rows, a.r, &blocks);
    if (blocks <= 0) return cudaSuccess;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(blocks);
    note_launch();
    a.f32 ? read_latent_fp4_kernel<float><<<grid, kThreads, 0, s>>>(p)
          : read_latent_fp4_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mla
