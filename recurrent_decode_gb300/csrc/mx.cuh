// mx.cuh -- microscaled blocks: 32 consecutive values of a row that share one
// power of two, kept as its biased exponent s (one byte: 2^(s - 127), 255 = no
// number).  The two element formats and the power each block takes:
//
//   MXFP4   4 bits a value, sign and one of 0, 1/2, 1, 3/2, 2, 3, 4, 6;
//           s - 127 is the least e >= -127 with max |x| <= 6 * 2^e
//   MXINT8  8 bits a value, q / 64 with q in -127 .. 127;
//           s - 127 is the least e >= -126 with max |x| <= 127/64 * 2^e
//           (at most 127: fp32 values within 2^-7 of the type's end are cut to it)
//
// Formats and the byte's meaning are those of the Open Compute Project's
// microscaling specification (v1.0).  It leaves the choice of the power open; the least one that cuts off
// no value is taken here, so the largest value of a block, which carries most of
// a sum, is never off by more than half a step.  x * 2^-e is exact in fp32 (or
// below every threshold of the grid), so a code depends on the value alone: to
// the nearest grid point, ties to the even code.  A block that holds an infinity
// or NaN gets s = 255 and reads back as NaN.
//
// An MXFP4 matrix of R rows and K columns is a row of tiles of 128 rows x 256
// columns, ordered (row tile, column tile), each 17,408 contiguous bytes:
//   bytes 0 .. 1023     two chunks of 512 bytes, columns 0-127 and 128-255: the
//                       power of row r, block j of the chunk at
//                       (r % 32) * 16 + (r / 32) * 4 + j
//   bytes 1024 .. 17407 the codes of row r at 128 r: 16 bytes a block, block j at
//                       place j ^ (r & 7), its values in order, low half first
// The first is the order in which the tensor cores take powers from tensor
// memory, the second the 128-byte swizzle of their shared-memory operand: a tile
// is fetched by one contiguous bulk copy and used as it lies.  Columns K and up
// of a tile hold zeros; rows R and up hold anything (they enter no kept result).
#pragma once
#include <cuda_bf16.h>

#include "internal.cuh"

namespace rk {

constexpr int MX_BLOCK = 32;
constexpr int MX_TILE_M = 128;
constexpr int MX_TILE_K = 256;
constexpr uint32_t MX_SCALE_BYTES = 1024;  // of one tile
constexpr uint32_t MX_TILE_BYTES = MX_SCALE_BYTES + MX_TILE_M * MX_TILE_K / 2;

enum MxType : int { MX_F32 = 0, MX_F16 = 1, MX_BF16 = 2 };
enum MxFormat : int { MXFP4 = 0, MXINT8 = 1 };

// One quantised product y = act(xq wq^T); see launch_mx_linear.
struct MxLinearParams {
    const uint8_t *x, *w;  // MXFP4 matrices [B][K], [N][K]
    void *y;
    int64_t ldy;
    int B, N, K;
    int act;  // 0 none, 1 relu(.)^2
    uint32_t *err;
};
// type: MxType of y.  pdl: the kernel before it on the stream writes x and lets
// this one start early.
void launch_mx_linear(const MxLinearParams &p, int type, const LaunchCfg &lc, cudaError_t *e);

// The slot pool of a ctx, for saving and loading states (mx_ctx_states).
struct MxCtxStates {
    float *wkv, *att, *ffn;
    int L, H, n_slots, n_entries, n, format, V;
    const int32_t *slots, *entries;
    uint8_t *cache;
    uint32_t *err;
    float *occ;                 // load: occurrence counts and draw counters that restart
    unsigned long long *ndraw;
    void *stream;
};
int mx_ctx_states(bool save, const MxCtxStates &c, const char **err_msg);

#ifdef __CUDACC__
__device__ __forceinline__ float mx_power(uint32_t s) {  // 2^(s - 127), s < 255
    return __uint_as_float(s ? s << 23 : 1u << 22);
}
__device__ __forceinline__ float mx_inverse(uint32_t s) {  // 2^(127 - s), s < 255
    return __uint_as_float(s < 254u ? (254u - s) << 23 : 1u << 22);
}
// The power of a block from the bits of its largest |x| (the bits of non-negative
// floats order like the floats, infinity and NaN last).
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale(uint32_t top) {
    const int e = (int)(top >> 23);
    if (e == 255) return 255u;
    const uint32_t frac = top & 0x7FFFFFu;
    if (FMT == MXFP4) return (uint32_t)max(0, e - 2 + (frac > 0x400000u));  // 6 = 1.5 * 2^2
    return (uint32_t)min(254, max(1, e + (frac > 0x7E0000u)));              // 127/64 = 1.984375
}

// Eight values on the MXFP4 grid: nearest, ties to even, past 6 to 6.
__device__ __forceinline__ uint32_t fp4_pack8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// The values of eight codes (fp16 holds them exactly).
__device__ __forceinline__ void fp4_unpack8(uint32_t r, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(r));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*(const __half2 *)&h[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
// Eight floats at a 32-byte aligned address, by one access.
__device__ __forceinline__ void ld_v8(float (&v)[8], const float *p) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ void st_v8(float *p, const float (&v)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// Largest |x| bits over the four lanes that hold a block's 32 values.
__device__ __forceinline__ uint32_t mx_quad_top(const float (&v)[8]) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
    return max(t, __shfl_xor_sync(0xffffffffu, t, 2));
}
#endif

}  // namespace rk
