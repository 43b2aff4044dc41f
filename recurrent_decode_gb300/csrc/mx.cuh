// mx.cuh -- microscaled blocks: 32 consecutive values of a row that share one
// power of two, kept as its biased exponent s (one byte: 2^(s - 127), 255 = no
// number).  The two element formats and the power each block takes:
//
//   MXFP4   4 bits a value, sign and one of 0, 1/2, 1, 3/2, 2, 3, 4, 6;
//           s - 127 is the least e >= -127 with max |x| <= 6 * 2^e
//   MXINT8  8 bits a value, q / 64 with q in -127 .. 127;
//           s - 127 is the least e >= -126 with max |x| <= 127/64 * 2^e
//           (at most 127: values in the last 128th of fp32's range are cut to it)
//
// Formats and the byte's meaning are those of the Open Compute Project's microscaling
// specification (v1.0).  It leaves the choice of the power open; the least one that
// cuts off no value is taken here, so the largest value of a block, which carries most
// of a sum, is never off by more than half a step.  x * 2^-e is exact in fp32 (or
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
    const void *rows;      // if not null, what x is quantised from: rows of type rtype, ldr apart,
    int rtype, rvec;       // rvec: on 16-byte (fp32: 32-byte) boundaries
    int over;              // they may share memory with y
    int64_t ldr;
    void *y;
    int64_t ldy;
    int B, N, K;
    int act;  // 0 none, 1 relu(.)^2
    uint32_t *err;
};
// type: MxType of y.  Where p.rows is given and the product is not one that quantises
// them itself, quantize(ctx) is called first to launch the kernel that writes p.x; the
// product then starts early, beside it.
void launch_mx_linear(const MxLinearParams &p, int type, cudaStream_t stream, cudaError_t (*quantize)(void *),
                      void *ctx, cudaError_t *e);

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
// The values of eight codes of a block of power s.
__device__ __forceinline__ void mx4_values(uint32_t code, uint32_t s, float (&v)[8]) {
    fp4_unpack8(code, v);
    const float f = s == 255u ? __uint_as_float(0x7FC00000u) : mx_power(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= f;
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

// Eight neighbouring values of a row as a lane holds them between load and use: in
// 16-bit types two a word, so that four lines in flight take 16 registers.
template <int T>
struct MxElem;
template <>
struct MxElem<MX_F32> {
    using type = float;
    struct Eight {
        float v[8];
    };
    static __device__ __forceinline__ void load(Eight &u, const float *p) { ld_v8(u.v, p); }
    static __device__ __forceinline__ void store(float *p, const float (&v)[8]) { st_v8(p, v); }
    static __device__ __forceinline__ void store_aligned(float *p, const float (&v)[8]) {  // to shared memory
        *(float4 *)p = *(const float4 *)&v[0];
        *(float4 *)(p + 4) = *(const float4 *)&v[4];
    }
    static __device__ __forceinline__ void set(Eight &u, int i, float v) { u.v[i] = v; }
    static __device__ __forceinline__ uint32_t top(const Eight &u) { return mx_quad_top(u.v); }
    // A line of `cols` values off the grid, neighbours by neighbouring lanes, and its
    // turn through shared memory (room for 256) to eight neighbours a lane; the same back.
    static __device__ __forceinline__ void gather(Eight &u, float &, const float *p, int cols, int lane) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u.v[i] = i * 32 + lane < cols ? p[i * 32 + lane] : 0.0f;
    }
    static __device__ __forceinline__ void turn(Eight &u, float, const float *, float *room, int lane) {
#pragma unroll
        for (int i = 0; i < 8; ++i) room[i * 32 + lane] = u.v[i];
        __syncwarp();
        *(float4 *)&u.v[0] = *(const float4 *)(room + lane * 8);
        *(float4 *)&u.v[4] = *(const float4 *)(room + lane * 8 + 4);
    }
    static __device__ __forceinline__ void scatter(float *p, const float *room, int cols, int lane) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * 32 + lane < cols) p[i * 32 + lane] = room[i * 32 + lane];
    }
    static __device__ __forceinline__ float up(const Eight &u, int i) { return u.v[i]; }
    static __device__ __forceinline__ float down(float v) { return v; }
};
// 16-bit types.  Their bits without the sign order like their values (infinity and
// NaN last), as pairs of unsigned halves.
template <typename E>
struct MxHalves {
    using type = E;
    struct Eight {
        uint32_t w[4];
    };
    static __device__ __forceinline__ void load(Eight &u, const E *p) { *(uint4 *)u.w = *(const uint4 *)p; }
    static __device__ __forceinline__ void set(Eight &u, int i, E v) { ((E *)u.w)[i] = v; }
    // As for fp32, by words of two values from the first word on that lies in the row;
    // the value before it, where there is one, is `edge` (lane 0).
    static __device__ __forceinline__ int skip(const E *p) { return (int)((uintptr_t)p >> 1 & 1u); }
    static __device__ __forceinline__ void gather(Eight &u, E &edge, const E *p, int cols, int lane) {
        const int e0 = skip(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = e0 + (j * 32 + lane) * 2;
            u.w[j] = e + 2 <= cols ? *(const uint32_t *)(p + e) : (e < cols ? *(const unsigned short *)(p + e) : 0u);
        }
        if (e0 && lane == 0) edge = p[0];
    }
    static __device__ __forceinline__ void turn(Eight &u, E edge, const E *p, E *room, int lane) {
        const int e0 = skip(p);
        unsigned short *h = (unsigned short *)room;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = e0 + (j * 32 + lane) * 2;
            if (e0 == 0) {
                ((uint32_t *)room)[j * 32 + lane] = u.w[j];
            } else {
                h[e] = (unsigned short)u.w[j];
                if (e < 255) h[e + 1] = (unsigned short)(u.w[j] >> 16);
            }
        }
        if (e0 && lane == 0) room[0] = edge;
        __syncwarp();
        *(uint4 *)u.w = *(const uint4 *)(room + lane * 8);
    }
    static __device__ __forceinline__ void scatter(E *p, const E *room, int cols, int lane) {
        const int e0 = skip(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = e0 + (j * 32 + lane) * 2;
            if (e + 2 <= cols) {
                const unsigned short *h = (const unsigned short *)room + e;
                *(uint32_t *)(p + e) = (uint32_t)h[0] | (uint32_t)h[1] << 16;
            } else if (e < cols) {
                p[e] = room[e];
            }
        }
        if (e0 && lane == 0) p[0] = room[0];
    }
    static __device__ __forceinline__ uint32_t top_bits(const Eight &u) {
        uint32_t m = __vmaxu2(__vmaxu2(u.w[0] & 0x7FFF7FFFu, u.w[1] & 0x7FFF7FFFu),
                              __vmaxu2(u.w[2] & 0x7FFF7FFFu, u.w[3] & 0x7FFF7FFFu));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
        return max(m >> 16, m & 0xFFFFu);
    }
};
template <>
struct MxElem<MX_F16> : MxHalves<__half> {
    static __device__ __forceinline__ uint32_t top(const Eight &u) {
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top_bits(u))));
    }
    static __device__ __forceinline__ float up(const Eight &u, int i) {
        return __half2float(((const __half *)u.w)[i]);
    }
    static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ void store_aligned(__half *p, const float (&v)[8]) { store(p, v); }
    static __device__ __forceinline__ void store(__half *p, const float (&v)[8]) {
        __half2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        *(uint4 *)p = *(const uint4 *)h;
    }
};
template <>
struct MxElem<MX_BF16> : MxHalves<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t top(const Eight &u) { return top_bits(u) << 16; }
    static __device__ __forceinline__ float up(const Eight &u, int i) {
        return __uint_as_float(i & 1 ? u.w[i >> 1] & 0xFFFF0000u : u.w[i >> 1] << 16);
    }
    static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ void store_aligned(__nv_bfloat16 *p, const float (&v)[8]) { store(p, v); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8]) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        *(uint4 *)p = *(const uint4 *)h;
    }
};

// A block's power and a lane's eight codes of a line (256 columns of a row, eight a
// lane); lanes 0 and 16 get the word of their half line's four powers.
template <int T>
__device__ __forceinline__ uint32_t mx4_line(const typename MxElem<T>::Eight &u, uint32_t &powers) {
    const uint32_t s = mx_scale<MXFP4>(MxElem<T>::top(u));
    const float f = mx_inverse(s);  // a block without a number: its codes do not matter
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = MxElem<T>::up(u, i) * f;
    powers = s | __shfl_down_sync(0xffffffffu, s, 4) << 8;
    powers |= __shfl_down_sync(0xffffffffu, powers, 8) << 16;
    return fp4_pack8(v);
}
#endif

}  // namespace rk
