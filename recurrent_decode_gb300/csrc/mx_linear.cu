// mx_linear.cu -- y[b][n] = act(sum_k x[b][k] w[n][k]) of two MXFP4 matrices
// (layout: mx.cuh), fp32 sums, y in fp32, fp16 or bf16.
//
// A plain form first: one thread a result, a block's 32 products as whole numbers
// of quarters (exact), then the two powers of two, then the running fp32 sum.
#include "mx.cuh"

namespace rk {

// Twice the value of each of four codes (the low or high nibbles of a word's bytes) as signed bytes.
__device__ __forceinline__ uint32_t fp4_twice(uint32_t n) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = (n >> (8 * i)) & 15u;
        const int m = (int)((0xC8643210u >> (4 * (c & 7u))) & 15u);
        r |= ((uint32_t)(c & 8u ? -m : m) & 255u) << (8 * i);
    }
    return r;
}

template <typename O>
__device__ __forceinline__ void mx_put(O *y, float v);
template <>
__device__ __forceinline__ void mx_put(float *y, float v) { *y = v; }
template <>
__device__ __forceinline__ void mx_put(__half *y, float v) { *y = __float2half_rn(v); }
template <>
__device__ __forceinline__ void mx_put(__nv_bfloat16 *y, float v) { *y = __float2bfloat16_rn(v); }

template <typename O>
__global__ void __launch_bounds__(256) mx_linear_kernel(const MxLinearParams p) {
    const int n = blockIdx.x * 16 + (threadIdx.x & 15), b = blockIdx.y * 16 + (threadIdx.x >> 4);
    if (n >= p.N || b >= p.B) return;
    const int kt = (p.K + MX_TILE_K - 1) / MX_TILE_K, blocks = (p.K + MX_BLOCK - 1) / MX_BLOCK;
    const int rb = b % MX_TILE_M, rn = n % MX_TILE_M;
    const uint8_t *xb = p.x + (int64_t)(b / MX_TILE_M) * kt * MX_TILE_BYTES;
    const uint8_t *wb = p.w + (int64_t)(n / MX_TILE_M) * kt * MX_TILE_BYTES;
    float acc = 0.0f;
    for (int k = 0; k < blocks; ++k) {
        const int64_t tile = (int64_t)(k / 8) * MX_TILE_BYTES;
        const int j = k % 8;
        const uint4 cx = *(const uint4 *)(xb + tile + MX_SCALE_BYTES + rb * 128 + ((j ^ (rb & 7)) << 4));
        const uint4 cw = *(const uint4 *)(wb + tile + MX_SCALE_BYTES + rn * 128 + ((j ^ (rn & 7)) << 4));
        const uint32_t sx = xb[tile + (j >> 2) * 512 + (rb & 31) * 16 + (rb >> 5) * 4 + (j & 3)];
        const uint32_t sw = wb[tile + (j >> 2) * 512 + (rn & 31) * 16 + (rn >> 5) * 4 + (j & 3)];
        int dot = 0;
        const uint32_t ax[4] = {cx.x, cx.y, cx.z, cx.w}, aw[4] = {cw.x, cw.y, cw.z, cw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dot = __dp4a((int)fp4_twice(ax[i]), (int)fp4_twice(aw[i]), dot);
            dot = __dp4a((int)fp4_twice(ax[i] >> 4), (int)fp4_twice(aw[i] >> 4), dot);
        }
        const float nan = __uint_as_float(0x7FC00000u);
        acc += (float)dot * 0.25f * (sx == 255u ? nan : mx_power(sx)) * (sw == 255u ? nan : mx_power(sw));
    }
    if (p.act) {
        acc = acc > 0.0f ? acc * acc : (acc != acc ? acc : 0.0f);
    }
    mx_put((O *)p.y + (int64_t)b * p.ldy + n, acc);
}

void launch_mx_linear(const MxLinearParams &p, int type, const LaunchCfg &lc, cudaError_t *e) {
    const dim3 grid((p.N + 15) / 16, (p.B + 15) / 16);
    if (type == MX_F32) mx_linear_kernel<float><<<grid, 256, 0, lc.stream>>>(p);
    else if (type == MX_F16) mx_linear_kernel<__half><<<grid, 256, 0, lc.stream>>>(p);
    else mx_linear_kernel<__nv_bfloat16><<<grid, 256, 0, lc.stream>>>(p);
    const cudaError_t r = cudaGetLastError();
    if (r != cudaSuccess) *e = r;
}

}  // namespace rk
