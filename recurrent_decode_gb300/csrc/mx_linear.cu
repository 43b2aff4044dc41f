// mx_linear.cu -- y[b][n] = act(sum_k x[b][k] w[n][k]) of two MXFP4 matrices
// (layout: mx.cuh), fp32 sums, y in fp32, fp16 or bf16.
//
// The block-scaled tensor-core product does the whole inner formula: an
// instruction takes 64 columns of 4-bit codes of both sides and, for every row,
// the powers of the two 32-column blocks, and adds sum 2^(ea + eb) (a . b) to an
// fp32 accumulator.  Nothing is widened on the way, which is what bounds the int8
// weights.  128 weight rows form the M side and the tokens the N side (padded to
// 16, at most 256), so a decode batch reads each weight once.
//
// One CTA computes one tile of 128 outputs x up to 256 tokens over a range of
// column tiles of 256:
//   warp 0      bulk copies of whole tiles -- codes and powers as they lie, no
//               tensor map -- into a ring of stages; the weights of the first
//               stages are requested before the wait for the kernel that
//               quantises x
//   warp 1      per stage: powers from shared into tensor memory (tcgen05.cp, in
//               order before the products of the same thread), four products
//   warps 2-9   accumulator -> activation -> y; lane = output, so a warp's store
//               of one token covers 32 neighbouring outputs
// Each stage has columns of its own for its powers: they are overwritten only
// after the commit that also frees the stage's shared memory.
#include <algorithm>

#include "mx.cuh"

namespace rk {

constexpr int MXL_EPI_WARPS = 8;
constexpr int MXL_THREADS = 64 + 32 * MXL_EPI_WARPS;
constexpr int MXL_MAX_STAGES = 8;
constexpr uint32_t MXL_SMEM_MAX = 227 * 1024 - 256;  // a CTA's dynamic part

struct MxLinearArgs {
    MxLinearParams p;
    int kt;       // column tiles
    int nt;       // tokens of a full tile, a multiple of 16
    int stages;
    uint32_t xbytes;  // shared memory of a stage's x: both records' powers, then the codes
    uint32_t ncols;   // tensor memory columns
    uint32_t sfcol;   // first column of the powers
};

// Descriptor of 32 rows of 16 bytes, one after another (tcgen05.cp of powers).
__device__ __forceinline__ uint64_t sdesc_powers(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
// 128 rows' powers of four blocks: row r to lane r % 32 (of every quarter), column r / 32.
__device__ __forceinline__ void tmem_cp_powers(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// D[tmem] (+)= sum over two blocks of 2^(ea + eb) A B^T, codes packed two a byte.
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// Instruction descriptor: both sides 4-bit (code 1), powers of two as scales
// (bit 23), K = 64; `half` selects the bytes 0-1 or 2-3 of every scale word.
__device__ __forceinline__ uint32_t idesc_mxf4(int N, int half) {
    return 1u << 7 | 1u << 10 | (uint32_t)(N >> 3) << 17 | 1u << 23 | 1u << 27 | (uint32_t)half << 5 | (uint32_t)half << 30;
}

template <typename O>
__device__ __forceinline__ O mx_out(float v);
template <>
__device__ __forceinline__ float mx_out(float v) { return v; }
template <>
__device__ __forceinline__ __half mx_out(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 mx_out(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float mx_act(float v, int act) {
    return act ? (v > 0.0f ? v * v : (v != v ? v : 0.0f)) : v;
}

template <typename O>
__global__ void __launch_bounds__(MXL_THREADS, 1) mx_linear_kernel(const __grid_constant__ MxLinearArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[MXL_MAX_STAGES], empty[MXL_MAX_STAGES], done;
    __shared__ uint32_t tmem_slot, s_abort, s_ok;
    uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = a.stages, kt = a.kt;
    const int rt = blockIdx.x, b0 = blockIdx.y * a.nt;
    const int rows = min(a.nt, a.p.B - b0);       // tokens of this tile
    const int npad = (rows + 15) & ~15;
    const uint32_t stage_bytes = MX_TILE_BYTES + a.xbytes;
    volatile uint32_t *abort_flag = &s_abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&done, 1);
        s_abort = 0u;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, a.ncols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            const uint8_t *w = a.p.w + (int64_t)rt * kt * MX_TILE_BYTES;
            const uint8_t *x0 = a.p.x + (int64_t)(b0 / MX_TILE_M) * kt * MX_TILE_BYTES;
            const uint8_t *x1 = x0 + (int64_t)kt * MX_TILE_BYTES;
            const uint32_t n0 = (uint32_t)min(npad, MX_TILE_M) * 128u, n1 = (uint32_t)max(npad - MX_TILE_M, 0) * 128u;
            const uint32_t bytes = MX_TILE_BYTES + MX_SCALE_BYTES + n0 + (n1 ? MX_SCALE_BYTES + n1 : 0u);
            auto load_w = [&](int k, int st) {
                mbar_expect_tx(&full[st], bytes);
                bulk_g2s(base + st * stage_bytes, w + (int64_t)k * MX_TILE_BYTES, MX_TILE_BYTES, &full[st]);
            };
            auto load_x = [&](int k, int st) {
                uint8_t *to = base + st * stage_bytes + MX_TILE_BYTES;
                const int64_t at = (int64_t)k * MX_TILE_BYTES;
                bulk_g2s(to + MX_SCALE_BYTES, x0 + at, MX_SCALE_BYTES + n0, &full[st]);
                if (n1) {
                    bulk_g2s(to, x1 + at, MX_SCALE_BYTES, &full[st]);
                    bulk_g2s(to + 2 * MX_SCALE_BYTES + n0, x1 + at + MX_SCALE_BYTES, n1, &full[st]);
                }
            };
            const int npre = min(S, kt);
            for (int k = 0; k < npre; ++k) load_w(k, k);
            pdl_wait();
            for (int k = 0; k < npre; ++k) load_x(k, k);
            int k = npre;
            for (; k < kt; ++k) {
                const int st = k % S;
                if (!mbar_wait(&empty[st], (uint32_t)(k / S - 1) & 1u, abort_flag)) {
                    *abort_flag = 1u;
                    atomicOr(a.p.err, ERR_TIMEOUT);
                    break;
                }
                load_w(k, st);
                load_x(k, st);
            }
            // no copy may be in flight when the CTA ends
            for (int j = max(0, k - S); j < k; ++j)
                if (!mbar_wait_any(&full[j % S], (uint32_t)(j / S) & 1u)) break;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t id0 = idesc_mxf4(npad, 0), id1 = idesc_mxf4(npad, 1);
            const uint32_t xsf = npad > MX_TILE_M ? 8u : 4u;  // columns of one chunk of x's powers
            bool ok = true;
            for (int k = 0; k < kt; ++k) {
                const int st = k % S;
                if (!mbar_wait(&full[st], (uint32_t)(k / S) & 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sw = smem_u32(base + st * stage_bytes), sx = sw + MX_TILE_BYTES;
                const uint32_t sfa = tmem + a.sfcol + (uint32_t)st * 24u, sfb = sfa + 8u;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tmem_cp_powers(sfa + h * 4, sdesc_powers(sw + h * 512));
                    tmem_cp_powers(sfb + h * xsf, sdesc_powers(sx + MX_SCALE_BYTES + h * 512));
                    if (npad > MX_TILE_M) tmem_cp_powers(sfb + h * xsf + 4, sdesc_powers(sx + h * 512));
                }
                // a last tile of K % 256 columns: the instructions past them would add zeros
                const int ni = min(4, (a.p.K - k * MX_TILE_K + 63) / 64);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < ni)
                        mma_mxf4(tmem, sdesc_k128(sw + MX_SCALE_BYTES + i * 32), sdesc_k128(sx + 2 * MX_SCALE_BYTES + i * 32),
                                 (i & 1) ? id1 : id0, sfa + (i >> 1) * 4, sfb + (i >> 1) * xsf, (k | i) ? 1u : 0u);
                mma_commit(&empty[st]);
            }
            if (!ok) {
                *abort_flag = 1u;
                atomicOr(a.p.err, ERR_TIMEOUT);
            }
            mma_commit(&done);
            if (!ok) mbar_wait_any(&done, 0u);  // no product may be in flight when the CTA ends
        }
    } else {
        pdl_wait();  // y may have readers before the kernel this one follows
        const int et = threadIdx.x - 64, qd = warp & 3, grp = (warp - 2) >> 2;
        if (et == 0) s_ok = mbar_wait(&done, 0u, abort_flag) ? 1u : 0u;
        named_bar(1, 32 * MXL_EPI_WARPS);
        if (s_ok) {
            (void)mbar_try_wait(&done, 0u);
            tc_fence_after();
            const int n = rt * MX_TILE_M + qd * 32 + lane;
            O *y = (O *)a.p.y + (int64_t)b0 * a.p.ldy + n;
            for (int c = grp * 16; c < npad; c += 16 * (MXL_EPI_WARPS / 4)) {
                float v[16];
                tmem_ld16(tmem + ((uint32_t)(qd * 32) << 16) + (uint32_t)c, v);
                if (n < a.p.N) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < rows) y[(int64_t)(c + j) * a.p.ldy] = mx_out<O>(mx_act(v[j], a.p.act));
                }
            }
        } else if (et == 0) {
            *abort_flag = 1u;
            atomicOr(a.p.err, ERR_TIMEOUT);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, a.ncols);
    }
}

void launch_mx_linear(const MxLinearParams &p, int type, const LaunchCfg &lc, cudaError_t *e) {
    MxLinearArgs a;
    a.p = p;
    a.kt = (p.K + MX_TILE_K - 1) / MX_TILE_K;
    a.nt = std::min(256, (p.B + 15) & ~15);
    a.xbytes = 2 * MX_SCALE_BYTES + (uint32_t)a.nt * 128u;
    const uint32_t stage = MX_TILE_BYTES + a.xbytes;
    a.stages = (int)std::min<uint32_t>(4, (MXL_SMEM_MAX - 1024) / stage);
    a.sfcol = (uint32_t)a.nt;
    a.ncols = 32;
    while (a.ncols < a.sfcol + 24u * a.stages) a.ncols <<= 1;
    // A CTA's part of the SM's shared memory is at least its part of tensor memory,
    // so that CTAs that fit beside each other never wait for columns.
    const uint32_t smem = std::min(MXL_SMEM_MAX, std::max(1024 + a.stages * stage, a.ncols * 456u));
    const void *fn = type == MX_F32   ? (const void *)mx_linear_kernel<float>
                     : type == MX_F16 ? (const void *)mx_linear_kernel<__half>
                                      : (const void *)mx_linear_kernel<__nv_bfloat16>;
    cudaError_t r = ensure_smem_attr(fn, (int)smem);
    if (r == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((p.N + MX_TILE_M - 1) / MX_TILE_M), (unsigned)((p.B + a.nt - 1) / a.nt));
        cfg.blockDim = dim3(MXL_THREADS);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = lc.stream;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = lc.pdl ? 1 : 0;
        void *args[] = {&a};
        r = cudaLaunchKernelExC(&cfg, fn, args);
    }
    if (r != cudaSuccess) *e = r;
}

}  // namespace rk
