// q4.cu -- 4-bit matrices with group scales (layout: q4.cuh): packing, quantisation and its
// inverse, and the product with the few rows of a decode step.
#include <cstdio>
#include <cstring>

#include "../../include/rwkv7.h"
#include "q4.cuh"
#include "span.h"

namespace rk {

constexpr int Q4_THREADS = 256;

// ---------------------------------------------------------------------------
// The product with up to 16 rows of x.  The codes become 16-bit whole numbers (1024 + q less
// 1024 + zero in fp16, 128 + q in bf16: exact), the products of x and those are exact in fp32, and
// a group's sum is multiplied by its scale as it joins the row's.
//
// One CTA a SM takes a run of row tiles, and its 16 warps equal shares of those tiles' column
// tiles, counted through, so that all SMs and all warps have the same bytes to stream.  A
// warp fetches its own records six ahead into a ring of its own, with no barrier between warps: six
// of 16 warps are 100 KB in flight an SM.  x lies in shared memory, in the order in which the
// operand registers take it.  A share that ends inside a row tile leaves its part of the sum, and
// the parts are added in order at the end.
//
// What bounds it is the instructions next to the memory: 64 codes a lane take 72 to widen, and all in
// all a record takes a warp 155 of 187 at first (a masked-or written in C is two of them), 20 % of the
// tensor pipe.  2560 x 65536, one row: 19.2 us (89 MB, 13.2 at the copy rate; 2.6 before the first
// and about 3 after the last byte); 4096 x 16384, four rows: 10.1 (5.1).  One warp a row tile with loads to
// registers took 46 us for the former, operands kept by tiles of 64 columns 28.
// ---------------------------------------------------------------------------
// c = a b + c, or a b.
template <bool BF, bool FIRST>
__device__ __forceinline__ void q4_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
#define Q4_MMA(types)                                                                                                \
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." types ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "       \
                 "{%10,%11,%12,%13};"                                                                                \
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])                                                    \
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(FIRST ? 0.0f : c[0]),           \
                   "f"(FIRST ? 0.0f : c[1]), "f"(FIRST ? 0.0f : c[2]), "f"(FIRST ? 0.0f : c[3]))
    if constexpr (BF) Q4_MMA("bf16.bf16");
    else Q4_MMA("f16.f16");
#undef Q4_MMA
}

constexpr int QR_WARPS = 16;
constexpr int QR_AHEAD = 6;  // column tiles of each warp in flight

struct Q4RowsArgs {
    Q4LinearParams p;
    int chunk, chunks;  // column tiles whose x fits shared memory at once, and how many such runs
    int rows;           // row tiles of a CTA, at most
    uint32_t xat, slots, sums;  // where in shared memory x, the partial sums and their totals lie
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
    return v;
}

// A CTA takes a run of row tiles, its warps equal shares of their column tiles counted through.
// G: groups of a column tile.
template <bool BF, int NT, int G, bool ZERO>
__global__ void __launch_bounds__(32 * QR_WARPS, 1) q4_rows_kernel(const __grid_constant__ Q4RowsArgs a) {
    extern __shared__ __align__(16) char smem[];
    constexpr uint32_t RECORD = q4_record(Q4_COLS / G, ZERO), RING = QR_AHEAD * RECORD;
    constexpr uint32_t MORE = (RECORD - Q4_CODES) / 16;  // lanes that fetch scales and zeros
    constexpr int PART = 128 * NT;                       // sums of a row tile
    const Q4LinearParams &p = a.p;
    const Q4Matrix &m = p.w;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int r0 = (int)((int64_t)m.rt * blockIdx.x / gridDim.x), R = (int)((int64_t)m.rt * (blockIdx.x + 1) / gridDim.x) - r0;
    const int B = p.B;  // 8 NT at most
    const uint32_t base = smem_u32(smem), ring = base + warp * RING, mine = ring + lane * 16;
    float *slots = (float *)(smem + a.slots), *sums = (float *)(smem + a.sums);
    // Where a lane's x lies: a row's 128 columns are 256 bytes, the 64 of every second 32 columns
    // changed about in odd rows, so that eight lanes' 16 bytes are in different banks.  Rows past
    // the last: any row, their sums are not stored.
    uint32_t xeven[NT], xodd[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int row = min(8 * j + g, B - 1);
        xeven[j] = base + a.xat + row * 256 + t * 16 + (row & 1) * 64;
        xodd[j] = base + a.xat + row * 256 + t * 16 - (row & 1) * 64;
    }
    const uint32_t xstep = B * 256;
    for (int c = 0; c < a.chunks; ++c) {
        const int k0 = c * a.chunk, kc = min(a.chunk, m.kt - k0), U = R * kc;
        const int u0 = (int)((int64_t)U * warp / QR_WARPS), u1 = (int)((int64_t)U * (warp + 1) / QR_WARPS);
        int r = u0 / kc, k = u0 - r * kc;
        const uint8_t *src = m.data + ((int64_t)(r0 + r) * m.kt + k0 + k) * RECORD + lane * 16;
        const uint32_t skip = (uint32_t)(m.kt - kc) * RECORD;  // from a row tile's last to the next one's first
        int left = u1 - u0, run = min(left, kc - k);           // tiles to fetch, in all and one after another
        auto fetch = [&](uint32_t to) {
            if (run > 0) {
                cp16(mine + to, src);
                cp16(mine + to + 512, src + 512);
                if (lane < MORE) cp16(mine + to + Q4_CODES, src + Q4_CODES);
                src += RECORD;
                if (--run == 0) {
                    src += skip;
                    left -= kc - k, k = 0;
                    run = min(left, kc);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int n = run;  // tiles of the row tile at hand
        const int first = k;
        for (int i = 0; i < QR_AHEAD - 1; ++i) fetch(i * RECORD);
        // x of these columns
        for (int i = tid; i < kc * 16 * B; i += 32 * QR_WARPS) {
            const int kt = i / (16 * B), q = i - kt * 16 * B, row = q >> 4, col = (k0 + kt) * Q4_COLS + (q & 15) * 8;
            const uint16_t *x = (const uint16_t *)p.x + row * p.ldx;
            const uint32_t to = a.xat + (uint32_t)(kt * B + row) * 256 + ((q & 15) ^ (row & 1) * 4) * 16;
            if (p.xvec && col + 8 <= m.K) cp16(base + to, x + col);
            else *(uint4 *)(smem + to) = q4_x8(x, col, m.K);
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        if (u0 == u1)  // no tile, but a place among those of its row tile
            for (int i = lane; i < PART; i += 32) slots[(r + warp) * PART + i] = 0.0f;
        uint32_t at = 0, before = (QR_AHEAD - 1) * RECORD, xat = (uint32_t)first * xstep;
        for (int rest = u1 - u0; rest > 0; xat = 0, ++r) {
            float tot[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[j][i] = 0.0f;
            rest -= n;
            for (; n > 0; --n) {
                fetch(before);
                asm volatile("cp.async.wait_group %0;" ::"n"(QR_AHEAD - 1) : "memory");
                __syncwarp();
                float2 f[G];
                Q4Zero z[G];
                const uint32_t q0 = ring + g * 4 + at, z0 = ZERO ? ring + g * 2 + at : 0;
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const uint32_t s = lds4(q0 + Q4_CODES + 32 * i);
                    f[i] = __half22float2(*(const __half2 *)&s);
                    const uint32_t zz = ZERO ? lds2(z0 + Q4_CODES + 32 * G + 16 * i) : 0x0808u;
                    z[i] = q4_zero<BF>(zz & 0xFFu, zz >> 8);
                }
                float acc[NT][4];
                uint4 code;
                uint32_t xe[NT], xo[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) xe[j] = xeven[j] + xat, xo[j] = xodd[j] + xat;
#pragma unroll
                for (int h = 0; h < 4; ++h) {  // 32 columns
                    if (h % 2 == 0) code = lds16(mine + at + h * 256);
                    uint4 v[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) v[j] = lds16((h & 1 ? xo[j] : xe[j]) + h * 64);
                    const uint32_t word[2] = {h & 1 ? code.z : code.x, h & 1 ? code.w : code.y};
                    constexpr int PER = 4 / G;  // such parts of a group
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint32_t q[4];
                        q4_widen<BF>(word[w], z[h / PER], q);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const uint32_t x0 = w ? v[j].z : v[j].x, x1 = w ? v[j].w : v[j].y;
                            if (w == 0 && h % PER == 0) q4_mma<BF, true>(acc[j], q, x0, x1);
                            else q4_mma<BF, false>(acc[j], q, x0, x1);
                        }
                    }
                    if (h % PER == PER - 1) {
                        const float2 e = f[h / PER];
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            tot[j][0] = fmaf(e.x, acc[j][0], tot[j][0]), tot[j][1] = fmaf(e.x, acc[j][1], tot[j][1]);
                            tot[j][2] = fmaf(e.y, acc[j][2], tot[j][2]), tot[j][3] = fmaf(e.y, acc[j][3], tot[j][3]);
                        }
                    }
                }
                __syncwarp();  // read before its place is fetched into again, by the next turn
                before = at;
                at = at + RECORD == RING ? 0 : at + RECORD;
                xat += xstep;
            }
            n = min(rest, kc);
            // a row tile's share: rows g and g + 8, columns 2t and 2t + 1 of each eight
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float *o = slots + (r + warp) * PART + (8 * j + 2 * t) * 16 + g;
                o[0] = tot[j][0], o[16] = tot[j][1], o[8] = tot[j][2], o[24] = tot[j][3];
            }
        }
        __syncthreads();
        for (int i = tid; i < R * 16 * B; i += 32 * QR_WARPS) {
            const int b = i / (R * 16), n = i - b * R * 16, row = n >> 4;
            // the warps that have tiles row * kc and (row + 1) * kc - 1
            const int w0 = (int)(((int64_t)QR_WARPS * (row * kc + 1) - 1) / U), w1 = (int)(((int64_t)QR_WARPS * ((row + 1) * kc) - 1) / U);
            const float *q = slots + (row + w0) * PART + b * 16 + (n & 15);
            float v = 0.0f;
            for (int w = w0; w <= w1; ++w, q += PART) v += *q;
            if (a.chunks > 1) {
                if (c > 0) v += sums[i];
                if (c + 1 < a.chunks) {
                    sums[i] = v;
                    continue;
                }
            }
            if (r0 * 16 + n < m.N) q4_store(p, b, r0 * 16 + n, v);
        }
        if (c + 1 < a.chunks) __syncthreads();
    }
}

template <bool BF, int NT, bool ZERO>
static const void *q4_rows_fn(int group) {
    return group == 32   ? (const void *)q4_rows_kernel<BF, NT, 4, ZERO>
           : group == 64 ? (const void *)q4_rows_kernel<BF, NT, 2, ZERO>
                         : (const void *)q4_rows_kernel<BF, NT, 1, ZERO>;
}
template <bool BF, int NT>
static const void *q4_rows_fn(int group, bool zero) {
    return zero ? q4_rows_fn<BF, NT, true>(group) : q4_rows_fn<BF, NT, false>(group);
}

void launch_q4_rows(const Q4LinearParams &p, int xtype, cudaStream_t stream, cudaError_t *e) {
    static_assert(RWKV7_Q4_FEW_ROWS == 16, "two tiles of eight rows of x at most");
    const int nt = p.B <= 8 ? 1 : 2, group = p.w.group;
    const bool zero = p.w.zeros != 0, bf = xtype == MX_BF16;
    const void *fn = nt == 1 ? (bf ? q4_rows_fn<true, 1>(group, zero) : q4_rows_fn<false, 1>(group, zero))
                             : (bf ? q4_rows_fn<true, 2>(group, zero) : q4_rows_fn<false, 2>(group, zero));
    constexpr uint32_t most = 226 * 1024;
    Q4RowsArgs a;
    memset(&a, 0, sizeof a);
    a.p = p;
    const int B = p.B, limit = 32 / nt;
    const int ctas = p.w.rt < 152 ? p.w.rt : 152 * ((p.w.rt + 152 * limit - 1) / (152 * limit));
    a.rows = (p.w.rt + ctas - 1) / ctas;
    const uint32_t part = 512u * nt;
    a.slots = QR_WARPS * QR_AHEAD * q4_record(group, zero);
    a.xat = a.slots + (a.rows + QR_WARPS - 1) * part;
    const uint32_t room = most - a.xat, all = (uint32_t)a.rows * 16 * B * 4;
    a.chunk = p.w.kt, a.chunks = 1;
    if ((uint64_t)p.w.kt * 256 * B > room) {
        const int fit = (int)((room - all) / (256u * B));
        a.chunks = (p.w.kt + fit - 1) / fit;
        a.chunk = (p.w.kt + a.chunks - 1) / a.chunks;
        a.chunks = (p.w.kt + a.chunk - 1) / a.chunk;
    }
    const uint32_t end = a.xat + (uint32_t)a.chunk * 256 * B;
    a.sums = end;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(32 * QR_WARPS);
    cfg.dynamicSmemBytes = end + (a.chunks > 1 ? all : 0);
    cfg.stream = stream;
    void *args[] = {&a};
    cudaError_t r = ensure_smem_attr(fn, (int)most);
    if (r == cudaSuccess) r = cudaLaunchKernelExC(&cfg, fn, args);
    if (r != cudaSuccess) *e = r;
}

// ---------------------------------------------------------------------------
// Laying out, quantising, reading back.  Done once where weights are loaded.
// ---------------------------------------------------------------------------
// A lane's 16 bytes of half c of a tile from the codes q(row half, column).
template <typename Q>
__device__ __forceinline__ uint4 q4_words(int t, Q q) {
    uint32_t w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int c = 32 * (s >> 1) + 8 * t + 4 * (s & 1);
        w[s] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // pairs
            const int half = i & 1, k = c + 2 * (i >> 1);
            w[s] |= (q(half, k) & 15u) << (4 * i) | (q(half, k + 1) & 15u) << (4 * i + 16);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread takes a lane's words of half a tile (64 threads a tile), or the scale and zero of a
// row's group (16 * 128 / group).
__global__ void __launch_bounds__(Q4_THREADS) q4_pack_kernel(const uint8_t *values, int64_t ldv, const __half *scales,
                                                             int64_t lds, const uint8_t *zeros, int64_t ldz, Q4Matrix o) {
    const int of_tile = Q4_COLS / o.group, each = 64 + 16 * of_tile, groups = (o.K + o.group - 1) / o.group;
    const int64_t all = (int64_t)o.rt * o.kt * each;
    const uint32_t record = q4_record(o.group, o.zeros);
    for (int64_t i = (int64_t)blockIdx.x * Q4_THREADS + threadIdx.x; i < all; i += (int64_t)gridDim.x * Q4_THREADS) {
        const int64_t tile = i / each;
        const int j = (int)(i - tile * each), rt = (int)(tile / o.kt), kt = (int)(tile - (int64_t)rt * o.kt);
        uint8_t *at = o.data + tile * record;
        if (j < 64) {
            const int lane = j & 31, r0 = rt * 16 + (lane >> 2), k0 = kt * Q4_COLS + (j >> 5) * 64;
            ((uint4 *)at)[j] = q4_words(lane & 3, [&](int half, int k) -> uint32_t {
                const int r = r0 + 8 * half;
                return r < o.N && k0 + k < o.K ? values[r * ldv + k0 + k] : 8u;
            });
        } else {
            const int e = j - 64, r = rt * 16 + (e >> 1 & 7) + 8 * (e & 1), gr = kt * of_tile + (e >> 4);
            const bool in = r < o.N && gr < groups;
            ((__half *)(at + Q4_CODES))[e] = in ? scales[r * lds + gr] : __float2half_rn(0.0f);
            if (o.zeros) at[Q4_CODES + 32 * of_tile + e] = in ? zeros[r * ldz + gr] & 15u : 8u;
        }
    }
}

// CTA: a tile; a thread takes 16 neighbours of a row, a group's threads are neighbouring lanes.
template <int T>
__global__ void __launch_bounds__(128) q4_quantize_kernel(const typename MxElem<T>::type *x, int64_t ld, Q4Matrix o) {
    __shared__ uint8_t code[16][Q4_COLS + 4];
    const int tid = threadIdx.x, row = tid >> 3, seg = tid & 7;
    const int rt = blockIdx.x / o.kt, c0 = (blockIdx.x - rt * o.kt) * Q4_COLS;
    const int r = rt * 16 + row, k0 = c0 + seg * 16;
    float v[16], low = 0.0f, high = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float f = 0.0f;
        if (r < o.N && k0 + i < o.K) {
            if constexpr (T == MX_F32) f = x[r * ld + k0 + i];
            else if constexpr (T == MX_F16) f = __half2float(x[r * ld + k0 + i]);
            else f = __bfloat162float(x[r * ld + k0 + i]);
        }
        v[i] = f;
        top = max(top, __float_as_uint(f) & 0x7FFFFFFFu);
        low = fminf(low, f), high = fmaxf(high, f);
    }
    for (int off = 1; off < o.group / 16; off *= 2) {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
        high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, off));
    }
    const bool number = top < 0x7F800000u;
    const float span = o.zeros ? __fdiv_rn(__fsub_rn(high, low), 15.0f) : __fdiv_rn(__uint_as_float(top), 7.0f);
    const __half sh = number ? __float2half_rn(fminf(span, 65504.0f)) : __ushort_as_half(0x7E00);
    const float scale = __half2float(sh);
    const bool some = number && scale > 0.0f;
    float zero = 8.0f;
    if (o.zeros) zero = some ? fminf(fmaxf(rintf(__fdiv_rn(-low, scale)), 0.0f), 15.0f) : 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float q = some ? fminf(fmaxf(rintf(__fdiv_rn(v[i], scale)) + zero, 0.0f), 15.0f) : zero;
        code[row][seg * 16 + i] = (uint8_t)(int)(k0 + i < o.K ? q : 8.0f);
    }
    uint8_t *at = o.data + (int64_t)blockIdx.x * q4_record(o.group, o.zeros);
    if (seg % (o.group / 16) == 0) {
        const int e = seg * 16 / o.group * 16 + (row & 7) * 2 + (row >> 3);
        ((__half *)(at + Q4_CODES))[e] = sh;
        if (o.zeros) at[Q4_CODES + 32 * (Q4_COLS / o.group) + e] = (uint8_t)(int)zero;
    }
    __syncthreads();
    if (tid < 64) {
        const int lane = tid & 31, g = lane >> 2;
        ((uint4 *)at)[tid] = q4_words(lane & 3, [&](int half, int k) -> uint32_t {
            return code[g + 8 * half][(tid >> 5) * 64 + k];
        });
    }
}

template <int T>
__global__ void __launch_bounds__(Q4_THREADS) q4_dequantize_kernel(const Q4Matrix m, typename MxElem<T>::type *y, int64_t ld) {
    const int64_t all = (int64_t)m.rt * m.kt * 64;
    const uint32_t record = q4_record(m.group, m.zeros);
    for (int64_t i = (int64_t)blockIdx.x * Q4_THREADS + threadIdx.x; i < all; i += (int64_t)gridDim.x * Q4_THREADS) {
        const int j = (int)(i & 63), lane = j & 31, g = lane >> 2, t = lane & 3;
        const int rt = (int)((i >> 6) / m.kt), kt = (int)((i >> 6) - (int64_t)rt * m.kt);
        const uint8_t *at = m.data + (i >> 6) * record;
        const uint4 code = ((const uint4 *)at)[j];
        const uint32_t word[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int c = (j >> 5) * 64 + 32 * (s >> 1) + 8 * t + 4 * (s & 1), gr = c / m.group;
            const float2 f = __half22float2(((const __half2 *)(at + Q4_CODES))[gr * 8 + g]);
            const uint32_t z = m.zeros ? ((const uint16_t *)(at + Q4_CODES + 32 * (Q4_COLS / m.group)))[gr * 8 + g] : 0x0808u;
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // half e & 1, column e >> 1
                const int r = rt * 16 + g + 8 * (e & 1), k = kt * Q4_COLS + c + (e >> 1);
                if (r >= m.N || k >= m.K) continue;
                const uint32_t q = word[s] >> (4 * (e & 1) + 8 * (e >> 2) + 16 * (e >> 1 & 1)) & 15u;
                y[r * ld + k] = MxElem<T>::down((e & 1 ? f.y : f.x) * (float)((int)q - (int)(e & 1 ? z >> 8 : z & 0xFFu)));
            }
        }
    }
}

}  // namespace rk

// ---------------------------------------------------------------------------
// C entry points
// ---------------------------------------------------------------------------
using namespace rk;
namespace {

thread_local char g_q4_msg[192];

int q4_fail(const char **err_msg, int code, const char *fmt, long long a = 0, long long b = 0) {
    snprintf(g_q4_msg, sizeof g_q4_msg, fmt, a, b);
    if (err_msg) *err_msg = g_q4_msg;
    return code;
}
int q4_done(const char **err_msg, const char *what, cudaError_t e) {
    if (e == cudaSuccess) return RWKV7_OK;
    snprintf(g_q4_msg, sizeof g_q4_msg, "%s: %s", what, cudaGetErrorString(e));
    if (err_msg) *err_msg = g_q4_msg;
    return RWKV7_ECUDA;
}

int q4_size(const char **err_msg, int64_t rows, int64_t cols, int32_t group) {
    if (rows < 1 || cols < 1 || rows > RWKV7_MX_MAX_DIM || cols > RWKV7_MX_MAX_DIM)
        return q4_fail(err_msg, RWKV7_EINVAL, "rows and cols must be 1 .. 2^24 (rows=%lld, cols=%lld)", rows, cols);
    if (group != 32 && group != 64 && group != 128)
        return q4_fail(err_msg, RWKV7_EINVAL, "a group of %lld columns: 32, 64 or 128", group);
    const int64_t tiles = (rows + Q4_ROWS - 1) / Q4_ROWS * ((cols + Q4_COLS - 1) / Q4_COLS);
    if (tiles > INT32_MAX) return q4_fail(err_msg, RWKV7_EINVAL, "%lld rows of %lld columns are too many", rows, cols);
    return RWKV7_OK;
}
Q4Matrix q4_matrix(const void *q4, int64_t rows, int64_t cols, int32_t group, bool zeros) {
    Q4Matrix m;
    m.data = static_cast<uint8_t *>(const_cast<void *>(q4));
    m.N = (int)rows, m.K = (int)cols, m.group = group, m.zeros = zeros;
    m.rt = (int)((rows + Q4_ROWS - 1) / Q4_ROWS), m.kt = (int)((cols + Q4_COLS - 1) / Q4_COLS);
    return m;
}
MxSpan q4_span(const void *q4, int64_t rows, int64_t cols, int32_t group, bool zeros) {
    return MxSpan(q4, 1, (int64_t)rwkv7_q4_bytes(rows, cols, group, zeros), 0, 1);
}
// Rows of a type against a matrix.
int q4_rows_check(const char **err_msg, const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, const void *q4,
                  int32_t group, bool zeros) {
    if (dtype < RWKV7_F32 || dtype > RWKV7_BF16) return q4_fail(err_msg, RWKV7_EINVAL, "unknown dtype %lld", dtype);
    if (rows > 1 && ld < cols) return q4_fail(err_msg, RWKV7_EINVAL, "row stride %lld is below cols=%lld", ld, cols);
    if (!x || !q4) return q4_fail(err_msg, RWKV7_EINVAL, "null pointer argument");
    const int size = dtype == RWKV7_F32 ? 4 : 2;
    if ((uintptr_t)x % size) return q4_fail(err_msg, RWKV7_EINVAL, "the rows' pointer is not aligned to its type");
    if ((uintptr_t)q4 & 15u) return q4_fail(err_msg, RWKV7_EINVAL, "a 4-bit matrix must be 16-byte aligned");
    if (mx_share(MxSpan(x, rows, cols, ld, size), q4_span(q4, rows, cols, group, zeros)))
        return q4_fail(err_msg, RWKV7_EINVAL, "the rows and the 4-bit matrix overlap");
    return RWKV7_OK;
}
unsigned q4_grid(int64_t threads) {
    const int64_t blocks = (threads + Q4_THREADS - 1) / Q4_THREADS;
    return (unsigned)(blocks < 152 * 64 ? blocks : 152 * 64);
}

}  // namespace

extern "C" {

size_t rwkv7_q4_bytes(int64_t rows, int64_t cols, int32_t group, int32_t zeros) {
    if (q4_size(nullptr, rows, cols, group)) return 0;
    const size_t rt = (size_t)((rows + Q4_ROWS - 1) / Q4_ROWS), kt = (size_t)((cols + Q4_COLS - 1) / Q4_COLS);
    return rt * kt * q4_record(group, zeros != 0);
}

int rwkv7_q4_pack(const uint8_t *d_values, int64_t ldv, const void *d_scales, int64_t lds, const uint8_t *d_zeros,
                  int64_t ldz, int64_t rows, int64_t cols, int32_t group, void *d_q4, void *cuda_stream,
                  const char **err_msg) {
    if (err_msg) *err_msg = "";
    if (int rc = q4_size(err_msg, rows, cols, group)) return rc;
    const int64_t ng = (cols + group - 1) / group;
    if (rows > 1 && (ldv < cols || lds < ng || (d_zeros && ldz < ng)))
        return q4_fail(err_msg, RWKV7_EINVAL, "a row stride is below the row's %lld values or %lld groups", cols, ng);
    if (!d_values || !d_scales || !d_q4) return q4_fail(err_msg, RWKV7_EINVAL, "null pointer argument");
    if ((uintptr_t)d_scales & 1u) return q4_fail(err_msg, RWKV7_EINVAL, "the scales' pointer is not aligned to its type");
    if ((uintptr_t)d_q4 & 15u) return q4_fail(err_msg, RWKV7_EINVAL, "a 4-bit matrix must be 16-byte aligned");
    const MxSpan m = q4_span(d_q4, rows, cols, group, d_zeros != nullptr);
    if (mx_share(MxSpan(d_values, rows, cols, ldv, 1), m) || mx_share(MxSpan(d_scales, rows, ng, lds, 2), m) ||
        (d_zeros && mx_share(MxSpan(d_zeros, rows, ng, ldz, 1), m)))
        return q4_fail(err_msg, RWKV7_EINVAL, "the matrix overlaps what it is laid out from");
    const Q4Matrix o = q4_matrix(d_q4, rows, cols, group, d_zeros != nullptr);
    const int64_t threads = (int64_t)o.rt * o.kt * (64 + 16 * (Q4_COLS / group));
    q4_pack_kernel<<<q4_grid(threads), Q4_THREADS, 0, static_cast<cudaStream_t>(cuda_stream)>>>(
        d_values, ldv, static_cast<const __half *>(d_scales), lds, d_zeros, ldz, o);
    return q4_done(err_msg, "packing", cudaGetLastError());
}

int rwkv7_q4_quantize(const void *d_x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, int32_t group, int32_t zeros,
                      void *d_q4, void *cuda_stream, const char **err_msg) {
    if (err_msg) *err_msg = "";
    if (int rc = q4_size(err_msg, rows, cols, group)) return rc;
    if (int rc = q4_rows_check(err_msg, d_x, dtype, rows, cols, ld, d_q4, group, zeros != 0)) return rc;
    const Q4Matrix o = q4_matrix(d_q4, rows, cols, group, zeros != 0);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)o.rt * (unsigned)o.kt);
    cfg.blockDim = dim3(128);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cudaError_t e;
    if (dtype == RWKV7_F32) e = cudaLaunchKernelEx(&cfg, q4_quantize_kernel<MX_F32>, (const float *)d_x, ld, o);
    else if (dtype == RWKV7_F16) e = cudaLaunchKernelEx(&cfg, q4_quantize_kernel<MX_F16>, (const __half *)d_x, ld, o);
    else e = cudaLaunchKernelEx(&cfg, q4_quantize_kernel<MX_BF16>, (const __nv_bfloat16 *)d_x, ld, o);
    return q4_done(err_msg, "quantising", e);
}

int rwkv7_q4_dequantize(const void *d_q4, int64_t rows, int64_t cols, int32_t group, int32_t zeros, void *d_y, int32_t dtype,
                        int64_t ld, void *cuda_stream, const char **err_msg) {
    if (err_msg) *err_msg = "";
    if (int rc = q4_size(err_msg, rows, cols, group)) return rc;
    if (int rc = q4_rows_check(err_msg, d_y, dtype, rows, cols, ld, d_q4, group, zeros != 0)) return rc;
    const Q4Matrix m = q4_matrix(d_q4, rows, cols, group, zeros != 0);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(q4_grid((int64_t)m.rt * m.kt * 64));
    cfg.blockDim = dim3(Q4_THREADS);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cudaError_t e;
    if (dtype == RWKV7_F32) e = cudaLaunchKernelEx(&cfg, q4_dequantize_kernel<MX_F32>, m, (float *)d_y, ld);
    else if (dtype == RWKV7_F16) e = cudaLaunchKernelEx(&cfg, q4_dequantize_kernel<MX_F16>, m, (__half *)d_y, ld);
    else e = cudaLaunchKernelEx(&cfg, q4_dequantize_kernel<MX_BF16>, m, (__nv_bfloat16 *)d_y, ld);
    return q4_done(err_msg, "reading back", e);
}

size_t rwkv7_q4_room_bytes(int64_t B, int64_t K) {
    if (B < 0 || K < 1 || B > RWKV7_MX_MAX_DIM || K > RWKV7_MX_MAX_DIM) return 0;
    return (size_t)B * (size_t)((K + 7) / 8) * 16;
}

int rwkv7_q4_linear(const void *d_x, int32_t x_dtype, int64_t ldx, int64_t B, const void *d_w_q4, int64_t N, int64_t K,
                    int32_t group, int32_t zeros, void *d_y, int32_t y_dtype, int64_t ldy, int32_t activation, void *d_room,
                    uint32_t *d_err, void *cuda_stream, const char **err_msg) {
    if (err_msg) *err_msg = "";
    if (int rc = q4_size(err_msg, N, K, group)) return rc;
    if (B < 0 || B > RWKV7_MX_MAX_DIM) return q4_fail(err_msg, RWKV7_EINVAL, "B=%lld is outside 0 .. 2^24", B);
    if (x_dtype != RWKV7_F16 && x_dtype != RWKV7_BF16)
        return q4_fail(err_msg, RWKV7_EINVAL, "x must be fp16 or bf16 (dtype %lld)", x_dtype);
    if (y_dtype < RWKV7_F32 || y_dtype > RWKV7_BF16)
        return q4_fail(err_msg, RWKV7_EINVAL, "unknown output dtype %lld", y_dtype);
    if (activation != RWKV7_ACT_NONE && activation != RWKV7_ACT_RELU2)
        return q4_fail(err_msg, RWKV7_EINVAL, "unknown activation %lld", activation);
    if (B > 1 && ldx < K) return q4_fail(err_msg, RWKV7_EINVAL, "row stride %lld is below K=%lld", ldx, K);
    if (B > 1 && ldy < N) return q4_fail(err_msg, RWKV7_EINVAL, "output row stride %lld is below N=%lld", ldy, N);
    if (B > ((int64_t)1 << 38) / N) return q4_fail(err_msg, RWKV7_EINVAL, "an output of %lld x %lld is too large", B, N);
    if (B == 0) return RWKV7_OK;
    if (!d_x || !d_w_q4 || !d_y || !d_err) return q4_fail(err_msg, RWKV7_EINVAL, "null pointer argument");
    if ((uintptr_t)d_x & 1u) return q4_fail(err_msg, RWKV7_EINVAL, "the rows' pointer is not aligned to its type");
    if ((uintptr_t)d_y % (y_dtype == RWKV7_F32 ? 4 : 2))
        return q4_fail(err_msg, RWKV7_EINVAL, "the output pointer is not aligned to its type");
    if ((uintptr_t)d_w_q4 & 15u) return q4_fail(err_msg, RWKV7_EINVAL, "a 4-bit matrix must be 16-byte aligned");
    const MxSpan y(d_y, B, N, ldy, y_dtype == RWKV7_F32 ? 4 : 2);
    if (mx_share(y, MxSpan(d_x, B, K, ldx, 2)) || mx_share(y, q4_span(d_w_q4, N, K, group, zeros != 0)))
        return q4_fail(err_msg, RWKV7_EINVAL, "the output overlaps x or the matrix");
    Q4LinearParams p;
    memset(&p, 0, sizeof p);
    p.w = q4_matrix(d_w_q4, N, K, group, zeros != 0);
    p.x = d_x, p.ldx = ldx, p.y = d_y, p.ldy = ldy;
    p.B = (int)B, p.act = activation, p.ytype = y_dtype;
    p.xvec = ((uintptr_t)d_x & 15u) == 0 && (B == 1 || ldx % 8 == 0);
    p.room = d_room, p.err = d_err;
    cudaError_t e = cudaSuccess;
    // Up to 16 rows a warp's own products keep up with the memory; x in every SM's shared memory is what
    // they pay, copied by each and taken in turns from 80 to 110 KB on.  Past 256 KB of it the other kernel is
    // faster, unless it needs a second round of tiles: us by warps / by tcgen05, 4096 x 16384 in groups of 128: 4 rows
    // 13.1 / 16.8, 8 rows 17.6 / 16.9, 12 rows 23.7 / 17.3; 2560 x 10240, 64: 8 rows 11.7 / 11.7, 16 rows 19.9 /
    // 12.0; 65536 x 2560, 64: 16 rows 35.3 / 42.8.  Near the border the sizes alone do not tell: 128 KB of x by
    // 16384 x 4096, 16 rows, takes 18.9 / 16.3 in groups of 128 and 18.6 / 19.0 in groups of 64, by warps either way.
    if (B <= RWKV7_Q4_FEW_ROWS && (B * K <= RWKV7_Q4_FEW_VALUES || N > 152 * 128)) {
        launch_q4_rows(p, x_dtype, static_cast<cudaStream_t>(cuda_stream), &e);
    } else {
        if (!p.xvec) {
            const MxSpan room(d_room, 1, (int64_t)rwkv7_q4_room_bytes(B, K), 0, 1);
            if (!d_room || ((uintptr_t)d_room & 15u))
                return q4_fail(err_msg, RWKV7_EINVAL, "rows off the 16-byte grid need room, 16-byte aligned");
            if (mx_share(room, y) || mx_share(room, MxSpan(d_x, B, K, ldx, 2)) ||
                mx_share(room, q4_span(d_w_q4, N, K, group, zeros != 0)))
                return q4_fail(err_msg, RWKV7_EINVAL, "the room overlaps x, the matrix or the output");
        }
        launch_q4_tc(p, x_dtype, static_cast<cudaStream_t>(cuda_stream), &e);
    }
    return q4_done(err_msg, "4-bit product", e);
}

}  // extern "C"
