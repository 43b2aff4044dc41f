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
// A tile is 128 outputs x nt tokens over all of K.  One CTA a SM walks its share of
// the tiles; where there are fewer tiles than SMs the CTAs of a cluster share one
// tile's column tiles and add their partial sums through each other's shared memory,
// in rank order, so a result does not depend on timing.
//   warp 0       bulk copies of whole tiles of 128 x 256 -- codes and powers as they
//                lie, no tensor map -- into a ring of stages that runs on across
//                tiles; the weights of the first stages are requested before the wait
//                for the kernel that quantises x
//   warp 1       per stage: powers from shared into tensor memory (tcgen05.cp, in
//                order before the products of the same thread), four products
//   warps 2-17   the accumulator to registers, then, while the next tile's products
//                run, activation and y; lane = output, so a warp's store of one token
//                covers 32 neighbouring outputs
// Up to 16 rows of x of moderate length are quantised by these warps of every CTA
// themselves, into shared memory where they stay, while the first weights are on
// their way.  Not where y shares memory with them: a CTA's y would come under the rows
// that a later one has still to read.  A kernel of their own reads them all before
// any y is stored.
//
// Each stage has columns of its own for its powers: they are overwritten only
// after the commit that also frees the stage's shared memory.  A CTA takes all of
// tensor memory; its 226 KB of shared memory keep any other CTA that uses tensor
// memory off the SM, so none waits for columns that a waiting CTA holds.
//
// What bounds it (2.07 GHz): a stage of 128 outputs x 256 tokens x 256 columns takes
// 368 ns; its copies alone (52 KB out of L2 on every SM, 24 TB/s) take 332, its
// products and powers alone 342 (253 issued back to back; waits for stages that spin
// without ever looking at the clock give 303, but 363 together with the copies), so
// both sides are near their limits.  5.1 PFLOP/s over a 7.2B prefill key
// (4096 x 4096 x 16384, 108 us, 1365 W of 1400 when kept up).  128 tokens a tile (36 KB
// a stage for half the products) took 160 us there.  A single row of the 2.9B head
// streams 89 MB of weights in 18.6 us: 13.2 at the memory's rate, the rest before the
// first bytes arrive (2.3 us) and after the last.
// A tile that four CTAs share spends 4 us on its partial sums, 2.6 of them because
// they lie on other SMs (256 tokens; storing them there instead of fetching them took
// longer).
#include <algorithm>
#include <atomic>
#include <mutex>

#include "mx.cuh"

namespace rk {

constexpr int MXL_EPI_WARPS = 16;
constexpr int MXL_EPI_THREADS = 32 * MXL_EPI_WARPS;
constexpr int MXL_THREADS = 64 + MXL_EPI_THREADS;
constexpr int MXL_MAX_STAGES = 10;
constexpr int MXL_MAX_SPLIT = 8;  // CTAs of a portable cluster
constexpr uint32_t MXL_SMEM_MAX = 226 * 1024;  // a CTA's dynamic part
constexpr uint32_t MXL_SF = 24;  // tensor memory columns of a stage's powers: 8 of w, 2 x 8 of x
constexpr int MXL_TOKENS = 256;  // of a tile, at most
constexpr int MXL_CHUNKS = MXL_TOKENS / 16 / (MXL_EPI_WARPS / 4);  // of 16 tokens, that an epilogue warp holds

struct MxLinearArgs {
    MxLinearParams p;
    int kt;           // column tiles
    int nt;           // tokens of a full tile, a multiple of 16
    int rtiles;       // tiles along the outputs
    int tiles;        // all tiles, outputs fastest
    int stages;       // of the ring
    int split;        // CTAs of a cluster, which share one tile's column tiles
    int pack;         // y's rows allow stores of two (16-bit types) or four (split) neighbours
    uint32_t stage_bytes;
    uint32_t xres;    // x quantised here: where in shared memory its records lie; 0: x comes through the ring
    uint32_t ncols;   // tensor memory columns
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
    return 1u << 7 | 1u << 10 | (uint32_t)(N >> 3) << 17 | 1u << 23 | 1u << 27 | (uint32_t)half << 5 |
           (uint32_t)half << 30;
}

// 32 lanes x 16 columns on their way to v, which holds them after tmem_wait.
__device__ __forceinline__ void tmem_ask16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
#define MXL_16(v) "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), \
                  "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
__device__ __forceinline__ void tmem_wait(float (&v)[4][16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : MXL_16(v[0]), MXL_16(v[1]), MXL_16(v[2]), MXL_16(v[3])::"memory");
}
#undef MXL_16
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
// One stage: its powers into tensor memory, then `ni` products of 64 columns each.
// XC: tensor memory columns of x's powers for 128 columns of K (4 a record of 128
// tokens); off: the one of them in which the tile's first token lies.
template <int XC>
__device__ __forceinline__ void issue_stage(uint32_t tmem, uint32_t sw, uint32_t sx, uint32_t sfa, uint32_t sfb,
                                            uint32_t off, uint32_t id0, uint32_t id1, bool add, int ni) {
    tmem_cp_powers(sfa, sdesc_powers(sw));
    tmem_cp_powers(sfb, sdesc_powers(sx + MX_SCALE_BYTES));
    if (XC == 8) tmem_cp_powers(sfb + 4, sdesc_powers(sx));
    tmem_cp_powers(sfa + 4, sdesc_powers(sw + 512));
    tmem_cp_powers(sfb + XC, sdesc_powers(sx + MX_SCALE_BYTES + 512));
    if (XC == 8) tmem_cp_powers(sfb + XC + 4, sdesc_powers(sx + 512));
    sfb += off;
    const uint64_t da = sdesc_k128(sw + MX_SCALE_BYTES), db = sdesc_k128(sx + 2 * MX_SCALE_BYTES);
    if (ni == 4) {
        mma_mxf4(tmem, da, db, id0, sfa, sfb, add);
        mma_mxf4(tmem, da + 2, db + 2, id1, sfa, sfb, 1u);
        mma_mxf4(tmem, da + 4, db + 4, id0, sfa + 4, sfb + XC, 1u);
        mma_mxf4(tmem, da + 6, db + 6, id1, sfa + 4, sfb + XC, 1u);
    } else {
        mma_mxf4(tmem, da, db, id0, sfa, sfb, add);
        if (ni > 1) mma_mxf4(tmem, da + 2, db + 2, id1, sfa, sfb, 1u);
        if (ni > 2) mma_mxf4(tmem, da + 4, db + 4, id0, sfa + 4, sfb + XC, 1u);
    }
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four floats at this CTA's shared address `at` in the cluster's CTA `rank`.
__device__ __forceinline__ float4 ld_cluster(uint32_t at, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 t;\n\tmapa.shared::cluster.u32 t, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [t];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(at), "r"(rank)
        : "memory");
    return v;
}

__device__ __forceinline__ float mx_act(float v, int act) {
    return act ? (v > 0.0f ? v * v : (v != v ? v : 0.0f)) : v;
}
template <typename O>
struct MxOut;
template <>
struct MxOut<float> {
    static __device__ __forceinline__ float one(float v) { return v; }
};
template <>
struct MxOut<__half> {
    static __device__ __forceinline__ __half one(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ uint32_t two(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *(const uint32_t *)&h;
    }
};
template <>
struct MxOut<__nv_bfloat16> {
    static __device__ __forceinline__ __nv_bfloat16 one(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ uint32_t two(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *(const uint32_t *)&h;
    }
};

// Sixteen tokens (from column c of the tile, of `rows`) of a warp's 32 outputs, lane
// n's in v.  16-bit types: neighbouring lanes trade halves, so that each stores two
// outputs of every other token.
template <typename O>
__device__ __forceinline__ void store16(O *y, int64_t ldy, int c, int rows, int n, int N, bool pack, int act,
                                        float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = mx_act(v[j], act);
    if constexpr (sizeof(O) == 2) {
        if (pack) {
            const int odd = threadIdx.x & 1;
            O *z = y + n - odd + (int64_t)(c + odd) * ldy;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                const uint32_t w = odd ? MxOut<O>::two(got, v[j + 1]) : MxOut<O>::two(v[j], got);
                if (c + j + odd < rows) {
                    if ((n | 1) < N) *(uint32_t *)(z + (int64_t)j * ldy) = w;
                    else if ((n & ~1) < N) z[(int64_t)j * ldy] = MxOut<O>::one(odd ? got : v[j]);
                }
            }
            return;
        }
    }
    if (n < N) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (c + j < rows) y[n + (int64_t)(c + j) * ldy] = MxOut<O>::one(v[j]);
    }
}
// Four neighbouring outputs from n on of one token.
template <typename O>
__device__ __forceinline__ void store4(O *y, int n, int N, bool pack, int act, float4 s) {
    const float v[4] = {mx_act(s.x, act), mx_act(s.y, act), mx_act(s.z, act), mx_act(s.w, act)};
    if (pack && n + 3 < N) {
        if constexpr (sizeof(O) == 2)
            *(uint2 *)(y + n) = make_uint2(MxOut<O>::two(v[0], v[1]), MxOut<O>::two(v[2], v[3]));
        else
            *(float4 *)(y + n) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < N) y[n + j] = MxOut<O>::one(v[j]);
    }
}

constexpr uint32_t MXL_XREC = MX_SCALE_BYTES + 16 * 128;  // x's record of up to 16 rows x 256 columns
constexpr int MXL_XLINES = 4;                             // lines of x that an epilogue warp quantises, at most

// Epilogue warp `w`'s share of the B x kn lines (a line: 256 columns of a row) from
// column tile k0 on, into records at xres.
template <int T>
__device__ __forceinline__ void quantize_x(const MxLinearParams &p, uint8_t *xres, int k0, int kn, int w, int lane) {
    using L = MxElem<T>;
    using E = typename L::type;
    typename L::Eight u[MXL_XLINES];
#pragma unroll
    for (int i = 0; i < MXL_XLINES; ++i) {
        const int line = w + i * MXL_EPI_WARPS;
        if (line >= p.B * kn) break;
        const int k = line / p.B, r = line - k * p.B, c = (k0 + k) * MX_TILE_K + lane * 8;
        const E *src = (const E *)p.rows + r * p.ldr + c;
        if (p.rvec && c + 8 <= p.K) {
            L::load(u[i], src);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) L::set(u[i], j, c + j < p.K ? src[j] : L::down(0.0f));
        }
    }
#pragma unroll
    for (int i = 0; i < MXL_XLINES; ++i) {
        const int line = w + i * MXL_EPI_WARPS;
        if (line >= p.B * kn) break;
        const int k = line / p.B, r = line - k * p.B, blk = lane >> 2;
        uint8_t *rec = xres + k * MXL_XREC;
        uint32_t powers;
        uint8_t *code = rec + MX_SCALE_BYTES + r * 128 + ((blk ^ (r & 7)) << 4) + (lane & 3) * 4;
        *(uint32_t *)code = mx4_line<T>(u[i], powers);
        if ((lane & 15) == 0) *(uint32_t *)(rec + (blk >> 2) * 512 + r * 16) = powers;
    }
}

// Position in the ring: stage and the parity of its current use.
struct MxRing {
    int st = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++st == stages) st = 0, parity ^= 1u;
    }
};

// A tile: its rows of w, its tokens, and how many rows of x's one or two records of
// 128 hold them, padded to 16.  Tiles of 64 tokens start in the middle of every other
// record (off = 64), larger ones where a record does.
struct MxTile {
    int rt, b0, rows, npad, off, r0, r1;
    __device__ __forceinline__ MxTile(const MxLinearArgs &a, int t) {
        const int bt = t / a.rtiles;
        rt = t - bt * a.rtiles;
        b0 = bt * a.nt;
        rows = min(a.nt, a.p.B - b0);
        npad = (rows + 15) & ~15;
        off = b0 & (MX_TILE_M - 1);
        r0 = min(npad, MX_TILE_M);
        r1 = npad - r0;
    }
};

// The products of one tile, by a whole warp: what the instructions take stays
// uniform over it, and one elected lane issues them.  (Issued under a branch on the
// lane index, with a division for the ring position, a stage took 1.5 times as long.)
template <int XC>
__device__ __forceinline__ bool issue_tile(const MxTile &t, uint32_t tmem, uint32_t ring0, uint32_t x0, uint32_t sf0,
                                           uint32_t stage_bytes, int S, int kn, int last, MxRing &ring, uint64_t *full,
                                           uint64_t *empty, uint64_t *acc_full, volatile uint32_t *abort_flag) {
    const uint32_t id0 = idesc_mxf4(t.npad, 0), id1 = idesc_mxf4(t.npad, 1), off = (uint32_t)t.off >> 5;
    const bool leader = elect_one();
    for (int k = 0; k < kn; ++k) {
        if (!mbar_wait(&full[ring.st], ring.parity, abort_flag)) return false;
        tc_fence_after();
        const uint32_t sw = ring0 + (uint32_t)ring.st * stage_bytes, sfa = sf0 + (uint32_t)ring.st * MXL_SF;
        const uint32_t sx = x0 ? x0 + (uint32_t)k * MXL_XREC : sw + MX_TILE_BYTES;
        if (leader) {
            issue_stage<XC>(tmem, sw, sx, sfa, sfa + 8u, off, id0, id1, k > 0, k + 1 < kn ? 4 : last);
            mma_commit(&empty[ring.st]);
            if (k + 1 == kn) mma_commit(acc_full);
        }
        __syncwarp();
        ring.next(S);
    }
    return true;
}

template <typename O>
__global__ void __launch_bounds__(MXL_THREADS, 1) mx_linear_kernel(const __grid_constant__ MxLinearArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[MXL_MAX_STAGES], empty[MXL_MAX_STAGES], acc_full, acc_empty, x_ready;
    __shared__ uint32_t tmem_slot, s_abort;
    uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = a.stages, split = a.split;
    const int first = blockIdx.x / split, rank = blockIdx.x - first * split, step = gridDim.x / split;
    const int k0 = rank * a.kt / split, kn = (rank + 1) * a.kt / split - k0;  // this CTA's column tiles
    volatile uint32_t *abort_flag = &s_abort;

    auto load_w = [&](const MxTile &t, int k, int st) {
        const uint32_t xbytes = MX_SCALE_BYTES * (t.r1 ? 2 : 1) + (uint32_t)t.npad * 128u;
        mbar_expect_tx(&full[st], MX_TILE_BYTES + (a.xres ? 0u : xbytes));
        bulk_g2s(base + st * a.stage_bytes, a.p.w + ((int64_t)t.rt * a.kt + k0 + k) * MX_TILE_BYTES, MX_TILE_BYTES,
                 &full[st]);
    };
    const int npre = min(S, kn);  // stages of the first tile whose weights are requested at once
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_init(&acc_empty, MXL_EPI_WARPS);
        mbar_init(&x_ready, MXL_EPI_WARPS);
        s_abort = 0u;
        fence_barrier_init();
        const MxTile t(a, first);
        for (int k = 0; k < npre; ++k) load_w(t, k, k);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, a.ncols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

    if (warp == 0) {
        if (lane == 0) {
            auto load_x = [&](const MxTile &t, int k, int st) {
                if (a.xres) return;
                // powers of the second record, powers of the first, codes of both
                uint8_t *to = base + st * a.stage_bytes + MX_TILE_BYTES;
                const uint8_t *x0 = a.p.x + ((int64_t)(t.b0 / MX_TILE_M) * a.kt + k0 + k) * MX_TILE_BYTES;
                const uint32_t n0 = (uint32_t)t.r0 * 128u, n1 = (uint32_t)t.r1 * 128u;
                if (t.off == 0) {
                    bulk_g2s(to + MX_SCALE_BYTES, x0, MX_SCALE_BYTES + n0, &full[st]);
                } else {
                    bulk_g2s(to + MX_SCALE_BYTES, x0, MX_SCALE_BYTES, &full[st]);
                    bulk_g2s(to + 2 * MX_SCALE_BYTES, x0 + MX_SCALE_BYTES + t.off * 128, n0, &full[st]);
                }
                if (n1) {
                    const uint8_t *x1 = x0 + (int64_t)a.kt * MX_TILE_BYTES;
                    bulk_g2s(to, x1, MX_SCALE_BYTES, &full[st]);
                    bulk_g2s(to + 2 * MX_SCALE_BYTES + n0, x1 + MX_SCALE_BYTES, n1, &full[st]);
                }
            };
            {
                const MxTile t(a, first);
                pdl_wait();
                for (int k = 0; k < npre; ++k) load_x(t, k, k);
            }
            MxRing ring;
            int q = 0;
            bool ok = true;
            for (int i = first; i < a.tiles && ok; i += step) {
                const MxTile t(a, i);
                for (int k = 0; k < kn; ++k, ++q, ring.next(S)) {
                    if (q < npre) continue;
                    if (q >= S && !mbar_wait(&empty[ring.st], ring.parity ^ 1u, abort_flag)) {
                        *abort_flag = 1u;
                        atomicOr(a.p.err, ERR_TIMEOUT);
                        ok = false;
                        break;
                    }
                    load_w(t, k, ring.st);
                    load_x(t, k, ring.st);
                }
            }
            // no copy may be in flight when the CTA ends
            for (int j = max(0, q - S); j < q; ++j)
                if (!mbar_wait_any(&full[j % S], (uint32_t)(j / S) & 1u)) break;
        }
    } else if (warp == 1) {
        bool ok = true;
        int n = 0;
        MxRing ring;
        // a last tile of K % 256 columns: the instructions past them would add zeros
        const int last = min(4, (a.p.K - (k0 + kn - 1) * MX_TILE_K + 63) / 64);
        const uint32_t x0 = a.xres ? smem_u32(base + a.xres) - MX_SCALE_BYTES : 0u;
        if (a.xres) ok = mbar_wait(&x_ready, 0u, abort_flag);
        const uint32_t ring0 = smem_u32(base), sf0 = tmem + (uint32_t)a.nt;
        for (int i = first; i < a.tiles && ok; i += step, ++n) {
            const MxTile t(a, i);
            if (n > 0 && !mbar_wait(&acc_empty, (uint32_t)(n - 1) & 1u, abort_flag)) {
                ok = false;
                break;
            }
            ok = t.r1 ? issue_tile<8>(t, tmem, ring0, x0, sf0, a.stage_bytes, S, kn, last, ring, full, empty, &acc_full,
                                      abort_flag)
                      : issue_tile<4>(t, tmem, ring0, x0, sf0, a.stage_bytes, S, kn, last, ring, full, empty, &acc_full,
                                      abort_flag);
        }
        if (!ok && elect_one()) {
            *abort_flag = 1u;
            atomicOr(a.p.err, ERR_TIMEOUT);
            // no product may be in flight when the CTA ends
            mma_commit(&acc_full);
            mbar_wait_any(&acc_full, (uint32_t)n & 1u);
        }
    } else {
        pdl_wait();  // y may have readers before the kernel this one follows
        if (a.xres) {
            if (a.p.rtype == MX_F16) quantize_x<MX_F16>(a.p, base + a.xres, k0, kn, warp - 2, lane);
            else if (a.p.rtype == MX_BF16) quantize_x<MX_BF16>(a.p, base + a.xres, k0, kn, warp - 2, lane);
            else quantize_x<MX_F32>(a.p, base + a.xres, k0, kn, warp - 2, lane);
            fence_proxy_async();  // the tensor cores read it through the other proxy
            __syncwarp();
            if (lane == 0) mbar_arrive(&x_ready);
        }
        const int qd = warp & 3, grp = (warp - 2) >> 2, row = qd * 32 + lane;
        float *part = (float *)base;  // split: [npad][128] partial sums, over the ring once it is done with
        int n = 0;
        for (int i = first; i < a.tiles; i += step, ++n) {
            const MxTile t(a, i);
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full, (uint32_t)n & 1u, abort_flag))) {
                if (lane == 0) {
                    *abort_flag = 1u;
                    atomicOr(a.p.err, ERR_TIMEOUT);
                }
                break;
            }
            tc_fence_after();
            // All of the accumulator is asked for before any of it is waited for: until the
            // registers have it the next tile's products wait.
            const uint32_t acc = tmem + ((uint32_t)(qd * 32) << 16) + (uint32_t)(grp * 16);
            float v[MXL_CHUNKS][16] = {};
#pragma unroll
            for (int h = 0; h < MXL_CHUNKS; ++h)
                if ((h * (MXL_EPI_WARPS / 4) + grp) * 16 < t.npad)
                    tmem_ask16(acc + (uint32_t)(h * (MXL_EPI_WARPS / 4) * 16), v[h]);
            tmem_wait(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty);
            O *y = (O *)a.p.y + (int64_t)t.b0 * a.p.ldy;
#pragma unroll
            for (int h = 0; h < MXL_CHUNKS; ++h) {
                const int c = (h * (MXL_EPI_WARPS / 4) + grp) * 16;
                if (c >= t.npad) break;
                if (split > 1) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c + j) * MX_TILE_M + row] = v[h][j];
                } else {
                    store16<O>(y, a.p.ldy, c, t.rows, t.rt * MX_TILE_M + row, a.p.N, a.pack, a.p.act, v[h]);
                }
            }
        }
    }
    __syncwarp();
    if (split > 1) {
        // one tile a cluster: every CTA adds its share of the tokens, four outputs a thread
        const MxTile t(a, first);
        cluster_sync();
        if (warp >= 2) {
            const int n = t.rt * MX_TILE_M + lane * 4, c1 = (rank + 1) * t.rows / split;
            O *y = (O *)a.p.y + (int64_t)t.b0 * a.p.ldy;
            for (int c = rank * t.rows / split + warp - 2; c < c1; c += 2 * MXL_EPI_WARPS) {
                const int d = c + MXL_EPI_WARPS;  // a second token, its loads beside the first's
                const uint32_t at = smem_u32(base) + (uint32_t)(c * MX_TILE_M + lane * 4) * 4u;
                float4 v[2][MXL_MAX_SPLIT];
#pragma unroll
                for (int s = 0; s < MXL_MAX_SPLIT; ++s)
                    if (s < split) {
                        v[0][s] = ld_cluster(at, (uint32_t)s);
                        if (d < c1) v[1][s] = ld_cluster(at + MXL_EPI_WARPS * MX_TILE_M * 4u, (uint32_t)s);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 sum = v[h][0];
#pragma unroll
                    for (int s = 1; s < MXL_MAX_SPLIT; ++s)
                        if (s < split) sum.x += v[h][s].x, sum.y += v[h][s].y, sum.z += v[h][s].z, sum.w += v[h][s].w;
                    if (h == 0 || d < c1) store4<O>(y + (int64_t)(h ? d : c) * a.p.ldy, n, a.p.N, a.pack, a.p.act, sum);
                }
            }
        }
        cluster_sync();  // no CTA leaves while its partial sums are read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, a.ncols);
    }
}

namespace {

// How many clusters of 1 .. 8 CTAs, one CTA a SM, the current device runs at once.
struct MxClusters {
    int n[MXL_MAX_SPLIT + 1];
};
const MxClusters *max_clusters(const void *fn, cudaError_t *e) {
    static MxClusters known[64];
    static std::atomic<bool> done[64];
    static std::mutex mu;
    int dev = 0;
    *e = cudaGetDevice(&dev);
    if (*e != cudaSuccess) return nullptr;
    if (dev >= 64) {
        *e = cudaErrorInvalidDevice;
        return nullptr;
    }
    if (done[dev].load(std::memory_order_acquire)) return &known[dev];
    std::lock_guard<std::mutex> lk(mu);
    if (done[dev].load(std::memory_order_acquire)) return &known[dev];
    *e = ensure_smem_attr(fn, (int)MXL_SMEM_MAX);
    for (int s = 1; s <= MXL_MAX_SPLIT && *e == cudaSuccess; ++s) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)s * 256);
        cfg.blockDim = dim3(MXL_THREADS);
        cfg.dynamicSmemBytes = MXL_SMEM_MAX;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)s;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        *e = cudaOccupancyMaxActiveClusters(&known[dev].n[s], fn, &cfg);
    }
    if (*e != cudaSuccess) return nullptr;
    if (known[dev].n[1] < 1) {
        *e = cudaErrorInvalidConfiguration;
        return nullptr;
    }
    done[dev].store(true, std::memory_order_release);
    return &known[dev];
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Column tiles of x that a CTA keeps quantised: 16 leave the ring ten stages.  Quantising
// in the product takes one launch instead of two.
constexpr int MXL_XRES = 16;

// Tokens of a tile and CTAs of a cluster: the pair with the least estimate of a CTA's
// time from its first stage on, in ns.  A stage takes 250 + 0.6 nt (copies, powers and
// products; measured 290 at 16 tokens, 272 at 64, 310 at 128, 368 at 256), a tile's end
// 5 nt alone and 1000 + 17 nt in a cluster (partial sums through shared memory).
// Measured, chosen / next best, us: 256 x 4096 (K 4096) 64 tokens alone 9.2 / 256 tokens
// over 4 CTAs 11.1; 256 x 1024 (K 4096) 64 over 4 7.4 / 128 over 4 8.7; 512 x 4096 128
// alone 10.3 / 256 over 2 11.2; 1024 x 2560 256 10.3 / 128 12.0; 37 x 1337 (K 1000) alone
// 5.0 / over 2 5.8; 1 x 2560 (K 2560) over 5 5.5 / alone 7.2.
void choose(MxLinearArgs &a, const MxClusters &most) {
    const int whole = std::min(MXL_TOKENS, (a.p.B + 15) & ~15);
    double best = 1e30;
    for (int nt : {64, 128, whole}) {
        if (nt > whole) continue;
        const int tiles = a.rtiles * ceil_div(a.p.B, nt), rounds = ceil_div(tiles, most.n[1]);
        for (int s = 1; s <= MXL_MAX_SPLIT && 2 * s <= std::max(2, a.kt); ++s) {
            if (s > 1 && tiles > most.n[s]) continue;
            const double t = s > 1 ? ceil_div(a.kt, s) * (250 + 0.6 * nt) + 1000 + 17.0 * nt
                                   : rounds * (a.kt * (250 + 0.6 * nt) + 5.0 * nt);
            if (t < best) best = t, a.nt = nt, a.split = s;
        }
    }
}

}  // namespace

void launch_mx_linear(const MxLinearParams &p, int type, cudaStream_t stream, cudaError_t (*quantize)(void *),
                      void *ctx, cudaError_t *e) {
    const void *fn = type == MX_F32   ? (const void *)mx_linear_kernel<float>
                     : type == MX_F16 ? (const void *)mx_linear_kernel<__half>
                                      : (const void *)mx_linear_kernel<__nv_bfloat16>;
    MxLinearArgs a;
    a.p = p;
    a.kt = ceil_div(p.K, MX_TILE_K);
    a.rtiles = ceil_div(p.N, MX_TILE_M);
    const MxClusters *most = max_clusters(fn, e);
    if (!most) return;
    choose(a, *most);
    a.tiles = a.rtiles * ceil_div(p.B, a.nt);
    // Every CTA as many tiles as the one with most.
    const int clusters = a.split > 1 ? a.tiles : ceil_div(a.tiles, ceil_div(a.tiles, most->n[1]));
    a.stage_bytes = MX_TILE_BYTES + 2 * MX_SCALE_BYTES + (uint32_t)a.nt * 128u;
    uint32_t smem = MXL_SMEM_MAX - 1024;
    a.xres = 0;
    const int kn = ceil_div(a.kt, a.split);
    if (p.rows && !p.over && p.B <= 16 && p.B * kn <= MXL_XLINES * MXL_EPI_WARPS && kn <= MXL_XRES) {
        a.stage_bytes = MX_TILE_BYTES;
        smem -= (uint32_t)kn * MXL_XREC;
        a.xres = smem & ~1023u;
    } else if (p.rows) {
        *e = quantize(ctx);
        if (*e != cudaSuccess) return;
    }
    a.stages = std::min({MXL_MAX_STAGES, (int)(smem / a.stage_bytes), (512 - a.nt) / (int)MXL_SF});
    a.ncols = 512;
    const int size = type == MX_F32 ? 4 : 2;
    const int neigh = a.split > 1 ? 4 * size : 4;
    a.pack = (uintptr_t)p.y % neigh == 0 && p.ldy * size % neigh == 0;
    cudaError_t r = ensure_smem_attr(fn, (int)MXL_SMEM_MAX);
    if (r == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(clusters * a.split));
        cfg.blockDim = dim3(MXL_THREADS);
        cfg.dynamicSmemBytes = MXL_SMEM_MAX;
        cfg.stream = stream;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)a.split;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = p.rows && !a.xres ? 2 : 1;  // beside the kernel that quantises x
        void *args[] = {&a};
        r = cudaLaunchKernelExC(&cfg, fn, args);
    }
    if (r != cudaSuccess) *e = r;
}

}  // namespace rk
