// q4_tc.cu -- y[b][n] = act(sum over groups of scale * sum_k (q - zero) x[b][k]) on the 5th
// generation tensor cores, for more rows of x than q4.cu's product takes (layout: q4.cuh).
//
// 128 weight rows are the M side, the rows of x the N side (padded to 16, at most 128), so a
// weight is widened once for all of them.  The tensor cores add 16-bit products in fp32, but
// know no scales: a group's sum is made on its own in tensor memory, and eight warps for 64 rows of x
// take it out, multiply it by its row's scale and add it to sums they hold in registers, while
// others widen the next codes into tensor memory, from where the tensor cores read them.
//   warp 0      x: boxes of 64 columns by TMA into the ring's stages
//   warps 1-2   issue the products of every second group each, into accumulators in turn: one
//               issuer takes 46 ns an instruction for up to 128 rows of x, whatever their
//               number, and waits besides
//   warps 4-11  codes to whole numbers in the operand's layout: four warps the even stages of 128
//               columns, four the odd ones, each warp with a ring of its own for the records, copied
//               four stages ahead without a barrier
//   warps 12-19 accumulators to registers, scaled, and at a tile's end y: 32 weight rows, one a
//               lane, and 32 rows of x a warp, or 64 where there are more than 64
// Tensor memory: four stages of widened codes, 64 columns each, and four accumulators of up to 64
// rows of x or two of up to 128.
// One CTA a SM walks its share of the tiles, the rings running on across them; where there are
// few tiles the CTAs of a cluster share one tile's columns and add their sums through
// each other's shared memory, in rank order.
//
// A stage of 64 rows takes 470 ns with one group, 570 with two; of 128 rows 530 and 790.  The products
// alone would take 190 and 260, x's copies about as long, the hand-overs with nothing between them 220
// and 230: what bounds it is the hand-overs, each 100 to 200 cycles late, and the issue slots between them
// (47 % are taken at 128 rows).
// 64 x 10240 x 2560 in groups of 64: 13.0 us; 256 x 4096 x 16384 in groups of 128: 36.1 (17.6 by flops).
// On the way, the same two cases: one set of warps that widened a stage and then took out the one
// before 24 and 119 (the latencies of both in sequence); widened codes in shared memory, codes by loads
// to registers, a tile's end written with branches for each output 14.6 and 44.5; records copied for all
// warps by bulk copies of 1 KB 15.6 and 44.9 (50 ns a copy); for 128 rows sums of 32 rows a warp 39.6
// (16 such warps take issue slots, and left registers for the issuers short: they spilled), for 64 rows
// sums of 64 a warp 14.4; four sets of warps that widen 15.7 and 37.9 (registers); an early
// look at the next accumulator by an instruction that may rest 18.2 and 48.5 (it wakes late).
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>

#include "../../include/rwkv7.h"
#include "q4.cuh"

namespace rk {

constexpr int QT_WIDEN = 4, QT_WIDEN0 = 4;  // warps that widen a stage (two such sets), the first of them
constexpr int QT_SUMS0 = QT_WIDEN0 + 2 * QT_WIDEN;  // the first of the eight that hold the sums
constexpr int QT_THREADS = 32 * (QT_SUMS0 + 8);
// Registers a thread of the launch.  For up to 64 rows of x they are enough for everybody; for more the
// four warps that copy and issue and those that widen hand some to those that hold the sums.
constexpr int QT_REGS = 96;
constexpr int QT_AUX_REGS = 64, QT_WIDEN_REGS = 72, QT_SUMS_REGS = 136;
static_assert(128 * QT_AUX_REGS + 64 * QT_WIDEN * QT_WIDEN_REGS + 256 * QT_SUMS_REGS <= QT_THREADS * QT_REGS, "");
constexpr int QT_M = 128;
constexpr int QT_STAGES = 4;  // of the rings of widened codes and of x; even, as warps take every second one
constexpr int QT_AHEAD = 4;   // a warp's own stages of codes in flight
constexpr int QT_MAX_SPLIT = 8;
constexpr int QT_TOKENS = 128;
constexpr uint32_t QT_A = Q4_COLS / 2;  // columns of tensor memory of a stage's widened codes
constexpr uint32_t QT_A0 = 512 - QT_STAGES * QT_A;  // the first of them, after the accumulators
constexpr uint32_t QT_SMEM = 226 * 1024;
static_assert(1024 + QT_STAGES * 256 * QT_TOKENS + QT_AHEAD * 16 * q4_record(32, true) <= QT_SMEM, "");

struct Q4TcArgs {
    CUtensorMap x;
    Q4LinearParams p;
    int nt, rtiles, tiles, split;
};

struct QtRing {
    int st = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++st == QT_STAGES) st = 0, parity ^= 1u;
    }
};

__device__ __forceinline__ bool qt_elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
template <int N>
__device__ __forceinline__ void qt_fewer_regs() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void qt_more_regs() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
// Whether the phase is over; does not wait, as mbar_try_wait may for a while.
__device__ __forceinline__ bool qt_test_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// mbar_wait that asks for the time only once it has waited long.
__device__ __forceinline__ bool qt_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort) return false;
            const uint64_t t = gtimer();
            if (!t0) t0 = t;
            else if (t - t0 > WAIT_LIMIT_NS) return false;
        }
    }
}
__device__ __forceinline__ void qt_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 qt_ld_cluster(uint32_t at, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 t;\n\tmapa.shared::cluster.u32 t, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [t];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(at), "r"(rank)
        : "memory");
    return v;
}
__device__ __forceinline__ void qt_cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t qt_lds4(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t qt_lds2(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}
// Pairs of fp32 values in one 64-bit register.
using qt_f2 = unsigned long long;
__device__ __forceinline__ qt_f2 qt_pack(float a, float b) {
    qt_f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void qt_unpack(qt_f2 v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ qt_f2 qt_fma(qt_f2 a, qt_f2 b, qt_f2 c) {
    qt_f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// 32 lanes x 16 columns on their way to v, which holds them after qt_tmem_wait.
__device__ __forceinline__ void qt_tmem_ask(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
#define QT_16(v) "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), \
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
__device__ __forceinline__ void qt_tmem_wait(float (&v)[16], float (&w)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : QT_16(v), "+f"(w[0]), "+f"(w[1]), "+f"(w[2]), "+f"(w[3])::"memory");
    asm volatile("" : QT_16(w)::"memory");
}
#undef QT_16
__device__ __forceinline__ void qt_add(qt_f2 (&tot)[8], qt_f2 scale, const float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) tot[j] = qt_fma(scale, qt_pack(v[2 * j], v[2 * j + 1]), tot[j]);
}
// 16 rows x 64 16-bit values into tensor memory: four times 16 columns, of which lane 4 g + t holds pairs
// 2t and 2t + 1 of row g, then of row g + 8.
__device__ __forceinline__ void qt_tmem_put(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// CH: up to 64 CH rows of x (1 or 2).  G: groups of a stage.
template <bool BF, int CH, int G>
__global__ void __launch_bounds__(QT_THREADS, 1) q4_tc_kernel(const __grid_constant__ Q4TcArgs a) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int ACCS = 4 / CH, ACC = QT_A0 / ACCS;  // accumulators, and tensor memory columns of each
    __shared__ uint64_t full_a[QT_STAGES], full_x[QT_STAGES], empty[QT_STAGES], acc_full[4], acc_free[4];
    __shared__ uint32_t tmem_slot, s_abort;
    uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const Q4LinearParams &p = a.p;
    const Q4Matrix &m = p.w;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = a.split;
    const int first = blockIdx.x / split, rank = blockIdx.x - first * split, step = gridDim.x / split;
    const int k0 = (int)((int64_t)m.kt * rank / split), kn = (int)((int64_t)m.kt * (rank + 1) / split) - k0;
    volatile uint32_t *abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        for (int i = 0; i < QT_STAGES; ++i) {
            mbar_init(&full_a[i], QT_WIDEN);
            mbar_init(&full_x[i], 1);
            mbar_init(&empty[i], G > 1 ? 2 : 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 8);
        }
        s_abort = 0u;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    // The barriers and the tensor memory are there.  (Waited for by each role in its place: the first codes
    // are on their way by then, 0.5 us earlier; x's first stages before it made no call faster.)
    auto begin = [&]() {
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        return __shfl_sync(0xffffffffu, tmem_slot, 0);
    };
    const uint32_t half_x = (uint32_t)a.nt * 128u;  // a box of 64 columns
    const uint32_t record = q4_record(Q4_COLS / G, m.zeros);
    uint8_t *const codes = base + QT_STAGES * 2 * half_x;
    const int stages = first < a.tiles ? ((a.tiles - 1 - first) / step + 1) * kn : 0;

    if (CH == 2 && warp < QT_WIDEN0) qt_fewer_regs<QT_AUX_REGS>();
    if (warp == 0) {
        begin();
        if (lane == 0) {
            prefetch_tmap(&a.x);
            const uint64_t pol = policy_evict_last();
            QtRing ring;
            int q = 0;
            bool ok = true;
            for (int i = first; i < a.tiles && ok; i += step) {
                const int b0 = i / a.rtiles * a.nt;
                for (int k = 0; k < kn; ++k, ++q, ring.next()) {
                    if (q >= QT_STAGES && !qt_wait(&empty[ring.st], ring.parity ^ 1u, abort_flag)) {
                        *abort_flag = 1u;
                        atomicOr(p.err, ERR_TIMEOUT);
                        ok = false;
                        break;
                    }
                    uint8_t *to = base + ring.st * (2 * half_x);
                    mbar_expect_tx(&full_x[ring.st], 2 * half_x);
                    tma_load_2d(to, &a.x, &full_x[ring.st], (k0 + k) * Q4_COLS, b0, pol);
                    tma_load_2d(to + half_x, &a.x, &full_x[ring.st], (k0 + k) * Q4_COLS + 64, b0, pol);
                }
            }
            // no copy may be in flight when the CTA ends
            for (int j = max(0, q - QT_STAGES); j < q; ++j)
                if (!mbar_wait_any(&full_x[j % QT_STAGES], (uint32_t)(j / QT_STAGES) & 1u)) break;
        }
    } else if (warp <= 2) {
        const uint32_t idesc = idesc_f16(QT_M, a.nt) | (BF ? 1u << 7 | 1u << 10 : 0u);
        const uint32_t tmem = begin();
        const bool leader = qt_elect();
        const int mine = warp - 1;  // the groups whose number is so modulo 2
        QtRing ring;
        if (G == 1 && mine) ring.next();
        int acc = mine;
        uint32_t uses = 0;  // of all accumulators before this one's turn
        bool ok = true;
        for (int s = G == 1 ? mine : 0; s < stages && ok; s += G == 1 ? 2 : 1) {
            // All that a stage waits for is asked for at once: one answer takes 150 cycles.
            const bool x_in = mbar_try_wait(&full_x[ring.st], ring.parity), a_in = mbar_try_wait(&full_a[ring.st], ring.parity);
            const bool room = !uses || mbar_try_wait(&acc_free[acc], (uses - 1) & 1u);
            if (!(x_in && a_in && room))
                ok = qt_wait(&full_x[ring.st], ring.parity, abort_flag) && qt_wait(&full_a[ring.st], ring.parity, abort_flag) &&
                     (!uses || qt_wait(&acc_free[acc], (uses - 1) & 1u, abort_flag));
            const uint32_t ta = tmem + QT_A0 + (uint32_t)ring.st * QT_A;
            const uint64_t dx = sdesc_k128(smem_u32(base) + (uint32_t)ring.st * (2 * half_x));
#pragma unroll
            for (int v = 0; v < G; v += 2) {
                if (v > 0 && ok && uses) ok = qt_wait(&acc_free[acc], (uses - 1) & 1u, abort_flag);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t d = tmem + (uint32_t)(acc * ACC);
                    const int u = G == 1 ? 0 : v + mine;
#pragma unroll
                    for (int j = 0; j < 8 / G; ++j) {  // 16 columns each
                        const int c = u * (8 / G) + j;
                        mma_f16_ts(d, ta + 8 * c, dx + (uint64_t)((uint32_t)(c >> 2) * (half_x >> 4) + 2 * (c & 3)), idesc,
                                   j > 0);
                    }
                    mma_commit(&acc_full[acc]);
                    if (v + 2 >= G) mma_commit(&empty[ring.st]);
                }
                __syncwarp();
                acc += 2;
                if (acc >= ACCS) acc -= ACCS, ++uses;
            }
            ring.next();
            if (G == 1) ring.next();
        }
        if (!ok && qt_elect()) {
            *abort_flag = 1u;
            atomicOr(p.err, ERR_TIMEOUT);
            // no product may be in flight when the CTA ends
            mma_commit(&acc_full[acc]);
            mbar_wait_any(&acc_full[acc], uses & 1u);
        }
    } else if (warp >= QT_WIDEN0 && warp < QT_SUMS0) {
        // A warp takes two row tiles of a stage, one after the other; a set every second stage.
        const int w = (warp - QT_WIDEN0) % QT_WIDEN, set = (warp - QT_WIDEN0) / QT_WIDEN, g = lane >> 2, t = lane & 3;
        if (CH == 2) qt_fewer_regs<QT_WIDEN_REGS>();
        // The warp's own ring of pairs of records, with no barrier but for itself.
        const uint32_t pair = 2 * record, more = (record - Q4_CODES) / 16;  // lanes that fetch scales and zeros
        const uint32_t ring0 = smem_u32(codes) + (uint32_t)(warp - QT_WIDEN0) * QT_AHEAD * pair;
        const uint32_t mine = ring0 + (uint32_t)(4 * g + (t >> 1)) * 16 + (t & 1) * 4, zeros = ring0 + Q4_CODES + 32 * G + 2 * g;
        const uint8_t *src[2] = {};
        int ft = first - step, fk = kn, left = stages > set ? (stages - set + 1) / 2 : 0;  // to fetch
        uint32_t fat = ring0 + lane * 16;
        auto fetch = [&](int onward) {  // of the stage that many on
            if (left > 0) {
                --left, fk += onward;
                if (fk < kn) {
                    src[0] += (uint32_t)onward * record, src[1] += (uint32_t)onward * record;
                } else {
                    while (fk >= kn) fk -= kn, ft += step;
                    // Past the last row tile: the last one, whose sums are not stored.
                    const int rt = ft % a.rtiles * 8 + 2 * w;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        src[i] = m.data + ((int64_t)min(rt + i, m.rt - 1) * m.kt + k0 + fk) * record + lane * 16;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    qt_cp16(fat + i * record, src[i]);
                    qt_cp16(fat + i * record + 512, src[i] + 512);
                    if (lane < more) qt_cp16(fat + i * record + Q4_CODES, src[i] + Q4_CODES);
                }
                fat += pair;
                if (fat >= ring0 + QT_AHEAD * pair) fat -= QT_AHEAD * pair;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        fetch(set);
        for (int i = 1; i < QT_AHEAD - 1; ++i) fetch(2);
        const uint32_t tmem = begin();
        uint32_t at = 0;
        QtRing ring;
        if (set) ring.next();
        for (int n = set; n < stages; n += 2) {
            fetch(2);
            asm volatile("cp.async.wait_group %0;" ::"n"(QT_AHEAD - 1) : "memory");
            __syncwarp();
            uint32_t code[2][8];  // row tile, 16 columns: of rows g and g + 8 columns 4t .. 4t + 3
            uint32_t zero[2][G];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    code[i][c] = qt_lds4(mine + at + i * record + (c >> 2) * 512 + (c & 1) * 32 + (c >> 1 & 1) * 8);
#pragma unroll
                for (int u = 0; u < G; ++u) zero[i][u] = m.zeros ? qt_lds2(zeros + at + i * record + 16 * u) : 0x0808u;
            }
            __syncwarp();  // read before its place is fetched into again, by the next turn
            at = at + pair == QT_AHEAD * pair ? 0 : at + pair;
            if (n >= QT_STAGES && !__all_sync(0xffffffffu, qt_wait(&empty[ring.st], ring.parity ^ 1u, abort_flag))) {
                if (lane == 0) {
                    *abort_flag = 1u;
                    atomicOr(p.err, ERR_TIMEOUT);
                }
                break;
            }
            tc_fence_after();
            const uint32_t to = tmem + ((uint32_t)(32 * w) << 16) + QT_A0 + (uint32_t)ring.st * QT_A;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                Q4Zero z[G];
#pragma unroll
                for (int u = 0; u < G; ++u) z[u] = q4_zero<BF>(zero[i][u] & 0xFFu, zero[i][u] >> 8);
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // 64 columns
                    uint32_t v[16];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        uint32_t q[4];
                        q4_widen<BF>(code[i][4 * c + b], z[(4 * c + b) * G / 8], q);
                        v[4 * b] = q[0], v[4 * b + 1] = q[2], v[4 * b + 2] = q[1], v[4 * b + 3] = q[3];
                    }
                    qt_tmem_put(to + ((uint32_t)(16 * i) << 16) + 32 * c, v);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full_a[ring.st]);
            ring.next(), ring.next();
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp >= QT_SUMS0) {
        if (CH == 2) qt_more_regs<QT_SUMS_REGS>();
        const uint32_t tmem = begin();
        // A warp holds the sums of 32 weight rows, one a lane, and 32 CH rows of x.
        const int qd = warp & 3, grp = (warp - QT_SUMS0) >> 2, row = qd * 32 + lane;
        const int chunks = (a.nt - grp * 32 * CH) / 16;  // sixteens of those rows that there are, 2 or more: all
        qt_f2 tot[2 * CH][8];                            // pairs
#pragma unroll
        for (int h = 0; h < 2 * CH; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j) tot[h][j] = 0;
        int acc = 0;  // the accumulator whose turn it is, and the parity of its use
        uint32_t parity = 0;
        bool ready = false, ok = true;
        const uint32_t acc0 = tmem + ((uint32_t)(qd * 32) << 16) + (uint32_t)(grp * 32 * CH);
        float *part = (float *)base;  // split: [nt][128] sums, over the ring once it is done with
        // The next group's sums times scale, a half's bits.  Columns past the tile's rows of x are not stored.
        auto take = [&](uint32_t scale) {
            if (!__all_sync(0xffffffffu, ready) && !__all_sync(0xffffffffu, qt_wait(&acc_full[acc], parity, abort_flag)))
                return false;
            tc_fence_after();
            const uint32_t at = acc0 + (uint32_t)(acc * ACC);
            const float s = __half2float(__ushort_as_half((unsigned short)scale));
            const qt_f2 two = qt_pack(s, s);
#pragma unroll
            for (int b = 0; b < CH; ++b) {
                float v[2][16];
                qt_tmem_ask(at + 32 * b, v[0]);
                qt_tmem_ask(at + 32 * b + 16, v[1]);
                qt_tmem_wait(v[0], v[1]);
                if (b == CH - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_free[acc]);
                    if (++acc == ACCS) acc = 0, parity ^= 1u;
                    ready = qt_test_wait(&acc_full[acc], parity);  // the next one's answer takes a while
                }
                qt_add(tot[2 * b], two, v[0]), qt_add(tot[2 * b + 1], two, v[1]);
            }
            return true;
        };
        for (int i = first; i < a.tiles; i += step) {
            const int bt = i / a.rtiles, rt = (i - bt * a.rtiles) * 8 + (row >> 4);
            // scales, by fours and four groups ahead; past the last row tile the last one's
            const uint8_t *src = m.data + ((int64_t)min(rt, m.rt - 1) * m.kt + k0) * record + Q4_CODES + ((row & 7) * 2 + (row >> 3 & 1)) * 2;
            const int groups = kn * G;
            auto ahead = [&](int j) { return (uint32_t)*(const uint16_t *)(src + j / G * record + j % G * 32); };
            uint32_t scale[4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < groups) scale[j] = ahead(j);
            int q = 0;
            for (; q + 4 <= groups && ok; q += 4) {
                src += 4 / G * record;
                uint32_t next[4] = {};
                if (q + 8 <= groups) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) next[j] = ahead(j);
                } else {
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (q + 4 + j < groups) next[j] = ahead(j);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (ok) ok = take(scale[j]);
                    scale[j] = next[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (ok && q + j < groups) ok = take(scale[j]);
            if (!ok) {
                if (lane == 0) {
                    *abort_flag = 1u;
                    atomicOr(p.err, ERR_TIMEOUT);
                }
                break;
            }
            const int n = rt / 8 * QT_M + row;
#pragma unroll
            for (int b = 0; b < CH; ++b) {
                const int c0 = grp * 32 * CH + 32 * b, rows = min(a.nt, p.B - bt * a.nt) - c0;
                float o[32];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    qt_unpack(tot[2 * b + j / 16][j % 16 / 2], o[j], o[j + 1]);
                    tot[2 * b + j / 16][j % 16 / 2] = 0;
                }
                if (split > 1) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (32 * b + j < 16 * chunks) part[(c0 + j) * QT_M + row] = o[j];
                } else if (n < m.N) {
                    q4_store_rows(p, bt * a.nt + c0, n, rows, o);
                }
            }
        }
    } else {
        begin();
    }
    __syncwarp();
    if (split > 1) {
        // one tile a cluster: every CTA adds its share of the rows of x, four outputs a thread
        qt_cluster_sync();
        const int bt = first / a.rtiles, n = (first - bt * a.rtiles) * QT_M + lane * 4, b0 = bt * a.nt;
        const int rows = min(a.nt, p.B - b0), c1 = (rank + 1) * rows / split;
        for (int c = rank * rows / split + warp; c < c1; c += QT_THREADS / 32) {
            const uint32_t at = smem_u32(base) + (uint32_t)(c * QT_M + lane * 4) * 4u;
            float4 v[QT_MAX_SPLIT], sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int s = 0; s < QT_MAX_SPLIT; ++s)
                if (s < split) v[s] = qt_ld_cluster(at, (uint32_t)s);
#pragma unroll
            for (int s = 0; s < QT_MAX_SPLIT; ++s)
                if (s < split) sum.x += v[s].x, sum.y += v[s].y, sum.z += v[s].z, sum.w += v[s].w;
            const float o[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < m.N) q4_store(p, b0 + c, n + j, o[j]);
        }
        qt_cluster_sync();  // no CTA leaves while its sums are read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_slot, 512);
    }
}

// x with rows off the 16-byte grid, copied to rows on it.
__global__ void __launch_bounds__(256) q4_realign_kernel(const uint16_t *x, int64_t ldx, int B, int K, uint16_t *to, int ldt) {
    const int64_t all = (int64_t)B * (ldt / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t b = i / (ldt / 8);
        *(uint4 *)(to + i * 8) = q4_x8(x + b * ldx, (int)(i - b * (ldt / 8)) * 8, K);
    }
}

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_acquire);
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (PFN_cuTensorMapEncodeTiled_v12000)p;
        known.store(fn, std::memory_order_release);
    }
    return fn;
}

// How many clusters of 1 .. 8 CTAs, one CTA a SM, the current device runs at once.
struct Clusters {
    int n[QT_MAX_SPLIT + 1];
};
const Clusters *max_clusters(const void *fn, cudaError_t *e) {
    static Clusters known[64];
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
    *e = ensure_smem_attr(fn, (int)QT_SMEM);
    for (int s = 1; s <= QT_MAX_SPLIT && *e == cudaSuccess; ++s) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)s * 256);
        cfg.blockDim = dim3(QT_THREADS);
        cfg.dynamicSmemBytes = QT_SMEM;
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

// The warps' shares of the registers have to be there, or they would wait for them.  Asked once for
// each kernel.
cudaError_t has_registers(const void *fn, int ch) {
    static std::atomic<const void *> known[16];
    for (auto &k : known) {
        const void *f = k.load(std::memory_order_acquire);
        if (f == fn) return cudaSuccess;
        if (f) continue;
        cudaFuncAttributes at;
        const cudaError_t r = cudaFuncGetAttributes(&at, fn);
        if (r != cudaSuccess) return r;
        if (ch == 2 && at.numRegs != QT_REGS) return cudaErrorInvalidConfiguration;
        k.compare_exchange_strong(f, fn);
        return cudaSuccess;
    }
    return cudaErrorInvalidConfiguration;  // (12 kernels)
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Rows of x of a tile and CTAs of a cluster: the pair with the least estimate of a CTA's time in
// ns.  A stage takes 310 + 155 for each of its groups (measured 470 with one, 570 with two, 930 with
// four), with more than 64 rows 265 + 262 (530, 790, 1300); a tile's end 5 nt alone and 1000 + 17 nt in
// a cluster.
void choose(Q4TcArgs &a, const Clusters &most) {
    const Q4LinearParams &p = a.p;
    const int blocks = ceil_div(p.B, QT_TOKENS), whole = (ceil_div(p.B, blocks) + 15) & ~15;
    double best = 1e30;
    for (int nt : {64, whole}) {
        if (nt > whole) continue;
        const int tiles = a.rtiles * ceil_div(p.B, nt), rounds = ceil_div(tiles, most.n[1]);
        const double groups = Q4_COLS / p.w.group, stage = nt > 64 ? 265 + 262 * groups : 310 + 155 * groups;
        for (int s = 1; s <= QT_MAX_SPLIT && 2 * s <= std::max(2, p.w.kt); ++s) {
            if (s > 1 && tiles > most.n[s]) continue;
            const double t = s > 1 ? ceil_div(p.w.kt, s) * stage + 1000 + 17.0 * nt : rounds * (p.w.kt * stage + 5.0 * nt);
            if (t < best) best = t, a.nt = nt, a.split = s;
        }
    }
}

template <bool BF, int CH>
const void *tc_fn(int group) {
    return group == 32   ? (const void *)q4_tc_kernel<BF, CH, 4>
           : group == 64 ? (const void *)q4_tc_kernel<BF, CH, 2>
                         : (const void *)q4_tc_kernel<BF, CH, 1>;
}
template <bool BF>
const void *tc_fn(int ch, int group) {
    return ch == 1 ? tc_fn<BF, 1>(group) : tc_fn<BF, 2>(group);
}

}  // namespace

void launch_q4_tc(const Q4LinearParams &p, int xtype, cudaStream_t stream, cudaError_t *e) {
    Q4TcArgs a;
    memset(&a, 0, sizeof a);
    a.p = p;
    a.rtiles = ceil_div(p.w.N, QT_M);
    const bool bf = xtype == MX_BF16;
    const Clusters *most = max_clusters((const void *)q4_tc_kernel<false, 2, 1>, e);
    if (!most) return;
    choose(a, *most);
    a.tiles = a.rtiles * ceil_div(p.B, a.nt);
    if (!p.xvec) {
        const int ldt = (p.w.K + 7) & ~7;
        const int64_t blocks = ((int64_t)p.B * (ldt / 8) + 255) / 256;
        q4_realign_kernel<<<(unsigned)std::min<int64_t>(blocks, 152 * 64), 256, 0, stream>>>(
            (const uint16_t *)p.x, p.ldx, p.B, p.w.K, (uint16_t *)p.room, ldt);
        *e = cudaGetLastError();
        if (*e != cudaSuccess) return;
        a.p.x = p.room, a.p.ldx = ldt;
    }
    const auto encode = encode_fn();
    // (The stride of a single row stands for nothing, and need not be one that a map takes.)
    const int64_t ldx = p.B == 1 ? (p.w.K + 7) & ~7 : a.p.ldx;
    const cuuint64_t dims[2] = {(cuuint64_t)p.w.K, (cuuint64_t)p.B}, strides[1] = {(cuuint64_t)ldx * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)a.nt}, one[2] = {1, 1};
    if (!encode || encode(&a.x, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                          const_cast<void *>(a.p.x), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
        *e = cudaErrorInvalidValue;
        return;
    }
    const int ch = a.nt <= 64 ? 1 : 2;
    const void *fn = bf ? tc_fn<true>(ch, p.w.group) : tc_fn<false>(ch, p.w.group);
    // Every CTA as many tiles as the one with most.
    const int clusters = a.split > 1 ? a.tiles : ceil_div(a.tiles, ceil_div(a.tiles, most->n[1]));
    cudaError_t r = has_registers(fn, ch);
    if (r == cudaSuccess) r = ensure_smem_attr(fn, (int)QT_SMEM);
    if (r == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(clusters * a.split));
        cfg.blockDim = dim3(QT_THREADS);
        cfg.dynamicSmemBytes = QT_SMEM;
        cfg.stream = stream;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)a.split;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        void *args[] = {&a};
        r = cudaLaunchKernelExC(&cfg, fn, args);
    }
    if (r != cudaSuccess) *e = r;
}

}  // namespace rk
