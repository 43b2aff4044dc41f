// beam.cu -- beam search over state slots (calls: include/rwkv7.h).
//
// Selection.  Beam b of a request stands for the candidates (b, v), v a token, of score
//     s(b, v) = score[b] + x[b][v] - log sum_u exp x[b][u]
// and rank s / len^penalty; wanted are a request's k best, ties to the lowest b, then v.
// Within a beam the rank rises with x, so a beam's k largest logits are all it can send, and
// one pass over a row finds them together with its largest value and its sum.  A CTA takes a chunk
// of a row into registers and leaves its top, the sum of exp(x - top) and its k largest; the last
// CTA of a request to do so joins the request's chunks: norms, scores, ranks, the k best.
//
// k largest of n values without sorting them: the k-th largest of the maxima of M >= k
// groups of values is a value that at least k of them reach, and with M = 2k or more
// few others do.  What reaches it is listed, and each listed value's place is the number of
// those ahead of it.  Where values tie by the hundred the list may run over: then the k are
// taken one by one.
//
// Which of two beams' candidates is ahead depends on the sums' last bits.  Where a warp has a value
// within 1 of the top, exp(x - top) is 2^n times a polynomial of degree 6 (fitted to 2e-9; rounding
// leaves 8e-8, with a mean of 1e-9; 1 exactly for x = top); elsewhere, where no term has more than
// e^-1 of the largest one's weight, the hardware's 2^x does.  A thread adds its terms to a sum that
// starts at 1, no term being larger, so that the part cut off by each addition is known exactly and
// kept; the threads' sums are joined as whole multiples of 2^-40, and so are the chunks'.  Double
// precision is slow here (an operation of a warp takes 16 cycles of the SM; a launch of its own that
// took norms and ranks by it 12 us): the candidates' scores are pairs of fp32, high and low part,
// unless a score or what a length divides it by is out of their range.
//
// Measured (in a graph, with the 1 us that zeroes its tickets; by bytes at the copy rate): 4 rows of 65,536 fp32
// logits 8 us (0.15), 64 rows 12 (2.5), 192 rows 25 (7.4).  What is left is latency: a chunk's loads, its three
// barriers and its ticket follow one another, and the four CTAs that an SM's registers hold do not
// cover them (23 % of issue slots, 2.5 rounds of chunks of 8192 values).  Chunks of 4096: 37 us.
#include <cfloat>
#include <cstdio>
#include <cstring>

#include "../../include/rwkv7.h"
#include "beam.cuh"
#include "mx.cuh"
#include "span.h"

namespace rk {

constexpr int BR_THREADS = 256;
constexpr int BR_LIST = 512;   // values listed by a chunk
constexpr int BP_EACH = 4;     // candidates of a thread at a time
constexpr int BP_LIST = 512;   // listed at a time

// Pairs of fp32 values in one 64-bit register.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) {
    f2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 both(float v) { return pack2(v, v); }

// exp of two values <= 0; below -87 about 1e-38.
__device__ __forceinline__ f2 exp_pair(f2 d) {
    float a, b;
    unpack2(d, a, b);
    d = pack2(fmaxf(a, -87.0f), fmaxf(b, -87.0f));
    const f2 magic = both(12582912.0f);  // 1.5 * 2^23: adding it rounds to whole numbers
    const f2 t = fma2(d, both(1.44269502162933349609f), magic);
    f2 f = fma2(d, both(1.44269502162933349609f), sub2(magic, t));
    f = fma2(d, both(1.92596298909109e-08f), f);
    f2 r = both(0x1.41fbbcp-13f);  // 2^f - 1 = f * polynomial, |f| <= 1/2
    r = fma2(r, f, both(0x1.5f3e52p-10f));
    r = fma2(r, f, both(0x1.3b2d4cp-7f));
    r = fma2(r, f, both(0x1.c6aee8p-5f));
    r = fma2(r, f, both(0x1.ebfbdcp-3f));
    r = fma2(r, f, both(0x1.62e430p-1f));
    r = fma2(r, f, both(1.0f));
    float n0, n1;
    unpack2(t, n0, n1);
    unpack2(r, a, b);
    a = __uint_as_float(__float_as_uint(a) + (__float_as_uint(n0) << 23));
    b = __uint_as_float(__float_as_uint(b) + (__float_as_uint(n1) << 23));
    return pack2(a, b);
}

// The same for terms of little weight: 2^x of the hardware.
__device__ __forceinline__ f2 exp_pair_fast(f2 d) {
    const f2 t = mul2(d, both(1.44269502162933349609f));
    float a, b;
    unpack2(t, a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    return pack2(a, b);
}
constexpr float BR_NEAR = -1.0f;

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A value and its place, larger for larger values and, among equal ones, for earlier places.
__device__ __forceinline__ unsigned long long value_key(float v, uint32_t at) {
    const uint32_t u = __float_as_uint(v + 0.0f);  // -0 is 0
    return (unsigned long long)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (uint32_t)~at;
}
__device__ __forceinline__ float key_value(unsigned long long key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// 16 bytes of a row.
template <int T>
struct BeamVec {
    static constexpr int N = T == MX_F32 ? 4 : 8;
    using type = typename MxElem<T>::type;
    static __device__ __forceinline__ float up(type v) {
        if constexpr (T == MX_F32) return v;
        else if constexpr (T == MX_F16) return __half2float(v);
        else return __bfloat162float(v);
    }
    static constexpr uint32_t NONE = T == MX_F32 ? 0xFF800000u : T == MX_F16 ? 0xFC00FC00u : 0xFF80FF80u;  // -infinity
    // Those from value c of a row of V on, c a multiple of N less what the row starts past a 16-byte boundary.
    static __device__ __forceinline__ uint4 load(const type *x, int c, int V) {
        if (c >= 0 && c + N <= V) return __ldcs((const uint4 *)(x + c));
        uint32_t w[4] = {NONE, NONE, NONE, NONE};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (c + i < 0 || c + i >= V) continue;
            if constexpr (T == MX_F32) w[i] = ((const uint32_t *)x)[c + i];
            else w[i / 2] = __byte_perm(w[i / 2], ((const uint16_t *)x)[c + i], i % 2 ? 0x5410 : 0x3254);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ void up(const uint4 &w, float *v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == MX_F32) {
                v[i] = __uint_as_float(u[i]);
            } else if constexpr (T == MX_F16) {
                const float2 f = __half22float2(*(const __half2 *)&u[i]);
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            } else {
                v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            }
        }
    }
};

// Groups of threads whose maxima give the bound: a power of two of at least 2k, and 32.
__host__ __device__ constexpr int beam_groups(int k, int threads) {
    int m = 32;
    while (m < 2 * k && m < threads) m *= 2;
    return m;
}

struct BeamRows {  // shared memory of a chunk
    unsigned long long list[BR_LIST], wide[BR_THREADS / 32];
    alignas(16) float gmax[BR_THREADS];
    float wmax[BR_THREADS / 32], bound;
    int listed;
};

// A warp's lanes' vectors w, each followed by the next lane's and the last lane's by the first one's next,
// moved on by S words and, of 16-bit values, `bits` bits: vectors from that place on.
template <int S, bool HALF, int n>
__device__ __forceinline__ void beam_move(uint4 (&w)[n + 1], int lane, int bits) {
#pragma unroll
    for (int j = 0; j < n; ++j) {
        const uint32_t a[4] = {w[j].x, w[j].y, w[j].z, w[j].w}, o[4] = {w[j + 1].x, w[j + 1].y, w[j + 1].z, w[j + 1].w};
        uint32_t t[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = a[i];
#pragma unroll
        for (int i = 0; i < S + HALF; ++i) t[4 + i] = __shfl_sync(0xffffffffu, lane ? a[i] : o[i], (lane + 1) & 31);
        if constexpr (HALF) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[S + i] = __funnelshift_r(t[S + i], t[S + i + 1], bits);
        }
        w[j] = make_uint4(t[S], t[S + 1], t[S + 2], t[S + 3]);
    }
}

// Chunk c of row r: values 256 E c .. 256 E (c + 1) - 1 of it, 32 E in a row for a warp.  Memory is
// read by vectors on 16-byte boundaries; where the row starts off them, the values are moved to
// the lanes that have them in every other row, so that rows of the same values have the same
// sums to the last bit, and equal beams the same ranks.
template <int T, int E, bool GRID>
__device__ __forceinline__ void beam_chunk(const BeamSelectParams &p, BeamRows &s, int row, int chunk) {
    using V = BeamVec<T>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const typename V::type *x = (const typename V::type *)p.logits + row * p.ld;
    constexpr int STEP = 32 * V::N, VECS = E / V::N;
    const int begin = chunk * (BR_THREADS * E), first = begin + warp * (32 * E) + lane * V::N;  // of the thread's first vector
    float v[E];
    if constexpr (GRID) {
        if (begin + BR_THREADS * E <= p.V) {  // whole vectors throughout
            uint4 w[VECS];
#pragma unroll
            for (int j = 0; j < VECS; ++j) w[j] = __ldcs((const uint4 *)(x + first + j * STEP));
#pragma unroll
            for (int j = 0; j < VECS; ++j) V::up(w[j], v + j * V::N);
        } else {
#pragma unroll
            for (int j = 0; j < VECS; ++j) {
                const int at = first + j * STEP;
                if (at + V::N <= p.V) {
                    V::up(__ldcs((const uint4 *)(x + at)), v + j * V::N);
                } else {
#pragma unroll
                    for (int i = 0; i < V::N; ++i) v[j * V::N + i] = at + i < p.V ? V::up(x[at + i]) : -INFINITY;
                }
            }
        }
    } else {
        const int shift = (int)(((uintptr_t)x / sizeof(*x)) % V::N);  // values past a boundary
        uint4 w[VECS + 1];
        const int from = begin + warp * (32 * E);
        if (from >= shift && from + 32 * E + V::N - shift <= p.V) {  // whole vectors throughout the warp
#pragma unroll
            for (int j = 0; j < VECS; ++j) w[j] = __ldcs((const uint4 *)(x + first - shift + j * STEP));
            if (lane == 0) w[VECS] = __ldcs((const uint4 *)(x + first - shift + VECS * STEP));
        } else {
#pragma unroll
            for (int j = 0; j < VECS; ++j) w[j] = V::load(x, first - shift + j * STEP, p.V);
            if (lane == 0) w[VECS] = V::load(x, first - shift + VECS * STEP, p.V);
        }
        constexpr bool HALF = T != MX_F32;
        const int bits = HALF ? shift % 2 * 16 : 0;
        switch (shift * (int)sizeof(*x) / 4) {
        case 0:
            if (HALF && bits) beam_move<0, HALF, VECS>(w, lane, bits);
            break;
        case 1: beam_move<1, HALF, VECS>(w, lane, bits); break;
        case 2: beam_move<2, HALF, VECS>(w, lane, bits); break;
        default: beam_move<3, HALF, VECS>(w, lane, bits);
        }
#pragma unroll
        for (int j = 0; j < VECS; ++j) V::up(w[j], v + j * V::N);
    }
    float mine = v[0];
#pragma unroll
    for (int i = 1; i < E; ++i) mine = max_nan(mine, v[i]);
    if (!(mine < INFINITY)) {  // infinity or NaN: no candidates, like -infinity
        mine = -INFINITY;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (!(v[i] < INFINITY)) v[i] = -INFINITY;
            mine = fmaxf(mine, v[i]);
        }
    }
    const int M = beam_groups(p.k, BR_THREADS), per = BR_THREADS / M;
    {
        float w = mine;
        if (per == 1) s.gmax[tid] = w;
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
            w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, off));
            if (2 * off == per && (lane & (per - 1)) == 0) s.gmax[tid / per] = w;
        }
        if (lane == 0) s.wmax[warp] = w;
    }
    if (tid == 0) s.listed = 0, s.bound = -INFINITY;
    __syncthreads();
    float top = s.wmax[0];
#pragma unroll
    for (int i = 1; i < BR_THREADS / 32; ++i) top = fmaxf(top, s.wmax[i]);
    const int64_t out = (int64_t)row * p.chunks + chunk;
    unsigned long long *keys = p.keys + out * p.k;
    if (top == -INFINITY) {
        if (tid < p.k) keys[tid] = 0ull;
        if (tid == 0) p.tops[out] = top, p.sums[out] = 0ull;
        return;
    }
    if (tid < M) {  // the k-th largest of the groups' maxima
        const float m = s.gmax[tid];
        int ahead = 0;
        for (int j = 0; j < M; j += 4) {
            const float4 o = *(const float4 *)(s.gmax + j);
            ahead += (o.x > m || (o.x == m && j < tid)) + (o.y > m || (o.y == m && j + 1 < tid)) +
                     (o.z > m || (o.z == m && j + 2 < tid)) + (o.w > m || (o.w == m && j + 3 < tid));
        }
        if (ahead == p.k - 1) s.bound = m;
    }
    {
        f2 sum = both(1.0f), rest = both(0.0f);
        const f2 t2 = both(top);
        auto add = [&](f2 e) {
            const f2 n = add2(sum, e);
            rest = add2(rest, sub2(e, sub2(n, sum)));  // what the addition cut off, exactly
            sum = n;
        };
        if (__any_sync(0xffffffffu, mine - top > BR_NEAR)) {
#pragma unroll
            for (int i = 0; i < E; i += 2) add(exp_pair(sub2(pack2(v[i], v[i + 1]), t2)));
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 2) add(exp_pair_fast(sub2(pack2(v[i], v[i + 1]), t2)));
        }
        float s0, s1, r0, r1;
        unpack2(sum, s0, s1);
        unpack2(rest, r0, r1);
        // sums are multiples of 2^-23 below 2^5, the rest below 2^-14
        long long q = ((long long)__float2int_rn((s0 - 1.0f) * 0x1p23f) << 17) + __float2int_rn(r0 * 0x1p40f);
        q += ((long long)__float2int_rn((s1 - 1.0f) * 0x1p23f) << 17) + __float2int_rn(r1 * 0x1p40f);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
        if (lane == 0) s.wide[warp] = (unsigned long long)q;
    }
    __syncthreads();
    if (tid == 0) {
        unsigned long long q = 0;
#pragma unroll
        for (int i = 0; i < BR_THREADS / 32; ++i) q += s.wide[i];
        p.tops[out] = top, p.sums[out] = q;
    }
    const float least = fmaxf(s.bound, -FLT_MAX);  // -infinity is no candidate
    if (mine >= least) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (v[i] >= least) {
                const int n = atomicAdd(&s.listed, 1);
                if (n < BR_LIST) s.list[n] = value_key(v[i], (uint32_t)(first + (i / V::N) * STEP + i % V::N));
            }
        }
    }
    __syncthreads();
    const int n = s.listed;
    if (n <= BR_LIST) {
        for (int i = tid; i < n; i += BR_THREADS) {
            const unsigned long long key = s.list[i];
            int ahead = 0;
            for (int j = 0; j < n; ++j) ahead += s.list[j] > key;
            if (ahead < p.k) keys[ahead] = key;
        }
        if (tid >= n && tid < p.k) keys[tid] = 0ull;
        return;
    }
    unsigned long long last = ~0ull;
    for (int r = 0; r < p.k; ++r) {  // one by one
        unsigned long long best = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const unsigned long long key =
                v[i] > -INFINITY ? value_key(v[i], (uint32_t)(first + (i / V::N) * STEP + i % V::N)) : 0ull;
            if (key < last && key > best) best = key;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
        __syncthreads();
        if (lane == 0) s.wide[warp] = best;
        __syncthreads();
        best = s.wide[0];
#pragma unroll
        for (int i = 1; i < BR_THREADS / 32; ++i) best = max(best, s.wide[i]);
        if (tid == 0) keys[r] = best;
        last = best;  // 0: none left, and none below it
    }
}

// Order of 64-bit reals, and of pairs of fp32 whose second is at most half a step of the first, as of
// unsigned words; 0 stands for none.
__device__ __forceinline__ unsigned long long rank_key(double v) {
    const long long u = __double_as_longlong(v + 0.0);
    return (unsigned long long)(u < 0 ? ~u : u | (long long)0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t order32(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long rank_key(float high, float low) {
    return (unsigned long long)order32(high) << 32 | order32(low);
}

// Sums of two fp32 values as a value and what it cut off, which is half a step of it at most.
__device__ __forceinline__ float2 two_sum(float a, float b) {
    const float t = a + b, u = t - a;
    return make_float2(t, (a - (t - u)) + (b - u));
}

__device__ __forceinline__ float2 times(float2 a, float2 b) {
    const float t = a.x * b.x;
    return two_sum(t, fmaf(a.x, b.x, -t) + fmaf(a.x, b.y, a.y * b.x));
}

// log(z 2^-shift), z > 0, to 1e-9 as such a pair: z 2^-shift = m 2^e with m in [0.7, 1.42], log m =
// 2 artanh(t), t = (m - 1) / (m + 1), by its series, of which only the first term needs two parts.
__device__ __forceinline__ float2 beam_log(unsigned long long z, int shift) {
    int e = 63 - __clzll((long long)z);
    z <<= 63 - e;
    e -= shift;
    float mh = (float)(uint32_t)(z >> 40) * 0x1p-23f, ml = (float)((uint32_t)(z >> 16) & 0xFFFFFFu) * 0x1p-47f;
    if (mh > 1.41421356f) mh *= 0.5f, ml *= 0.5f, ++e;
    const float2 d = two_sum(1.0f, mh);
    const float r = __frcp_rn(d.x), n = mh - 1.0f, q = n * r;
    const float rest = (fmaf(-q, d.y + ml, fmaf(-q, d.x, n)) + ml) * r;
    const float t2 = q * q;
    float c = 1.0f / 11;
    c = fmaf(c, t2, 1.0f / 9);
    c = fmaf(c, t2, 1.0f / 7);
    c = fmaf(c, t2, 1.0f / 5);
    c = fmaf(c, t2, 1.0f / 3);
    const float f = (float)e;
    const float2 a = two_sum(f * 0.693145751953125f, 2.0f * q);  // 15 bits of log 2: exact
    return two_sum(a.x, a.y + (f * 1.42860682030941723212e-6f + (2.0f * rest + 2.0f * q * t2 * c)));
}
// n^-p, n >= 1, 0 <= p <= 16, to 1e-8: the exponential by its series to the ninth power.
__device__ __forceinline__ double beam_scale(int n, double p) {
    const float2 l = beam_log((unsigned long long)n, 0);
    const double y = -p * ((double)l.x + (double)l.y);
    const float k = rintf((float)y * 1.44269504f);
    const double r = fma((double)k, -0.69314718055994530942, y);
    double e = 1.0 / 362880;
    e = fma(e, r, 1.0 / 40320);
    e = fma(e, r, 1.0 / 5040);
    e = fma(e, r, 1.0 / 720);
    e = fma(e, r, 1.0 / 120);
    e = fma(e, r, 1.0 / 24);
    e = fma(e, r, 1.0 / 6);
    e = fma(e, r, 0.5);
    e = fma(e, r, 1.0);
    e = fma(e, r, 1.0);
    return __longlong_as_double(__double_as_longlong(e) + ((long long)k << 52));
}

__device__ __forceinline__ int beam_length(int n, bool ended) { return ended || n == INT32_MAX ? n : n + 1; }

struct BeamPick {  // shared memory of a request
    double scale[BEAM_MAX_WIDTH];
    float score[BEAM_MAX_WIDTH];
    float2 norm[BEAM_MAX_WIDTH], diff[BEAM_MAX_WIDTH], pair[BEAM_MAX_WIDTH];  // pairs; diff: score - norm, pair: scale
    unsigned long long lkey[BP_LIST], bkey[BEAM_MAX_K], gmax[BR_THREADS], wkey[BR_THREADS / 32];
    uint32_t lat[BP_LIST], bat[BEAM_MAX_K], wat[BR_THREADS / 32];
    float lscore[BP_LIST], bscore[BEAM_MAX_K];
    unsigned long long bound;
    int listed, wide;              // wide: ranks go by doubles
    uint8_t kind[BEAM_MAX_WIDTH];  // 0 none, 1 a row's candidates, 2 ended: itself
};

// The k best of request g from what its rows' chunks left.
__device__ __forceinline__ void beam_pick(const BeamSelectParams &p, BeamPick &s, int g) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.k;
    const int of_beam = p.chunks * k, total = p.W * of_beam;
    const unsigned long long *keys = p.keys + (int64_t)g * total;
    unsigned long long word[BP_EACH];  // asked for first, needed last
#pragma unroll
    for (int i = 0; i < BP_EACH; ++i) {
        const int j = i * BR_THREADS + tid;
        word[i] = j < total ? __ldcg(keys + j) : 0ull;
    }
    if (tid == 0) s.wide = 0;
    __syncthreads();
    for (int b = warp; b < p.W; b += BR_THREADS / 32) {  // a warp a beam: its norm
        const int64_t row = (int64_t)g * p.W + b;
        const float *tops = p.tops + row * p.chunks;
        const unsigned long long *sums = p.sums + row * p.chunks;
        const float score = p.scores[row];
        float mine = lane < p.chunks ? __ldcg(tops + lane) : -INFINITY, top = -INFINITY;
        unsigned long long q = lane < p.chunks ? __ldcg(sums + lane) : 0ull, sum = 0;
        int kind = fabsf(score) < INFINITY ? (p.ended && p.ended[row] ? 2 : 1) : 0;
        if (kind == 1) {
            for (int c = lane; c < p.chunks; c += 32) top = fmaxf(top, c == lane ? mine : __ldcg(tops + c));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            for (int c = lane; c < p.chunks; c += 32) {
                if (c != lane) mine = __ldcg(tops + c), q = __ldcg(sums + c);
                float f, unused;
                unpack2(exp_pair(both(fmaxf(mine, -FLT_MAX) - fmaxf(top, -FLT_MAX))), f, unused);
                // q f, f <= 1, cut to a unit of 2^-40: f 2^63 holds all of f's bits, which stand far down where
                // this chunk lies far below the row's top (q may be 8192 terms; of f 2^31 they took off 3e-5)
                sum += __umul64hi(q << 1, (unsigned long long)(f * 0x1p63f));
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (sum == 0) sum = ~0ull;  // 2^24 terms of 1: 2^64
            if (top == -INFINITY) kind = 0;
        }
        if (lane == 0) {
            float2 norm = make_float2(0.0f, 0.0f);
            if (kind == 1) {
                const float2 l = beam_log(sum, 40);
                norm = two_sum(top, l.x);
                norm = two_sum(norm.x, norm.y + l.y);
            }
            float2 diff = two_sum(score, -norm.x);
            diff = two_sum(diff.x, diff.y - norm.y);
            s.score[b] = score, s.kind[b] = (uint8_t)kind, s.norm[b] = norm, s.diff[b] = diff;
            if (kind && !(fabsf(diff.x) < 1e30f)) s.wide = 1;  // a logit added in fp32 might overflow
        }
    }
    if (p.penalty != 0.0 && tid >= BR_THREADS - BEAM_MAX_WIDTH) {
        const int b = tid - (BR_THREADS - BEAM_MAX_WIDTH);
        const int64_t row = (int64_t)g * p.W + b;
        if (b < p.W) {
            const double c = beam_scale(max(1, beam_length(p.lengths[row], p.ended && p.ended[row])), p.penalty);
            const float high = (float)c;
            s.scale[b] = c, s.pair[b] = make_float2(high, (float)(c - (double)high));
            if (high < 1e-15f) s.wide = 1;  // the low parts would fall below fp32's numbers
        }
    }
    __syncthreads();
    const int M = beam_groups(k, BR_THREADS), per = BR_THREADS / M;
    const bool wide = s.wide != 0, ranked = p.penalty != 0.0;
    int have = 0;  // in bkey, bat, bscore, best first
    for (int base = 0; base < total; base += BR_THREADS * BP_EACH) {
        unsigned long long key[BP_EACH], mine = 0;
        uint32_t at[BP_EACH];
        float score[BP_EACH];
#pragma unroll
        for (int i = 0; i < BP_EACH; ++i) {
            const int j = base + i * BR_THREADS + tid;
            key[i] = 0, at[i] = 0, score[i] = 0.0f;
            if (j < total) {
                const int b = j / of_beam, kind = s.kind[b];
                const unsigned long long w = base ? __ldcg(keys + j) : word[i];
                if (kind == 1 && w) {
                    const float x = key_value(w);
                    at[i] = (uint32_t)b * (uint32_t)p.V + ~(uint32_t)w;
                    if (wide) {
                        const double d = (double)s.score[b] + (double)x - ((double)s.norm[b].x + (double)s.norm[b].y);
                        key[i] = rank_key(ranked ? d * s.scale[b] : d), score[i] = (float)d;
                    } else {
                        float2 d = two_sum(s.diff[b].x, x);
                        d = two_sum(d.x, d.y + s.diff[b].y);
                        score[i] = d.x;
                        if (ranked) d = times(d, s.pair[b]);
                        key[i] = rank_key(d.x, d.y);
                    }
                } else if (kind == 2 && j == b * of_beam) {
                    at[i] = (uint32_t)b * (uint32_t)p.V + (uint32_t)p.end_token;
                    score[i] = s.score[b];
                    const float2 d = ranked && !wide ? times(make_float2(s.score[b], 0.0f), s.pair[b]) : make_float2(s.score[b], 0.0f);
                    key[i] = !wide ? rank_key(d.x, d.y) : rank_key(ranked ? (double)s.score[b] * s.scale[b] : (double)s.score[b]);
                }
            }
            mine = max(mine, key[i]);
        }
        {
            unsigned long long w = mine;
            if (per == 1) s.gmax[tid] = w;
#pragma unroll
            for (int off = 1; off < 32; off *= 2) {
                w = max(w, __shfl_xor_sync(0xffffffffu, w, off));
                if (2 * off == per && (lane & (per - 1)) == 0) s.gmax[tid / per] = w;
            }
        }
        if (tid == 0) s.listed = have, s.bound = 0ull;
        if (tid < have) s.lkey[tid] = s.bkey[tid], s.lat[tid] = s.bat[tid], s.lscore[tid] = s.bscore[tid];
        __syncthreads();
        if (tid < M) {
            const unsigned long long m = s.gmax[tid];
            int ahead = 0;
            for (int j = 0; j < M; ++j) ahead += s.gmax[j] > m || (s.gmax[j] == m && j < tid);
            if (ahead == k - 1) s.bound = m;
        }
        __syncthreads();
        unsigned long long least = max(s.bound, 1ull);
        if (have == k) least = max(least, s.bkey[k - 1]);
        if (mine >= least) {
#pragma unroll
            for (int i = 0; i < BP_EACH; ++i)
                if (key[i] >= least) {
                    const int n = atomicAdd(&s.listed, 1);
                    if (n < BP_LIST) s.lkey[n] = key[i], s.lat[n] = at[i], s.lscore[n] = score[i];
                }
        }
        __syncthreads();
        const int n = s.listed;
        if (n <= BP_LIST) {
            for (int i = tid; i < n; i += BR_THREADS) {
                const unsigned long long m = s.lkey[i];
                const uint32_t a = s.lat[i];
                int ahead = 0;
                for (int j = 0; j < n; ++j) ahead += s.lkey[j] > m || (s.lkey[j] == m && s.lat[j] < a);
                if (ahead < k) s.bkey[ahead] = m, s.bat[ahead] = a, s.bscore[ahead] = s.lscore[i];
            }
            have = min(n, k);
        } else {  // one by one, from what is held so far (b) and registers
            unsigned long long last = ~0ull;
            uint32_t last_at = 0;
            const unsigned long long bk = tid < have ? s.bkey[tid] : 0ull;
            const uint32_t ba = tid < have ? s.bat[tid] : 0u;
            const float bs = tid < have ? s.bscore[tid] : 0.0f;
            for (int r = 0; r < k; ++r) {
                unsigned long long best = 0;
                uint32_t best_at = ~0u;
                float best_score = 0.0f;
#pragma unroll
                for (int i = 0; i <= BP_EACH; ++i) {
                    const unsigned long long m = i < BP_EACH ? key[i < BP_EACH ? i : 0] : bk;
                    const uint32_t a = i < BP_EACH ? at[i < BP_EACH ? i : 0] : ba;
                    const bool after = m < last || (m == last && a > last_at);
                    if (m && after && (m > best || (m == best && a < best_at)))
                        best = m, best_at = a, best_score = i < BP_EACH ? score[i < BP_EACH ? i : 0] : bs;
                }
                const unsigned long long own = best;
                const uint32_t own_at = best_at;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    const unsigned long long m = __shfl_xor_sync(0xffffffffu, best, off);
                    const uint32_t a = __shfl_xor_sync(0xffffffffu, best_at, off);
                    if (m > best || (m == best && a < best_at)) best = m, best_at = a;
                }
                __syncthreads();
                if (lane == 0) s.wkey[warp] = best, s.wat[warp] = best_at;
                __syncthreads();
                best = s.wkey[0], best_at = s.wat[0];
                for (int i = 1; i < BR_THREADS / 32; ++i)
                    if (s.wkey[i] > best || (s.wkey[i] == best && s.wat[i] < best_at)) best = s.wkey[i], best_at = s.wat[i];
                if (best && own == best && own_at == best_at) s.bkey[r] = best, s.bat[r] = best_at, s.bscore[r] = best_score;
                last = best, last_at = best_at;
            }
            have = k;  // the list ran over, so there are k
        }
        __syncthreads();
    }
    if (tid >= k) return;
    const int64_t out = (int64_t)g * k + tid;
    int32_t token = -1, parent = -1, length = 0;
    float score = -INFINITY;
    bool ended = false;
    if (tid < have) {
        const uint32_t a = s.bat[tid];
        parent = (int32_t)(a / (uint32_t)p.V);
        token = (int32_t)(a - (uint32_t)parent * (uint32_t)p.V);
        score = s.bscore[tid];
        const bool itself = s.kind[parent] == 2;
        if (p.lengths) length = beam_length(p.lengths[(int64_t)g * p.W + parent], itself);
        ended = itself || token == p.end_token;
    }
    p.tokens[out] = token, p.parents[out] = parent, p.scores_out[out] = score;
    if (p.lengths_out) p.lengths_out[out] = length;
    if (p.ended_out) p.ended_out[out] = ended;
}

template <int T, int E, bool GRID>
__global__ void __launch_bounds__(BR_THREADS, 4) beam_select_kernel(const BeamSelectParams p) {
    __shared__ union Shared {
        BeamRows rows;
        BeamPick pick;
        __device__ Shared() {}
    } s;
    __shared__ bool last;
    const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks, g = row / p.W;
    // of a beam that has ended or has no score nothing is read
    if (fabsf(p.scores[row]) < INFINITY && !(p.ended && p.ended[row])) beam_chunk<T, E, GRID>(p, s.rows, row, chunk);
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const uint32_t n = (uint32_t)p.W * p.chunks;
        last = atomicAdd(&p.tickets[g], 1u) == n - 1;
        if (last) p.tickets[g] = 0u;  // for the next call
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    beam_pick(p, s.pick, g);
}

// ---------------------------------------------------------------------------
// Reordering.  The state of a beam is where its slot says, so that most of a reordering
// is a new table of slots: a parent's first child keeps the parent's slot.  Only the
// parent's other children need a state of their own, and there are as many of them as
// beams without children, whose slots they take.  No slot is read and written, so all
// copies may run at once and in place; a state with several new copies is read once.
//
// Every CTA works the plan out for itself (up to 1024 beams, in shared memory), which
// takes less time than a launch of its own, then takes its share of the heads: 16 KB
// read and, for every copy, written.  Memory bounds it: 32 states of the 2.9B shape, 1.38 GB, 227 us
// (6.1 TB/s; the copy rate would take 204), one of the 7.2B shape to 15 slots, 0.55 GB, 94 us (5.9; 82).
// ---------------------------------------------------------------------------
constexpr int RO_THREADS = 256;
constexpr int RO_EACH = BEAM_MAX_SLOTS / RO_THREADS;  // beams a thread plans for
constexpr int RO_TABLE = 2 * BEAM_MAX_SLOTS;
constexpr int RO_HEAD = HS * HS;

struct ReorderShared {
    int32_t slot[BEAM_MAX_SLOTS];
    int32_t children[BEAM_MAX_SLOTS];  // of each beam; then where the next copy of it goes in `to`
    int32_t first[BEAM_MAX_SLOTS];     // its first child
    int32_t to[BEAM_MAX_SLOTS];        // slots of copies, a source's next to one another
    int32_t table[RO_TABLE];           // beams by slot
    unsigned long long total[RO_THREADS / 32];
    int16_t parent[BEAM_MAX_SLOTS];
    uint16_t source[BEAM_MAX_SLOTS];     // beams copied from
    uint16_t start[BEAM_MAX_SLOTS + 1];  // where a source's copies start in `to`
    uint16_t free[BEAM_MAX_SLOTS];       // beams without children
    uint16_t place[BEAM_MAX_SLOTS];      // which of those gives this beam its slot (RO_STAYS: its parent does)
    uint8_t bad[BEAM_MAX_SLOTS];         // requests left out
    int sources;
};
constexpr uint16_t RO_STAYS = 0xFFFF;

__global__ void __launch_bounds__(RO_THREADS) reorder_kernel(const ReorderParams p) {
    __shared__ ReorderShared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.G * p.W, W = p.W;
    for (int i = tid; i < RO_TABLE; i += RO_THREADS) s.table[i] = -1;
    for (int i = tid; i < n; i += RO_THREADS) {
        const int parent = p.parents[i];
        s.slot[i] = p.slots[i];
        s.parent[i] = (int16_t)(parent >= -1 && parent < W ? parent : W);
        s.children[i] = 0, s.first[i] = n;
        if (i < p.G) s.bad[i] = 0;
    }
    __syncthreads();
    // A request is left out where an index is out of range or a slot is met twice in the call.
    for (int i = tid; i < n; i += RO_THREADS) {
        const int slot = s.slot[i], parent = s.parent[i], g = i / W;
        if (parent == W) s.bad[g] = 1;
        else if (parent >= 0) atomicAdd(&s.children[g * W + parent], 1), atomicMin(&s.first[g * W + parent], i);
        if ((uint32_t)slot >= (uint32_t)p.n_slots) {
            s.bad[g] = 1;
            continue;
        }
        uint32_t h = (uint32_t)slot * 2654435761u >> 21;  // 11 bits; the table is at most half full
        for (int tries = 0; tries < RO_TABLE; ++tries, h = (h + 1) % RO_TABLE) {
            const int old = atomicCAS(&s.table[h], -1, i);
            if (old < 0) break;
            if (s.slot[old] == slot) {
                s.bad[g] = s.bad[old / W] = 1;
                break;
            }
        }
    }
    __syncthreads();
    // How many beams before each one need a slot, have no child, are copied, and their copies: four
    // counts of 16 bits.  A request has as many that need a slot as have no child, so the n-th of
    // those in the call and the n-th of these are of one request.
    unsigned long long count[RO_EACH], sum = 0;
#pragma unroll
    for (int e = 0; e < RO_EACH; ++e) {
        const int i = tid * RO_EACH + e;
        unsigned long long c = 0;
        if (i < n && !s.bad[i / W]) {
            const int parent = s.parent[i], mine = s.children[i];
            c = !(parent >= 0 && s.first[i / W * W + parent] == i);
            c |= (unsigned long long)(mine == 0) << 16;
            if (mine > 1) c |= 1ull << 32 | (unsigned long long)(mine - 1) << 48;
        }
        count[e] = c, sum += c;
    }
    unsigned long long before = sum;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before += o;
    }
    if (lane == 31) s.total[warp] = before;
    __syncthreads();
    before -= sum;
    for (int i = 0; i < warp; ++i) before += s.total[i];
#pragma unroll
    for (int e = 0; e < RO_EACH; ++e) {
        const int i = tid * RO_EACH + e;
        const unsigned long long c = count[e];
        if (i < n) {
            s.place[i] = c & 1 ? (uint16_t)before : RO_STAYS;
            if (c >> 16 & 1) s.free[before >> 16 & 0xFFFF] = (uint16_t)i;
            if (c >> 32 & 1) {
                const int at = (int)(before >> 32 & 0xFFFF);
                s.source[at] = (uint16_t)i, s.start[at] = (uint16_t)(before >> 48);
                s.children[i] = (int)(before >> 48);
            }
        }
        before += c;
    }
    if (tid == RO_THREADS - 1) {
        s.sources = (int)(before >> 32 & 0xFFFF);
        s.start[s.sources] = (uint16_t)(before >> 48);
    }
    __syncthreads();
    for (int i = tid; i < n; i += RO_THREADS) {
        const int g = i / W, parent = s.parent[i];
        int slot = -1;
        if (!s.bad[g]) {
            if (s.place[i] == RO_STAYS) {
                slot = s.slot[g * W + parent];
            } else {
                slot = s.slot[s.free[s.place[i]]];
                if (parent >= 0) s.to[atomicAdd(&s.children[g * W + parent], 1)] = slot;
            }
        }
        if (blockIdx.x == 0) {
            p.slots_out[i] = slot;
            if (slot < 0 && p.err) atomicOr(p.err, ERR_SLOT);
        }
    }
    __syncthreads();
    const int heads = p.L * p.H;
    // An item: a source's head, and all its copies, whose order is each CTA's own.  (Four copies an item,
    // in one order, took 109 us where this takes 94: one 7.2B state to 15 slots.)
    int at = 0;
    int64_t begin = 0;  // the source's first item
    for (int64_t item = blockIdx.x;; item += gridDim.x) {
        while (item >= begin + heads && at < s.sources) begin += heads, ++at;
        if (at >= s.sources) break;
        const int hl = (int)(item - begin), layer = hl / p.H, head = hl - layer * p.H;
        const int c0 = s.start[at], c1 = s.start[at + 1];
        const int64_t src = (int64_t)layer * p.n_slots + s.slot[s.source[at]];
        const float *w = p.wkv + (src * p.H + head) * RO_HEAD;
        float v[2][8];
        ld_v8(v[0], w + tid * 8);
        ld_v8(v[1], w + tid * 8 + RO_HEAD / 2);
        float4 t;
        float *shift = tid < HS / 4 ? p.att : p.ffn;
        const int64_t ch = head * HS + (tid % (HS / 4)) * 4, d = (int64_t)p.H * HS;
        if (tid < HS / 2) t = *(const float4 *)(shift + src * d + ch);
        for (int c = c0; c < c1; ++c) {
            const int64_t dst = (int64_t)layer * p.n_slots + s.to[c];
            float *o = p.wkv + (dst * p.H + head) * RO_HEAD;
            st_v8(o + tid * 8, v[0]);
            st_v8(o + tid * 8 + RO_HEAD / 2, v[1]);
            if (tid < HS / 2) *(float4 *)(shift + dst * d + ch) = t;
            if (p.occ) {
                const int64_t a = (int64_t)p.V * hl / heads, b = (int64_t)p.V * (hl + 1) / heads;
                for (int64_t e = a + tid; e < b; e += RO_THREADS) p.occ[(int64_t)s.to[c] * p.V + e] = 0.0f;
                if (hl == 0 && tid == 0) p.ndraw[s.to[c]] = 0ull;
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

thread_local char g_beam_msg[192];

int beam_fail(const char **err_msg, int code, const char *fmt, long long a = 0, long long b = 0) {
    snprintf(g_beam_msg, sizeof g_beam_msg, fmt, a, b);
    if (err_msg) *err_msg = g_beam_msg;
    return code;
}
int beam_done(const char **err_msg, const char *what, cudaError_t e) {
    if (e == cudaSuccess) return RWKV7_OK;
    snprintf(g_beam_msg, sizeof g_beam_msg, "%s: %s", what, cudaGetErrorString(e));
    if (err_msg) *err_msg = g_beam_msg;
    return RWKV7_ECUDA;
}

constexpr int BEAM_SHORT = 8, BEAM_LONG = 32;  // values of a thread of beam_select_kernel
int beam_chunks(int V, int each) { return (V + BR_THREADS * each - 1) / (BR_THREADS * each); }

template <int T, bool GRID>
const void *beam_select_fn(bool longer) {
    return longer ? (const void *)beam_select_kernel<T, BEAM_LONG, GRID> : (const void *)beam_select_kernel<T, BEAM_SHORT, GRID>;
}
template <int T>
const void *beam_select_fn(bool longer, bool grid) {
    return grid ? beam_select_fn<T, true>(longer) : beam_select_fn<T, false>(longer);
}

bool share(const void *a, size_t an, const void *b, size_t bn) {
    return a && b && mx_share(MxSpan(a, 1, (int64_t)an, 0, 1), MxSpan(b, 1, (int64_t)bn, 0, 1));
}

}  // namespace

int rk::beam_reorder(ReorderParams &p, void *stream, const char **err_msg) {
    if (err_msg) *err_msg = "";
    if (p.L < 1 || p.H < 1 || p.n_slots < 1 || p.H > RWKV7_MX_MAX_DIM / p.L)
        return beam_fail(err_msg, RWKV7_EINVAL, "layers, heads and slots must be >= 1");
    if (p.G < 0 || p.W < 1 || p.W > BEAM_MAX_WIDTH || p.G > BEAM_MAX_SLOTS / p.W)
        return beam_fail(err_msg, RWKV7_EINVAL,
                         "%lld requests of %lld beams: at most 128 beams a request and 1024 in a call", p.G, p.W);
    if (p.G == 0) return RWKV7_OK;
    if (!p.wkv || !p.att || !p.ffn || !p.slots || !p.parents || !p.slots_out)
        return beam_fail(err_msg, RWKV7_EINVAL, "null pointer argument");
    if (((uintptr_t)p.wkv & 31u) || (((uintptr_t)p.att | (uintptr_t)p.ffn) & 15u))
        return beam_fail(err_msg, RWKV7_EINVAL, "wkv must be 32-byte aligned, the shift states 16-byte aligned");
    if (((uintptr_t)p.slots | (uintptr_t)p.parents | (uintptr_t)p.slots_out) & 3u)
        return beam_fail(err_msg, RWKV7_EINVAL, "the index arrays must be 4-byte aligned");
    const size_t bytes = (size_t)p.G * p.W * 4;
    if (share(p.slots_out, bytes, p.slots, bytes) || share(p.slots_out, bytes, p.parents, bytes))
        return beam_fail(err_msg, RWKV7_EINVAL, "the new slots overlap the old ones or the parents");
    // A source has two children at least.
    const int64_t items = (int64_t)p.G * (p.W / 2) * p.L * p.H;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items < 1 ? 1 : items < 152 * 5 ? items : 152 * 5));
    cfg.blockDim = dim3(RO_THREADS);
    cfg.stream = static_cast<cudaStream_t>(stream);
    void *args[] = {&p};
    return beam_done(err_msg, "reordering", cudaLaunchKernelExC(&cfg, (const void *)reorder_kernel, args));
}

extern "C" {

size_t rwkv7_beam_room_bytes(int32_t requests, int32_t width, int32_t vocab, int32_t k) {
    if (requests < 0 || width < 1 || width > BEAM_MAX_WIDTH || vocab < 1 || vocab > RWKV7_MX_MAX_DIM || k < 1 ||
        k > BEAM_MAX_K || requests > RWKV7_MX_MAX_DIM / width)
        return 0;
    // (For seven values more than there are: a size that callers know by now.)
    return (size_t)requests * width * beam_chunks(vocab + 7, BEAM_SHORT) * (8 * (size_t)k + 12) + 16;
}

int rwkv7_beam_select(const void *d_logits, int32_t dtype, int64_t ld, int32_t requests, int32_t width, int32_t vocab,
                      const float *d_scores, const uint8_t *d_ended, int32_t end_token, const int32_t *d_lengths,
                      double length_penalty, int32_t k, int32_t *d_tokens, int32_t *d_parents, float *d_scores_out,
                      int32_t *d_lengths_out, uint8_t *d_ended_out, void *d_room, uint32_t *d_tickets, void *cuda_stream,
                      const char **err_msg) {
    if (err_msg) *err_msg = "";
    if (requests < 0 || width < 1 || width > BEAM_MAX_WIDTH || requests > RWKV7_MX_MAX_DIM / width)
        return beam_fail(err_msg, RWKV7_EINVAL, "%lld requests of %lld beams: 1 .. 128 beams, at most 2^24 in all",
                         requests, width);
    if (vocab < 1 || vocab > RWKV7_MX_MAX_DIM)
        return beam_fail(err_msg, RWKV7_EINVAL, "a vocabulary of %lld: 1 .. 2^24", vocab);
    if (k < 1 || k > BEAM_MAX_K) return beam_fail(err_msg, RWKV7_EINVAL, "k=%lld is outside 1 .. %lld", k, BEAM_MAX_K);
    if (dtype < RWKV7_F32 || dtype > RWKV7_BF16) return beam_fail(err_msg, RWKV7_EINVAL, "unknown dtype %lld", dtype);
    const int64_t rows = (int64_t)requests * width;
    if (rows > 1 && ld < vocab) return beam_fail(err_msg, RWKV7_EINVAL, "row stride %lld is below vocab=%lld", ld, vocab);
    if (rows > INT32_MAX / beam_chunks(vocab, BEAM_SHORT))
        return beam_fail(err_msg, RWKV7_EINVAL, "%lld rows of %lld logits are too many", rows, vocab);
    if (!(length_penalty >= 0.0 && length_penalty <= 16.0))
        return beam_fail(err_msg, RWKV7_EINVAL, "length_penalty must be in 0 .. 16");
    if (length_penalty != 0.0 && !d_lengths)
        return beam_fail(err_msg, RWKV7_EINVAL, "a length penalty needs the beams' lengths");
    if (d_lengths_out && !d_lengths)
        return beam_fail(err_msg, RWKV7_EINVAL, "new lengths need the beams' lengths");
    if (end_token < -1 || end_token >= vocab)
        return beam_fail(err_msg, RWKV7_EINVAL, "end_token=%lld is outside -1 .. %lld", end_token, vocab - 1);
    if (d_ended && end_token < 0) return beam_fail(err_msg, RWKV7_EINVAL, "ended beams need an end_token");
    if (requests == 0) return RWKV7_OK;
    if (!d_logits || !d_scores || !d_tokens || !d_parents || !d_scores_out || !d_room || !d_tickets)
        return beam_fail(err_msg, RWKV7_EINVAL, "null pointer argument");
    const int size = dtype == RWKV7_F32 ? 4 : 2;
    if ((uintptr_t)d_logits % size) return beam_fail(err_msg, RWKV7_EINVAL, "the logits' pointer is not aligned to its type");
    if (((uintptr_t)d_scores | (uintptr_t)d_lengths | (uintptr_t)d_tokens | (uintptr_t)d_parents | (uintptr_t)d_scores_out |
         (uintptr_t)d_lengths_out | (uintptr_t)d_tickets) & 3u)
        return beam_fail(err_msg, RWKV7_EINVAL, "arrays of 32-bit values must be 4-byte aligned");
    if ((uintptr_t)d_room & 15u) return beam_fail(err_msg, RWKV7_EINVAL, "the room must be 16-byte aligned");
    BeamSelectParams p;
    memset(&p, 0, sizeof p);
    p.logits = d_logits, p.ld = ld;
    p.G = requests, p.W = width, p.V = vocab, p.k = k;
    p.scores = d_scores, p.ended = d_ended, p.end_token = end_token;
    p.lengths = d_lengths, p.penalty = length_penalty;
    p.tokens = d_tokens, p.parents = d_parents, p.scores_out = d_scores_out;
    p.lengths_out = d_lengths_out, p.ended_out = d_ended_out;
    {   // inputs and the room against what is written
        const size_t out = (size_t)requests * k, in = (size_t)rows;
        const void *w[] = {d_tokens, d_parents, d_scores_out, d_lengths_out, d_ended_out, d_room, d_tickets};
        const size_t wn[] = {4 * out, 4 * out, 4 * out, 4 * out, out, rwkv7_beam_room_bytes(requests, width, vocab, k),
                             4 * (size_t)requests};
        const void *r[] = {d_scores, d_lengths, d_ended};
        const size_t rn[] = {4 * in, 4 * in, in};
        for (int i = 0; i < 7; ++i) {
            bool meets = w[i] && mx_share(MxSpan(d_logits, rows, vocab, ld, size), MxSpan(w[i], 1, (int64_t)wn[i], 0, 1));
            for (int j = 0; j < 3; ++j) meets |= share(w[i], wn[i], r[j], rn[j]);
            for (int j = 0; j < i; ++j) meets |= share(w[i], wn[i], w[j], wn[j]);
            if (meets) return beam_fail(err_msg, RWKV7_EINVAL, "an output or the room overlaps an input or another output");
        }
    }
    // Chunks of 8192 values have a quarter of the barriers and lists of chunks of 2048; while they are
    // fewer than the SMs, the latter spread a row over more of them.  us with the longer / shorter ones: 32
    // rows of 65,536 values 10.8 / 13.0, 256 rows of 8,000 10.0 / 13.0, 256 rows of 2,000 (one
    // chunk either way) 9.9 / 8.2.
    const bool longer = beam_chunks(vocab, BEAM_SHORT) > 1 && rows * beam_chunks(vocab, BEAM_LONG) >= 152;
    p.chunks = beam_chunks(vocab, longer ? BEAM_LONG : BEAM_SHORT);
    const int64_t lists = rows * p.chunks;
    p.tickets = d_tickets;
    p.keys = static_cast<unsigned long long *>(d_room);
    p.sums = p.keys + lists * k;
    p.tops = reinterpret_cast<float *>(p.sums + lists);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)lists);
    cfg.blockDim = dim3(BR_THREADS);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    // Where every row is on the 16-byte grid, a kernel that moves nothing: 256 rows of 65,536 fp32 values 26.8 us,
    // 28.7 by the other, which takes 31.7 for 65,537; 256 of 65,536 and of 65,535 fp16 values 26.3 and 27.5.
    const bool grid = (uintptr_t)d_logits % 16 == 0 && (rows == 1 || ld * size % 16 == 0);
    const void *fn = dtype == RWKV7_F32   ? beam_select_fn<MX_F32>(longer, grid)
                     : dtype == RWKV7_F16 ? beam_select_fn<MX_F16>(longer, grid)
                                          : beam_select_fn<MX_BF16>(longer, grid);
    void *args[] = {&p};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    return beam_done(err_msg, "selecting beams", e);
}

int rwkv7_states_reorder(float *d_wkv, float *d_shift_att, float *d_shift_ffn, int32_t n_layer, int32_t n_head,
                         int32_t n_slots, const int32_t *d_slots, const int32_t *d_parents, int32_t requests,
                         int32_t width, int32_t *d_slots_out, void *cuda_stream, const char **err_msg) {
    ReorderParams p;
    memset(&p, 0, sizeof p);
    p.wkv = d_wkv, p.att = d_shift_att, p.ffn = d_shift_ffn;
    p.L = n_layer, p.H = n_head, p.n_slots = n_slots, p.G = requests, p.W = width;
    p.slots = d_slots, p.parents = d_parents, p.slots_out = d_slots_out;
    return beam_reorder(p, cuda_stream, err_msg);
}

}  // extern "C"
