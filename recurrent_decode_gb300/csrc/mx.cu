// mx.cu -- MXFP4 quantisation of rows and its inverse, and slot states saved to
// and loaded from a cache of MXINT8 or MXFP4 entries (formats: mx.cuh).
//
// All four kernels move each value once and do a handful of operations on it; eight
// neighbouring values belong to one lane and a block of 32 to four, whose largest
// value takes two shuffles.  Measured against the 6.8 TB/s of a plain copy:
//   states   sixteen of the 2.9B shape saved and loaded as MXINT8, 885 MB: 134 us, 6.6
//            TB/s; one 7.2B state saved and loaded into 48 slots, 1.7 GB: 259 us, 6.6.
//            Memory bounds them.  Stored 16 bytes a lane instead of 32 (two halves of
//            each sector at different times) the load took 341 us.
//   rows     4096 x 16384 bf16 to MXFP4, 170 MB: 29.7 us, 5.7 TB/s; back, 27.2 us, 6.3
//            TB/s.  Instructions come close to bounding them (issue slots 63-68 % busy):
//            one line a warp instead of four took 59 and 45 us; for 64 x 2560 four lines
//            a warp took 2.3 us instead of 1.6.  Four lines along a row instead of down a
//            column tile took 28.1 us there, but 30 instead of 23 for 65536 x 300 fp16,
//            whose rows end inside them.  Rows off the 16-byte grid, 8192 x 4001 fp16:
//            25 us and 18 back, against 17.5 and 15 for 4000 columns.
#include <cstdio>
#include <cstring>

#include "../../include/rwkv7.h"
#include "mx.cuh"

namespace rk {

struct MxRowsParams {
    void *x;  // [rows] at ld
    int64_t cols, ld;
    uint8_t *mx;
    int rows, kt;   // rows, column tiles
    int vec;        // the lanes' eight values start on 16-byte (fp32: 32-byte) boundaries in every row
    int per;        // rows of one column tile that a warp takes (1 or MXQ_LINES)
    int groups;     // such groups: ceil(rows / per) * kt
};

constexpr int MXQ_THREADS = 256;
constexpr int MXQ_LINES = 4;  // lines of a warp at most, their loads issued together
// From here on a warp takes them all: 64 warps for each SM are there without it, and
// with fewer lines one a warp spreads them over more SMs.
constexpr int MXQ_MANY = 152 * 64;

// A warp's lines (a line: 256 columns of a row): up to MXQ_LINES consecutive rows of one
// column tile.
template <typename E>
struct MxLines {
    E *x;            // the first line's values; the next lines' p.ld apart
    uint8_t *codes;  // its codes; the next lines' 128 bytes apart
    uint8_t *power;  // the word of powers of the lane's half; the next lines' 16 bytes apart
    int at, place;   // a lane's bytes within its block's codes; the block's place in the first line
    int n, cols;     // lines, columns of them that the matrix has
    __device__ __forceinline__ MxLines(const MxRowsParams &p, int group, int lane) {
        const int g = group / p.kt, t = group - g * p.kt, r = g * p.per, rr = r % MX_TILE_M;
        n = min(p.per, p.rows - r);
        cols = (int)min((int64_t)MX_TILE_K, p.cols - (int64_t)t * MX_TILE_K);
        x = (E *)p.x + r * p.ld + (int64_t)t * MX_TILE_K;
        uint8_t *tile = p.mx + ((int64_t)(r / MX_TILE_M) * p.kt + t) * MX_TILE_BYTES;
        codes = tile + MX_SCALE_BYTES + rr * 128;
        power = tile + (lane >> 4) * 512 + (rr & 31) * 16 + (rr >> 5) * 4;
        at = (lane & 3) * 4;
        place = (lane >> 2) ^ (rr & 7);
    }
    // Line l's.  Several lines start at a multiple of MXQ_LINES, so that l only sets low
    // bits of the row.
    __device__ __forceinline__ uint32_t *code(int l) const {
        return (uint32_t *)(codes + l * 128 + ((place ^ l) << 4) + at);
    }
};

// Eight values a lane.  Rows off the 16-byte grid are turned through shared memory.
template <int T>
__global__ void __launch_bounds__(MXQ_THREADS) mx4_quantize_kernel(const MxRowsParams p) {
    using L = MxElem<T>;
    using E = typename L::type;
    __shared__ __align__(16) E room[MXQ_THREADS / 32][MX_TILE_K];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = blockIdx.x * (MXQ_THREADS / 32) + warp;
    pdl_launch();  // a product of these rows may start fetching its weights
    if (group >= p.groups) return;
    const MxLines<E> in(p, group, lane);
    typename L::Eight u[MXQ_LINES];
    uint32_t w;
    if (p.vec && in.n == MXQ_LINES && in.cols == MX_TILE_K) {  // the usual case
#pragma unroll
        for (int l = 0; l < MXQ_LINES; ++l) L::load(u[l], in.x + l * p.ld + lane * 8);
#pragma unroll
        for (int l = 0; l < MXQ_LINES; ++l) {
            *in.code(l) = mx4_line<T>(u[l], w);
            if ((lane & 15) == 0) *(uint32_t *)(in.power + l * 16) = w;
        }
        return;
    }
    E edge[MXQ_LINES];
#pragma unroll
    for (int l = 0; l < MXQ_LINES; ++l) {
        if (l >= in.n) break;
        const E *x = in.x + l * p.ld;
        if (!p.vec) {
            L::gather(u[l], edge[l], x, in.cols, lane);
        } else if (lane * 8 + 8 <= in.cols) {
            L::load(u[l], x + lane * 8);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) L::set(u[l], i, lane * 8 + i < in.cols ? x[lane * 8 + i] : L::down(0.0f));
        }
    }
#pragma unroll
    for (int l = 0; l < MXQ_LINES; ++l) {
        if (l >= in.n) break;
        if (!p.vec) {
            __syncwarp();
            L::turn(u[l], edge[l], in.x + l * p.ld, room[warp], lane);
        }
        *in.code(l) = mx4_line<T>(u[l], w);
        if ((lane & 15) == 0) *(uint32_t *)(in.power + l * 16) = w;
    }
}

template <int T>
__global__ void __launch_bounds__(MXQ_THREADS) mx4_dequantize_kernel(const MxRowsParams p) {
    using L = MxElem<T>;
    using E = typename L::type;
    __shared__ __align__(16) E room[MXQ_THREADS / 32][MX_TILE_K];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = blockIdx.x * (MXQ_THREADS / 32) + warp;
    if (group >= p.groups) return;
    const MxLines<E> out(p, group, lane);
    uint32_t code[MXQ_LINES], s[MXQ_LINES];
    if (p.vec && out.n == MXQ_LINES && out.cols == MX_TILE_K) {  // the usual case
#pragma unroll
        for (int l = 0; l < MXQ_LINES; ++l) code[l] = *out.code(l), s[l] = out.power[l * 16 + ((lane >> 2) & 3)];
#pragma unroll
        for (int l = 0; l < MXQ_LINES; ++l) {
            float v[8];
            mx4_values(code[l], s[l], v);
            L::store(out.x + l * p.ld + lane * 8, v);
        }
        return;
    }
#pragma unroll
    for (int l = 0; l < MXQ_LINES; ++l) {
        if (l >= out.n) break;
        code[l] = *out.code(l), s[l] = out.power[l * 16 + ((lane >> 2) & 3)];
    }
#pragma unroll
    for (int l = 0; l < MXQ_LINES; ++l) {
        if (l >= out.n) break;
        float v[8];
        mx4_values(code[l], s[l], v);
        E *x = out.x + l * p.ld;
        if (!p.vec) {
            __syncwarp();
            L::store_aligned(room[warp] + lane * 8, v);
            __syncwarp();
            L::scatter(x, room[warp], out.cols, lane);
        } else if (lane * 8 + 8 <= out.cols) {
            L::store(x + lane * 8, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (lane * 8 + i < out.cols) x[lane * 8 + i] = L::down(v[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// States.  An entry holds one slot's state: codes of wkv [L][H][64][64], then
// the powers [L][H][128] (blocks of 32 along a state row), then the two shift
// states [L][2][d] as they are (3 % of the fp32 state; every later token mixes
// them in unscaled, so they stay exact).
// ---------------------------------------------------------------------------
constexpr int MXS_THREADS = 256;
constexpr int MX_HEAD = HS * HS;  // values of one head's state
constexpr int MXS_GROUPS = MX_HEAD / 8 / MXS_THREADS;  // groups of eight values a thread takes

struct MxStateParams {
    float *wkv, *att, *ffn;  // [L][n_slots][H][64][64], [L][n_slots][d] twice
    int L, H, n_slots, n_entries;
    const int32_t *slots, *entries;
    uint8_t *cache;
    int64_t entry_bytes;
    uint32_t *err;
    // load into a ctx: what a slot restarts with its new state (else null)
    float *occ;
    unsigned long long *ndraw;
    int V;
};

__host__ __device__ constexpr int64_t mx_codes(int64_t heads, int fmt) {
    return heads * (fmt == MXINT8 ? MX_HEAD : MX_HEAD / 2);
}

// Whether this CTA's pair i is one to carry out: both indices in range, and no
// earlier pair that writes the same target (one of two copies into the same place
// would win by chance: the first does, the others are reported).  A pair whose other
// index is out of range writes nothing, so it makes no later one a repeat.
__device__ __forceinline__ bool mx_pair_ok(const int32_t *target, int32_t t, int ntarget, const int32_t *other, int32_t o,
                                           int nother, int i, uint32_t *err, bool speak) {
    int dup = 0;  // both loads of a pair at once: with the second only where the first is met, 0.2 us more
    for (int j = threadIdx.x; j < i; j += MXS_THREADS) dup |= (target[j] == t) & ((uint32_t)other[j] < (uint32_t)nother);
    dup = __syncthreads_or(dup);
    const bool in = (uint32_t)t < (uint32_t)ntarget && (uint32_t)o < (uint32_t)nother;
    if (speak && threadIdx.x == 0 && (dup || !in)) atomicOr(err, in ? ERR_DUP : ERR_SLOT);
    return in && !dup;
}

// CTA (h, i): head h (of all layers' heads) of pair i; two groups of eight values a thread.
template <int FMT, bool SAVE>
__global__ void __launch_bounds__(MXS_THREADS) mx_state_kernel(const MxStateParams p) {
    const int hl = blockIdx.x, i = blockIdx.y;
    const int layer = hl / p.H, head = hl % p.H;
    const int32_t slot = p.slots[i], entry = p.entries[i];
    if (!(SAVE ? mx_pair_ok(p.entries, entry, p.n_entries, p.slots, slot, p.n_slots, i, p.err, hl == 0)
               : mx_pair_ok(p.slots, slot, p.n_slots, p.entries, entry, p.n_entries, i, p.err, hl == 0)))
        return;
    const int64_t heads = (int64_t)p.L * p.H;
    uint8_t *at = p.cache + (int64_t)entry * p.entry_bytes;
    uint8_t *codes = at + mx_codes(hl, FMT);
    at += mx_codes(heads, FMT);
    uint8_t *scales = at + (int64_t)hl * (MX_HEAD / MX_BLOCK);
    at += heads * (MX_HEAD / MX_BLOCK);
    float *shift = (float *)at + (int64_t)layer * 2 * p.H * HS;
    float *st = p.wkv + (((int64_t)layer * p.n_slots + slot) * p.H + head) * MX_HEAD;
    if (threadIdx.x < 2 * HS / 4) {  // the head's 64 channels of both shift states
        const int which = threadIdx.x / (HS / 4), c = head * HS + (threadIdx.x % (HS / 4)) * 4;
        float4 *a = (float4 *)((which ? p.ffn : p.att) + ((int64_t)layer * p.n_slots + slot) * p.H * HS + c);
        float4 *b = (float4 *)(shift + (int64_t)which * p.H * HS + c);
        if (SAVE) *b = *a;
        else *a = *b;
    }
    if (!SAVE && p.occ) {
        const int64_t a = (int64_t)p.V * hl / heads, b = (int64_t)p.V * (hl + 1) / heads;
        for (int64_t k = a + threadIdx.x; k < b; k += MXS_THREADS) p.occ[(int64_t)slot * p.V + k] = 0.0f;
        if (hl == 0 && threadIdx.x == 0) p.ndraw[slot] = 0ull;
    }
    if constexpr (SAVE) {
        float v[MXS_GROUPS][8];
#pragma unroll
        for (int i = 0; i < MXS_GROUPS; ++i) ld_v8(v[i], st + (threadIdx.x + i * MXS_THREADS) * 8);
#pragma unroll
        for (int i = 0; i < MXS_GROUPS; ++i) {
            const int g = threadIdx.x + i * MXS_THREADS;
            const uint32_t s = mx_scale<FMT>(mx_quad_top(v[i]));
            const float f = mx_inverse(s);  // a block without a number: its codes do not matter
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= f;
            if constexpr (FMT == MXFP4) {
                ((uint32_t *)codes)[g] = fp4_pack8(v[i]);
            } else {
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int q = min(127, max(-127, __float2int_rn(v[i][j] * 64.0f)));
                    w[j >> 2] |= ((uint32_t)q & 255u) << (8 * (j & 3));
                }
                ((uint2 *)codes)[g] = make_uint2(w[0], w[1]);
            }
            if ((g & 3) == 0) scales[g >> 2] = (uint8_t)s;
        }
    } else {
        uint32_t s[MXS_GROUPS];
        uint2 w[MXS_GROUPS];
#pragma unroll
        for (int i = 0; i < MXS_GROUPS; ++i) {
            const int g = threadIdx.x + i * MXS_THREADS;
            s[i] = scales[g >> 2];
            if constexpr (FMT == MXFP4) w[i].x = ((const uint32_t *)codes)[g];
            else w[i] = ((const uint2 *)codes)[g];
        }
#pragma unroll
        for (int i = 0; i < MXS_GROUPS; ++i) {
            float v[8];
            if constexpr (FMT == MXFP4) {
                fp4_unpack8(w[i].x, v);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = (float)(int8_t)((j < 4 ? w[i].x : w[i].y) >> (8 * (j & 3))) * (1.0f / 64.0f);
            }
            const float f = s[i] == 255u ? __uint_as_float(0x7FC00000u) : mx_power(s[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= f;
            st_v8(st + (threadIdx.x + i * MXS_THREADS) * 8, v);
        }
    }
}

}  // namespace rk

// ---------------------------------------------------------------------------
// C entry points
// ---------------------------------------------------------------------------
using namespace rk;
namespace {

thread_local char g_mx_msg[192];

int mx_fail(const char **err_msg, int code, const char *fmt, long long a = 0, long long b = 0) {
    snprintf(g_mx_msg, sizeof g_mx_msg, fmt, a, b);
    if (err_msg) *err_msg = g_mx_msg;
    return code;
}
int mx_done(const char **err_msg, const char *what, cudaError_t e) {
    if (e == cudaSuccess) return RWKV7_OK;
    snprintf(g_mx_msg, sizeof g_mx_msg, "%s: %s", what, cudaGetErrorString(e));
    if (err_msg) *err_msg = g_mx_msg;
    return RWKV7_ECUDA;
}
bool mx_size_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 1 && rows <= RWKV7_MX_MAX_DIM && cols <= RWKV7_MX_MAX_DIM;
}

// Rows in memory: `rows` of `width` bytes, `step` bytes apart (contiguous: one row).
struct MxSpan {
    uintptr_t at;
    uint64_t rows, width, step;
    MxSpan(const void *p, int64_t r, int64_t cols, int64_t ld, int size)
        : at((uintptr_t)p), rows((uint64_t)r), width((uint64_t)(cols * size)), step((uint64_t)ld * (uint64_t)size) {
        if (rows > 1 && step == width) width *= rows, rows = 1;
    }
    uintptr_t end() const { return at + (rows - 1) * step * (rows > 1) + width; }
};
MxSpan mx_matrix_span(const void *mx, int64_t rows, int64_t cols) {
    return MxSpan(mx, 1, (int64_t)rwkv7_mx4_bytes(rows, cols), 0, 1);
}
// Whether two of them, with rows, share a byte.  Certain where one is contiguous or both
// have the same step; otherwise true where their ends overlap.
bool mx_share(const MxSpan &a, const MxSpan &b) {
    if (a.end() <= b.at || b.end() <= a.at) return false;
    if (a.rows > 1 && b.rows > 1) {
        if (a.step != b.step) return true;
        const uint64_t gap = b.at >= a.at ? (b.at - a.at) % a.step : (a.step - (a.at - b.at) % a.step) % a.step;
        return gap < a.width || gap + b.width > a.step;  // b's columns against a's, and against a's next row
    }
    if (a.rows == 1 && b.rows == 1) return true;
    const MxSpan &r = a.rows > 1 ? a : b, &c = a.rows > 1 ? b : a;
    const uint64_t i = c.at < r.at + r.width ? 0 : (c.at - r.at - r.width) / r.step + 1;  // r's first row that ends past c.at
    return i < r.rows && r.at + i * r.step < c.end();
}

int mx_rows_check(MxRowsParams &p, const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, const void *mx,
                  const char **err_msg) {
    if (err_msg) *err_msg = "";
    if (!mx_size_ok(rows, cols))
        return mx_fail(err_msg, RWKV7_EINVAL, "rows must be >= 0 and cols >= 1, both at most 2^24 (rows=%lld, cols=%lld)",
                       rows, cols);
    if (dtype < RWKV7_F32 || dtype > RWKV7_BF16) return mx_fail(err_msg, RWKV7_EINVAL, "unknown dtype %lld", dtype);
    if (rows > 1 && ld < cols) return mx_fail(err_msg, RWKV7_EINVAL, "row stride %lld is below cols=%lld", ld, cols);
    if (rows > 0 && (!x || !mx)) return mx_fail(err_msg, RWKV7_EINVAL, "null pointer argument");
    const int size = dtype == RWKV7_F32 ? 4 : 2;
    if ((uintptr_t)x % size) return mx_fail(err_msg, RWKV7_EINVAL, "the rows' pointer is not aligned to its type");
    if ((uintptr_t)mx & 15u) return mx_fail(err_msg, RWKV7_EINVAL, "the MXFP4 matrix must be 16-byte aligned");
    p.x = const_cast<void *>(x);
    p.cols = cols;
    p.ld = ld;
    p.mx = static_cast<uint8_t *>(const_cast<void *>(mx));
    p.kt = (int)((cols + MX_TILE_K - 1) / MX_TILE_K);
    if (rows > (INT32_MAX - 4096) / p.kt)
        return mx_fail(err_msg, RWKV7_EINVAL, "%lld rows of %lld columns are too many", rows, cols);
    if (rows > 0 && mx_share(MxSpan(x, rows, cols, ld, size), mx_matrix_span(mx, rows, cols)))
        return mx_fail(err_msg, RWKV7_EINVAL, "the rows and the MXFP4 matrix overlap");
    p.rows = (int)rows;
    const int step = 8 * size;  // bytes of a lane's eight values
    p.vec = (uintptr_t)x % step == 0 && (rows <= 1 || ld * size % step == 0);
    p.per = rows * p.kt >= MXQ_MANY ? MXQ_LINES : 1;
    p.groups = (int)((rows + p.per - 1) / p.per * p.kt);
    return RWKV7_OK;
}

cudaError_t mx_launch_rows(const void *kernel, MxRowsParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.groups + MXQ_THREADS / 32 - 1) / (MXQ_THREADS / 32)));
    cfg.blockDim = dim3(MXQ_THREADS);
    cfg.stream = stream;
    void *args[] = {&p};
    return cudaLaunchKernelExC(&cfg, kernel, args);
}
const void *mx_quantize_fn(int dtype) {
    return dtype == MX_F32   ? (const void *)mx4_quantize_kernel<MX_F32>
           : dtype == MX_F16 ? (const void *)mx4_quantize_kernel<MX_F16>
                             : (const void *)mx4_quantize_kernel<MX_BF16>;
}
const void *mx_dequantize_fn(int dtype) {
    return dtype == MX_F32   ? (const void *)mx4_dequantize_kernel<MX_F32>
           : dtype == MX_F16 ? (const void *)mx4_dequantize_kernel<MX_F16>
                             : (const void *)mx4_dequantize_kernel<MX_BF16>;
}

int mx_states(bool save, MxStateParams &p, int32_t n, int32_t format, void *stream, const char **err_msg) {
    if (err_msg) *err_msg = "";
    if (p.L < 1 || p.H < 1 || p.n_slots < 1 || p.n_entries < 1 || p.H > RWKV7_MX_MAX_DIM / p.L)
        return mx_fail(err_msg, RWKV7_EINVAL, "layers, heads, slots and entries must be >= 1");
    if (n < 0 || n > RWKV7_STATES_MAX_PAIRS)
        return mx_fail(err_msg, RWKV7_EINVAL, "n=%lld is outside 0 .. %lld pairs a call", n, RWKV7_STATES_MAX_PAIRS);
    if (format != RWKV7_MXFP4 && format != RWKV7_MXINT8)
        return mx_fail(err_msg, RWKV7_EINVAL, "unknown format %lld", format);
    if (n == 0) return RWKV7_OK;
    if (!p.wkv || !p.att || !p.ffn || !p.slots || !p.entries || !p.cache || !p.err)
        return mx_fail(err_msg, RWKV7_EINVAL, "null pointer argument");
    if (((uintptr_t)p.wkv & 31u) || (((uintptr_t)p.att | (uintptr_t)p.ffn | (uintptr_t)p.cache) & 15u))
        return mx_fail(err_msg, RWKV7_EINVAL,
                       "wkv must be 32-byte aligned, the shift states and the cache 16-byte aligned");
    p.entry_bytes = (int64_t)rwkv7_state_entry_bytes(p.L, p.H, format);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.L * p.H), (unsigned)n);
    cfg.blockDim = dim3(MXS_THREADS);
    cfg.stream = static_cast<cudaStream_t>(stream);
    const void *fn = format == RWKV7_MXINT8
                         ? (save ? (const void *)mx_state_kernel<MXINT8, true>
                                 : (const void *)mx_state_kernel<MXINT8, false>)
                         : (save ? (const void *)mx_state_kernel<MXFP4, true>
                                 : (const void *)mx_state_kernel<MXFP4, false>);
    void *args[] = {&p};
    return mx_done(err_msg, save ? "saving states" : "loading states", cudaLaunchKernelExC(&cfg, fn, args));
}

}  // namespace

int rk::mx_ctx_states(bool save, const MxCtxStates &c, const char **err_msg) {
    MxStateParams p;
    memset(&p, 0, sizeof p);
    p.wkv = c.wkv, p.att = c.att, p.ffn = c.ffn;
    p.L = c.L, p.H = c.H, p.n_slots = c.n_slots, p.n_entries = c.n_entries;
    p.slots = c.slots, p.entries = c.entries;
    p.cache = c.cache, p.err = c.err;
    p.occ = c.occ, p.ndraw = c.ndraw, p.V = c.V;
    return mx_states(save, p, c.n, c.format, c.stream, err_msg);
}

extern "C" {

size_t rwkv7_mx4_bytes(int64_t rows, int64_t cols) {
    if (!mx_size_ok(rows, cols)) return 0;
    return (size_t)((rows + MX_TILE_M - 1) / MX_TILE_M) * (size_t)((cols + MX_TILE_K - 1) / MX_TILE_K) * MX_TILE_BYTES;
}

int rwkv7_mx4_quantize(const void *d_x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, void *d_mx,
                       void *cuda_stream, const char **err_msg) {
    MxRowsParams p;
    int rc = mx_rows_check(p, d_x, dtype, rows, cols, ld, d_mx, err_msg);
    if (rc || rows == 0) return rc;
    return mx_done(err_msg, "quantising",
                   mx_launch_rows(mx_quantize_fn(dtype), p, static_cast<cudaStream_t>(cuda_stream)));
}

int rwkv7_mx4_dequantize(const void *d_mx, int64_t rows, int64_t cols, void *d_y, int32_t dtype, int64_t ld,
                         void *cuda_stream, const char **err_msg) {
    MxRowsParams p;
    int rc = mx_rows_check(p, d_y, dtype, rows, cols, ld, d_mx, err_msg);
    if (rc || rows == 0) return rc;
    return mx_done(err_msg, "reading back",
                   mx_launch_rows(mx_dequantize_fn(dtype), p, static_cast<cudaStream_t>(cuda_stream)));
}

int rwkv7_mx4_linear(const void *d_x, int32_t x_dtype, int64_t ldx, void *d_x_mx, int64_t B, const void *d_w_mx, int64_t N,
                     int64_t K, void *d_y, int32_t y_dtype, int64_t ldy, int32_t activation, uint32_t *d_err,
                     void *cuda_stream, const char **err_msg) {
    if (err_msg) *err_msg = "";
    if (!mx_size_ok(B, K) || !mx_size_ok(N, K) || N < 1)
        return mx_fail(err_msg, RWKV7_EINVAL, "B must be >= 0, N and K >= 1, all at most 2^24 (N=%lld, K=%lld)", N, K);
    if (y_dtype < RWKV7_F32 || y_dtype > RWKV7_BF16)
        return mx_fail(err_msg, RWKV7_EINVAL, "unknown output dtype %lld", y_dtype);
    if (activation != RWKV7_ACT_NONE && activation != RWKV7_ACT_RELU2)
        return mx_fail(err_msg, RWKV7_EINVAL, "unknown activation %lld", activation);
    if (B > 1 && ldy < N) return mx_fail(err_msg, RWKV7_EINVAL, "output row stride %lld is below N=%lld", ldy, N);
    if (B > ((int64_t)1 << 42) / N)
        return mx_fail(err_msg, RWKV7_EINVAL, "an output of %lld x %lld is too large", B, N);
    if (B == 0) return RWKV7_OK;
    if (!d_x_mx || !d_w_mx || !d_y || !d_err) return mx_fail(err_msg, RWKV7_EINVAL, "null pointer argument");
    if ((uintptr_t)d_y % (y_dtype == RWKV7_F32 ? 4 : 2))
        return mx_fail(err_msg, RWKV7_EINVAL, "the output pointer is not aligned to its type");
    if (((uintptr_t)d_x_mx | (uintptr_t)d_w_mx) & 15u)
        return mx_fail(err_msg, RWKV7_EINVAL, "MXFP4 matrices must be 16-byte aligned");
    const MxSpan y(d_y, B, N, ldy, y_dtype == RWKV7_F32 ? 4 : 2);
    const MxSpan x_mx = mx_matrix_span(d_x_mx, B, K), w_mx = mx_matrix_span(d_w_mx, N, K);
    MxLinearParams p;
    memset(&p, 0, sizeof p);
    struct Rows {
        MxRowsParams q;
        int type;
        cudaStream_t stream;
    } rows;
    if (d_x) {
        int rc = mx_rows_check(rows.q, d_x, x_dtype, B, K, ldx, d_x_mx, err_msg);
        if (rc) return rc;
        rows.type = x_dtype;
        rows.stream = static_cast<cudaStream_t>(cuda_stream);
        p.rows = d_x, p.rtype = x_dtype, p.rvec = rows.q.vec, p.ldr = ldx;
        p.over = mx_share(MxSpan(d_x, B, K, ldx, x_dtype == RWKV7_F32 ? 4 : 2), y);
        if (mx_share(x_mx, w_mx)) return mx_fail(err_msg, RWKV7_EINVAL, "the room for x overlaps w");
    }
    if (mx_share(y, x_mx) || mx_share(y, w_mx))
        return mx_fail(err_msg, RWKV7_EINVAL, "the output overlaps an MXFP4 matrix of the product");
    p.x = static_cast<const uint8_t *>(d_x_mx);
    p.w = static_cast<const uint8_t *>(d_w_mx);
    p.y = d_y;
    p.ldy = ldy;
    p.B = (int)B, p.N = (int)N, p.K = (int)K;
    p.act = activation;
    p.err = d_err;
    cudaError_t e = cudaSuccess;
    launch_mx_linear(
        p, y_dtype, static_cast<cudaStream_t>(cuda_stream),
        [](void *r) {
            Rows &s = *static_cast<Rows *>(r);
            return mx_launch_rows(mx_quantize_fn(s.type), s.q, s.stream);
        },
        &rows, &e);
    return mx_done(err_msg, "MXFP4 product", e);
}

size_t rwkv7_state_entry_bytes(int32_t n_layer, int32_t n_head, int32_t format) {
    if (n_layer < 1 || n_head < 1 || n_head > RWKV7_MX_MAX_DIM / n_layer) return 0;
    if (format != RWKV7_MXFP4 && format != RWKV7_MXINT8) return 0;
    const int64_t heads = (int64_t)n_layer * n_head;
    return (size_t)(mx_codes(heads, format) + heads * (MX_HEAD / MX_BLOCK) + heads * 2 * HS * 4);
}

int rwkv7_states_save(const float *d_wkv, const float *d_shift_att, const float *d_shift_ffn, int32_t n_layer,
                      int32_t n_head, int32_t n_slots, const int32_t *d_slots, const int32_t *d_entries, int32_t n,
                      void *d_cache, int32_t n_entries, int32_t format, uint32_t *d_err, void *cuda_stream,
                      const char **err_msg) {
    MxStateParams p;
    memset(&p, 0, sizeof p);
    p.wkv = const_cast<float *>(d_wkv);
    p.att = const_cast<float *>(d_shift_att), p.ffn = const_cast<float *>(d_shift_ffn);
    p.L = n_layer, p.H = n_head, p.n_slots = n_slots, p.n_entries = n_entries;
    p.slots = d_slots, p.entries = d_entries;
    p.cache = static_cast<uint8_t *>(d_cache), p.err = d_err;
    return mx_states(true, p, n, format, cuda_stream, err_msg);
}

int rwkv7_states_load(float *d_wkv, float *d_shift_att, float *d_shift_ffn, int32_t n_layer, int32_t n_head,
                      int32_t n_slots, const int32_t *d_slots, const int32_t *d_entries, int32_t n, const void *d_cache,
                      int32_t n_entries, int32_t format, uint32_t *d_err, void *cuda_stream, const char **err_msg) {
    MxStateParams p;
    memset(&p, 0, sizeof p);
    p.wkv = d_wkv, p.att = d_shift_att, p.ffn = d_shift_ffn;
    p.L = n_layer, p.H = n_head, p.n_slots = n_slots, p.n_entries = n_entries;
    p.slots = d_slots, p.entries = d_entries;
    p.cache = static_cast<uint8_t *>(const_cast<void *>(d_cache)), p.err = d_err;
    return mx_states(false, p, n, format, cuda_stream, err_msg);
}

}  // extern "C"
