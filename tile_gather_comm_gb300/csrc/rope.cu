// rope.cu -- tgc_rope, tgc_rope_bwd, tgc_rope_freqs and tgc_kv_append: rotary positions of query and
// key heads, and the new tokens' keys and values on their way into the pages of a cache.
//
//   (a, b) -> s (a cos w - b sin w), s (b cos w + a sin w),  w = pos freq     (backward: -w)
//
// A pair is read, turned and written by one thread, so a call may write over its own input.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "act.cuh"
#include "internal.h"
#include "kv.cuh"
#include "prims.cuh"

namespace tgc {

// i / d for i * d < 2^32: one multiplication by ceil(2^32 / d), whose excess adds less than 1 / d to the quotient.
struct Divisor {
    uint32_t d, m;
    __device__ __forceinline__ int of(int i) const { return d == 1 ? i : (int)__umulhi((uint32_t)i, m); }
};
static Divisor divisor(int d) { return Divisor{(uint32_t)d, (uint32_t)(((uint64_t(1) << 32) + d - 1) / d)}; }

struct RopeParams {
    // 0 queries, 1 keys, 2 values (never turned; only with a cache)
    const void *in[3];
    void *out[3];
    int64_t in_t[3], in_h[3], out_t[3], out_h[3];
    int heads[3];
    const int32_t *pos;
    const double *freqs;
    int T, D, R;
    float scale, sign;
    // the cache that keys and values go to; none: keys go to out[1]
    bool cached;
    KvTable kv;
    const int32_t *table, *seqs;
    int64_t page_s, token_s;
    int tokens, rows;                 // of a block
    Divisor half, units, block_rows;  // pairs of a token, units of a row, rows of a block
};

// V elements as they lie in memory, read and written as two values at a time: kept as 16-bit elements they would take a
// register each and be put together again for every store.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    uint32_t w[V * sizeof(T) / 4];
    __device__ __forceinline__ F2 get(int i) const {
        if constexpr (sizeof(T) == 4) return f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return unpack16(w[i], std::is_same<T, __half>::value);
    }
    __device__ __forceinline__ void put(int i, F2 v) {
        if constexpr (sizeof(T) == 4) {
            const float2 f = split(v);
            w[2 * i] = __float_as_uint(f.x);
            w[2 * i + 1] = __float_as_uint(f.y);
        } else {
            w[i] = pack16(v, std::is_same<T, __half>::value);
        }
    }
    // one of the first two elements
    __device__ __forceinline__ void set(int i, T t) { reinterpret_cast<T *>(w)[i] = t; }
    __device__ __forceinline__ T at(int i) const { return reinterpret_cast<const T *>(w)[i]; }
};
template <typename T>
struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ void set(int, T t) { v = t; }
    __device__ __forceinline__ T at(int) const { return v; }
};

// A pair side by side, turned.
__device__ __forceinline__ F2 turned(F2 v, float c, float s) {
    const float2 f = split(v);
    return fma(f2(f.y, f.x), f2(-s, s), mul(v, every<F2>(c)));
}

// freq / 2 pi modulo a whole turn, in 2^-64 turns (signed: a negative one wraps).  1 / 2 pi in two terms, the rounding
// of the first one's product added to the second's: off by about 2^-106 of itself before it is rounded to 2^-64,
// where one product of doubles would be off by 2^-53, 2^-25 turns at 2^31 positions a radian apart.
__device__ __forceinline__ uint64_t turn_fraction(double freq) {
    constexpr double kHigh = 0x1.45f306dc9c883p+61, kLow = -0x1.6b01ec5417056p+7;  // their sum: 2^64 / (2 pi)
    constexpr double kTurn = 0x1p64;
    double high = __dmul_rn(freq, kHigh), low = __fma_rn(freq, kLow, __fma_rn(freq, kHigh, -high));
    if (fabs(high) >= kTurn / 2) {  // half a turn a position, or more
        high -= kTurn * rint(high / kTurn);
        low -= kTurn * rint(low / kTurn);
        if (high == kTurn / 2) high = -high;
    }
    return (uint64_t)__double2ll_rn(high) + (uint64_t)__double2ll_rn(low);
}

// One block: `tokens` tokens, `rows` of their heads.  First the sines and cosines of its tokens (one for each token
// and pair, which the heads share), then the heads, a thread taking units of V pairs (half layout: a vector of V from
// each half; interleaved: one vector of V / 2 pairs) or a vector of V elements to copy.
//
// The angle: freq / 2 pi, taken modulo 1, is held as a 64-bit fraction of a turn (turn_fraction), and its product with
// the position modulo 2^64 is the angle's: whole turns fall off the top.  The fraction is off by one 2^-64 at most, so
// the angle by 2^-33 turns at the farthest position; it is rounded to fp32 relative to itself (2^-23 of it), so that a
// small one keeps its bits, and sine and cosine are taken in fp32.  fp64 is needed once a pair and block.
//
// Bound by HBM where there are many tokens, by the launch where there are few.
constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;   // of a block at most
constexpr int kRopeRows = 1024;  // rows of a block at most: with 1024 units a row, i * d stays below 2^32 (Divisor)

// How a unit's elements lie: two vectors R/2 apart, of V pairs (half layout) or of V / 2 pairs each (interleaved); the
// same with an odd R/2, where the second vector is not aligned and goes element by element (and the last unit
// has one pair); one vector of V / 2 pairs; one pair of single elements.
enum RopeForm { kHalf, kHalfOdd, kHalfOne, kNear, kNearSingle, kNearOne };

// Units of a row that turn; those behind them copy V elements each.
__host__ __device__ inline int rope_turning(RopeForm form, int v, int R) {
    return form == kHalfOdd ? (R / 2 + 1) / 2 : form == kNearSingle ? R / v : R / 2 / v;
}

// Registers: 32 a thread, so that an SM holds 64 warps: with units taken several at a time in more registers fewer loads
// were under way in all (8192 tokens of 40 heads of 128 bf16: 29.7 us; 2 units 33 to 37, 4 units 33 to 73).
template <typename T, int V, RopeForm FORM>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const RopeParams p) {
    constexpr bool INTERLEAVED = FORM == kNear || FORM == kNearSingle || FORM == kNearOne;
    constexpr bool PAIR = FORM != kNearSingle;  // a unit that turns is two vectors
    constexpr int kTwos = V > 1 ? V / 2 : 1;
    using W = Vec<T, V>;
    extern __shared__ uint64_t s_freq[];                          // R/2
    float *s_cos = reinterpret_cast<float *>(s_freq + p.R / 2), *s_sin = s_cos + p.tokens * (p.R / 2);  // tokens x R/2, times scale
    __shared__ int64_t s_slot[kRopeTokens];
    __shared__ int s_pos[kRopeTokens];
    stream_wait();
    stream_release();
    const int tid = (int)threadIdx.x, half = p.R / 2;
    const int t0 = (int)blockIdx.x * p.tokens, tokens = p.T - t0 < p.tokens ? p.T - t0 : p.tokens;
    const int all_rows = p.heads[0] + p.heads[1] + p.heads[2];
    const int row0 = (int)blockIdx.y * p.rows, rows = all_rows - row0 < p.rows ? all_rows - row0 : p.rows;
    const int turning = rope_turning(FORM, V, p.R), units = (int)p.units.d;
    if (tid < tokens) {
        const int t = t0 + tid, pos = p.pos[t];
        int64_t slot = -1;
        if (p.cached && pos >= 0) {
            const int page = p.kv.page_at(p.table, p.seqs != nullptr ? p.seqs[t] : t, pos / p.kv.page_size);
            if (page >= 0) slot = page * p.page_s + pos % p.kv.page_size * p.token_s;
        }
        s_pos[tid] = pos;
        s_slot[tid] = slot;
    }
    for (int i = tid; i < half; i += kRopeThreads) s_freq[i] = turn_fraction(p.freqs[i]);
    __syncthreads();
    for (int i = tid; i < tokens * half; i += kRopeThreads) {
        const int t = p.half.of(i);
        const uint64_t angle = s_freq[i - t * half] * (uint64_t)(uint32_t)s_pos[t];
        float c, s;
        // its size in half turns: the halves one by one, as a conversion from 64 bits takes longer (8192 tokens of a head of 256
        // fp32: 7.65 and 7.47 us)
        const bool back = (int64_t)angle < 0;
        const uint64_t size = back ? 0 - angle : angle;
        const float half_turns = fmaf((float)(uint32_t)size, 0x1p-63f, (float)(uint32_t)(size >> 32) * 0x1p-31f);
        sincospif(back ? -half_turns : half_turns, &s, &c);
        s_cos[i] = c * p.scale;
        s_sin[i] = s * p.scale * p.sign;
    }
    __syncthreads();
    // the last block in y may have fewer rows than the divisor is for
    const Divisor by_rows = rows == (int)p.block_rows.d ? p.block_rows : Divisor{(uint32_t)rows, 0xffffffffu / (uint32_t)rows + 1u};
    const int n = tokens * rows * units;
    for (int i = tid; i < n; i += kRopeThreads) {
        const int r = p.units.of(i), unit = i - r * units, t = by_rows.of(r), row = r - t * rows + row0;
        const int set = row < p.heads[0] ? 0 : row < p.heads[0] + p.heads[1] ? 1 : 2;
        const int head = row - (set == 0 ? 0 : set == 1 ? p.heads[0] : p.heads[0] + p.heads[1]);
        if (s_pos[t] < 0) continue;
        const T *in = static_cast<const T *>(p.in[set]) + (t0 + t) * p.in_t[set] + head * p.in_h[set];
        T *out = static_cast<T *>(p.out[set]) + head * p.out_h[set];
        if (set > 0 && p.cached) {
            if (s_slot[t] < 0) continue;
            out += s_slot[t];
        } else {
            out += (t0 + t) * p.out_t[set];
        }
        const bool turns = unit < turning;
        const int a = !turns ? p.R + (unit - turning) * V : FORM == kNearOne ? 2 * unit : unit * V;
        const int b = a + (FORM == kNearOne ? 1 : half);  // the other vector of a unit that turns
        const bool both = FORM != kHalfOdd || !turns || a + 1 < half;  // not one pair alone
        W x, y;
        if (both) x = *reinterpret_cast<const W *>(in + a);
        else x.set(0, in[a]);
        if (PAIR && turns) {
            if constexpr (FORM == kHalfOdd) {
                y.set(0, in[b]);
                if (both) y.set(1, in[b + 1]);
            } else {
                y = *reinterpret_cast<const W *>(in + b);
            }
        }
        if (turns && set < 2) {
            const float *c = s_cos + t * half, *s = s_sin + t * half;
            if constexpr (V == 1) {
                const float va = to_f32(x.v), vb = to_f32(y.v);
                x.v = from_f32<T>(va * c[unit] - vb * s[unit]);
                y.v = from_f32<T>(vb * c[unit] + va * s[unit]);
            } else {
#pragma unroll
                for (int j = 0; j < kTwos; ++j) {
                    if constexpr (!INTERLEAVED) {  // two pairs
                        const F2 va = x.get(j), vb = y.get(j);
                        const int at = unit * V + 2 * j;
                        const F2 cc = f2(c[at], c[both ? at + 1 : at]), ss = f2(s[at], s[both ? at + 1 : at]);
                        x.put(j, fma(vb, mul(ss, every<F2>(-1.0f)), mul(va, cc)));
                        y.put(j, fma(va, ss, mul(vb, cc)));
                    } else {  // one in each vector
                        const int at = unit * kTwos + j;
                        x.put(j, turned(x.get(j), c[at], s[at]));
                        if constexpr (PAIR) y.put(j, turned(y.get(j), c[at + half / 2], s[at + half / 2]));
                    }
                }
            }
        }
        if (both) *reinterpret_cast<W *>(out + a) = x;
        else out[a] = x.at(0);
        if (PAIR && turns) {
            if constexpr (FORM == kHalfOdd) {
                out[b] = y.at(0);
                if (both) out[b + 1] = y.at(1);
            } else {
                *reinterpret_cast<W *>(out + b) = y;
            }
        }
    }
}

static int elem_bytes(tgc_dtype t) { return t == TGC_F32 ? 4 : t == TGC_BF16 || t == TGC_F16 ? 2 : 0; }

struct RopeShape {
    RopeForm form;
    int v;  // elements of a vector
};

// The widest vectors that pointers, strides and the parts of a head all keep: 16 bytes, two elements, one.
static RopeShape rope_shape(const RopeParams &p, bool interleaved, int es, const void *k_pages, const void *v_pages, int64_t head_s) {
    for (const int v : {16 / es, 2}) {
        bool fits = p.D % v == 0 && p.R % v == 0;
        auto at = [&](const void *q, int64_t a, int64_t b) {
            fits = fits && reinterpret_cast<uintptr_t>(q) % (v * es) == 0 && a % v == 0 && b % v == 0;
        };
        for (int i = 0; i < 3; ++i)
            if (p.heads[i] > 0) {
                at(p.in[i], p.in_t[i], p.in_h[i]);
                if (!p.cached || i == 0) at(p.out[i], p.out_t[i], p.out_h[i]);
            }
        if (p.cached) {
            at(k_pages, p.page_s, p.token_s);
            at(v_pages, head_s, 0);
        }
        if (!fits) continue;
        if (p.R / 2 % v == 0 && (v > 2 || !interleaved)) return {interleaved ? kNear : kHalf, v};
        if (v == 2) return {interleaved ? kNearSingle : kHalfOdd, 2};
    }
    return {interleaved ? kNearOne : kHalfOne, 1};
}

template <typename T>
static cudaError_t launch_rope_typed(const RopeParams &p, RopeShape f, dim3 grid, size_t smem, cudaStream_t stream) {
    constexpr int W = 16 / sizeof(T);
    auto go = [&](auto kernel) { return launch_overlapped(kernel, grid, dim3(kRopeThreads), smem, 1, stream, p); };
    switch (f.form) {
        case kHalf: return f.v == W ? go(rope_kernel<T, W, kHalf>) : go(rope_kernel<T, 2, kHalf>);
        case kHalfOdd: return go(rope_kernel<T, 2, kHalfOdd>);
        case kHalfOne: return go(rope_kernel<T, 1, kHalfOne>);
        case kNear: return go(rope_kernel<T, W, kNear>);
        case kNearSingle: return go(rope_kernel<T, 2, kNearSingle>);
        default: return go(rope_kernel<T, 1, kNearOne>);
    }
}

static int launch_rope(RopeParams &p, RopeShape f, tgc_dtype dtype, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const int sms = sm_count(dev), rows = p.heads[0] + p.heads[1] + p.heads[2], half = p.R / 2;
    const int units = rope_turning(f.form, f.v, p.R) + (p.D - p.R) / f.v;
    // Many tokens: up to 4 a block, so that its threads each have a sine to take.  Few: one a block, its rows cut
    // so that a thread has one unit.
    p.tokens = 1;
    while (p.tokens < kRopeTokens && p.T / (2 * p.tokens) >= 8 * sms) p.tokens *= 2;
    p.rows = rows < kRopeRows ? rows : kRopeRows;
    if (p.T < 4 * sms) p.rows = std::min(p.rows, (kRopeThreads + units - 1) / units);
    p.rows = std::max(p.rows, (rows + 65534) / 65535);  // a grid has 65535 blocks in y at most
    p.half = divisor(half > 0 ? half : 1);
    p.units = divisor(units);
    p.block_rows = divisor(p.rows);
    const dim3 grid((unsigned)((p.T + p.tokens - 1) / p.tokens), (unsigned)((rows + p.rows - 1) / p.rows));
    const size_t smem = (size_t)(p.tokens + 1) * (size_t)half * sizeof(float2);
    e = dtype == TGC_BF16  ? launch_rope_typed<__nv_bfloat16>(p, f, grid, smem, stream)
        : dtype == TGC_F16 ? launch_rope_typed<__half>(p, f, grid, smem, stream)
                           : launch_rope_typed<float>(p, f, grid, smem, stream);
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
}

#define TGC_TRY(expr)                     \
    do {                                  \
        const int rc_ = (expr);           \
        if (rc_ != TGC_OK) return rc_;    \
    } while (0)

// Sizes and the rotation that the calls of this file share.
static int rope_check(int64_t T, int64_t Hq, int64_t Hk, int64_t Hv, int64_t D, int64_t R, bool turn, float *scale,
                      int layout, int es) {
    if (es == 0) return TGC_ERR_DTYPE;
    if (T < 0 || T > TGC_MAX_SIZE || Hq < 0 || Hk < 0 || Hq > TGC_ROPE_MAX_HEADS || Hk > TGC_ROPE_MAX_HEADS ||
        Hq + Hk < 1 || Hq + Hk + Hv > TGC_ROPE_MAX_HEADS)
        return TGC_ERR_INVALID_ARG;
    if (D < 1 || D > TGC_ROPE_MAX_D || R > D || R % 2 != 0 || (turn ? R < 2 : R != 0)) return TGC_ERR_INVALID_ARG;
    if (layout != TGC_ROPE_HALF && layout != TGC_ROPE_INTERLEAVED) return TGC_ERR_INVALID_ARG;
    if (!std::isfinite(*scale)) return TGC_ERR_INVALID_ARG;
    if (*scale == 0.0f) *scale = 1.0f;
    return TGC_OK;
}

// An operand of heads that the call needs where it has any.
static int heads_given(const void *p, int64_t T, int64_t H, int64_t D, int es, int64_t *st, int64_t *sh) {
    TGC_TRY(heads_check(T, H, D, st, sh));
    if (H == 0 || T == 0) return TGC_OK;
    if (p == nullptr) return TGC_ERR_INVALID_ARG;
    return reinterpret_cast<uintptr_t>(p) % es == 0 ? TGC_OK : TGC_ERR_ALIGN;
}

static bool misaligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// In place only with the layout that it was read in: a thread then writes what it alone has read.
static bool bad_in_place(const void *in, const void *out, int64_t it, int64_t ih, int64_t ot, int64_t oh, int64_t T,
                         int64_t H) {
    return in == out && in != nullptr && ((T > 1 && it != ot) || (H > 1 && ih != oh));
}

static int rope_impl(tgc_rope_args a, float sign) {
    const int es = elem_bytes(a.dtype);
    TGC_TRY(rope_check(a.T, a.heads_q, a.heads_k, 0, a.D, a.R, true, &a.scale, a.layout, es));
    if (a.T == 0) return TGC_OK;
    if (a.pos == nullptr || a.freqs == nullptr) return TGC_ERR_INVALID_ARG;
    TGC_TRY(heads_given(a.q, a.T, a.heads_q, a.D, es, &a.q_t, &a.q_h));
    TGC_TRY(heads_given(a.q_out, a.T, a.heads_q, a.D, es, &a.qo_t, &a.qo_h));
    TGC_TRY(heads_given(a.k, a.T, a.heads_k, a.D, es, &a.k_t, &a.k_h));
    TGC_TRY(heads_given(a.k_out, a.T, a.heads_k, a.D, es, &a.ko_t, &a.ko_h));
    if (bad_in_place(a.q, a.q_out, a.q_t, a.q_h, a.qo_t, a.qo_h, a.T, a.heads_q) ||
        bad_in_place(a.k, a.k_out, a.k_t, a.k_h, a.ko_t, a.ko_h, a.T, a.heads_k))
        return TGC_ERR_INVALID_ARG;
    if (misaligned(a.pos, 4) || misaligned(a.freqs, 8)) return TGC_ERR_ALIGN;
    RopeParams p{};
    p.in[0] = a.q; p.in[1] = a.k;
    p.out[0] = a.q_out; p.out[1] = a.k_out;
    p.in_t[0] = a.q_t; p.in_t[1] = a.k_t; p.in_h[0] = a.q_h; p.in_h[1] = a.k_h;
    p.out_t[0] = a.qo_t; p.out_t[1] = a.ko_t; p.out_h[0] = a.qo_h; p.out_h[1] = a.ko_h;
    p.heads[0] = (int)a.heads_q; p.heads[1] = (int)a.heads_k;
    p.pos = a.pos; p.freqs = a.freqs;
    p.T = (int)a.T; p.D = (int)a.D; p.R = (int)a.R;
    p.scale = a.scale; p.sign = sign;
    const bool interleaved = a.layout == TGC_ROPE_INTERLEAVED;
    return launch_rope(p, rope_shape(p, interleaved, es, nullptr, nullptr, 0), a.dtype, a.stream);
}

static int append_impl(tgc_kv_append_args a) {
    const int es = elem_bytes(a.dtype);
    if (a.heads_k < 1) return TGC_ERR_INVALID_ARG;
    TGC_TRY(rope_check(a.T, a.heads_q, a.heads_k, a.heads_k, a.D, a.R, a.freqs != nullptr, &a.scale, a.layout, es));
    TGC_TRY(kv_table_check(a.num_pages, a.page_size, a.num_seqs, a.max_pages, &a.table_ld));
    if (a.seqs == nullptr && a.T > a.num_seqs) return TGC_ERR_INVALID_ARG;
    TGC_TRY(kv_pages_check(a.num_pages, a.page_size, a.heads_k, a.D, &a.page_s, &a.token_s, &a.head_s));
    if (a.T == 0) return TGC_OK;
    if (a.pos == nullptr || a.k == nullptr || a.v == nullptr) return TGC_ERR_INVALID_ARG;
    // no place for a key without any of these: then the queries alone are turned
    if (a.num_seqs > 0 && a.max_pages > 0) {
        if (a.table == nullptr || (a.num_pages > 0 && (a.k_pages == nullptr || a.v_pages == nullptr))) return TGC_ERR_INVALID_ARG;
    }
    TGC_TRY(heads_given(a.q, a.T, a.heads_q, a.D, es, &a.q_t, &a.q_h));
    TGC_TRY(heads_given(a.q_out, a.T, a.heads_q, a.D, es, &a.qo_t, &a.qo_h));
    TGC_TRY(heads_given(a.k, a.T, a.heads_k, a.D, es, &a.k_t, &a.k_h));
    TGC_TRY(heads_given(a.v, a.T, a.heads_k, a.D, es, &a.v_t, &a.v_h));
    if (bad_in_place(a.q, a.q_out, a.q_t, a.q_h, a.qo_t, a.qo_h, a.T, a.heads_q)) return TGC_ERR_INVALID_ARG;
    if (misaligned(a.pos, 4) || misaligned(a.freqs, 8) || misaligned(a.table, 4) || misaligned(a.seqs, 4) ||
        misaligned(a.k_pages, es) || misaligned(a.v_pages, es))
        return TGC_ERR_ALIGN;
    RopeParams p{};
    p.in[0] = a.q; p.in[1] = a.k; p.in[2] = a.v;
    p.out[0] = a.q_out; p.out[1] = a.k_pages; p.out[2] = a.v_pages;
    p.in_t[0] = a.q_t; p.in_t[1] = a.k_t; p.in_t[2] = a.v_t;
    p.in_h[0] = a.q_h; p.in_h[1] = a.k_h; p.in_h[2] = a.v_h;
    p.out_t[0] = a.qo_t; p.out_h[0] = a.qo_h; p.out_h[1] = p.out_h[2] = a.head_s;
    p.heads[0] = (int)a.heads_q; p.heads[1] = p.heads[2] = (int)a.heads_k;
    p.pos = a.pos; p.freqs = a.freqs; p.cached = true; p.table = a.table; p.seqs = a.seqs;
    p.T = (int)a.T; p.D = (int)a.D; p.R = (int)a.R;
    p.scale = a.scale; p.sign = 1.0f;
    p.kv = KvTable{(int)a.num_pages, (int)a.page_size, (int)a.num_seqs, (int)a.max_pages, a.table_ld};
    p.page_s = a.page_s; p.token_s = a.token_s;
    const bool interleaved = a.layout == TGC_ROPE_INTERLEAVED;
    return launch_rope(p, rope_shape(p, interleaved, es, a.k_pages, a.v_pages, a.head_s), a.dtype, a.stream);
}

}  // namespace tgc

extern "C" int tgc_rope(const tgc_rope_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::rope_impl(*args, 1.0f);
}

extern "C" int tgc_rope_bwd(const tgc_rope_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::rope_impl(*args, -1.0f);
}

extern "C" int tgc_kv_append(const tgc_kv_append_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::append_impl(*args);
}

extern "C" int tgc_rope_freqs(double *freqs, double *scale, int64_t R, double base, tgc_rope_scaling scaling, double factor,
                              double trained, double beta_fast, double beta_slow) {
    if (freqs == nullptr || R < 2 || R > TGC_ROPE_MAX_D || R % 2 != 0) return TGC_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base) || scaling < TGC_ROPE_NONE || scaling > TGC_ROPE_YARN)
        return TGC_ERR_INVALID_ARG;
    if (scaling != TGC_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return TGC_ERR_INVALID_ARG;
    if (scaling == TGC_ROPE_YARN && (!(trained > 0.0) || !std::isfinite(trained) || !(beta_slow > 0.0) ||
                                     !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
        return TGC_ERR_INVALID_ARG;
    if (scaling == TGC_ROPE_NTK && R > 2) base *= std::pow(factor, (double)R / (double)(R - 2));
    if (!std::isfinite(base)) return TGC_ERR_INVALID_ARG;  // it would leave every pair but the first standing still
    for (int64_t i = 0; i < R / 2; ++i) {
        double f = std::pow(base, -2.0 * (double)i / (double)R);
        if (scaling == TGC_ROPE_LINEAR) f /= factor;
        if (scaling == TGC_ROPE_YARN) {
            const double turns = trained * f / 6.283185307179586477;  // 2 pi
            double keep = (turns - beta_slow) / (beta_fast - beta_slow);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = f * keep + f / factor * (1.0 - keep);
        }
        freqs[i] = f;
    }
    if (scale != nullptr) *scale = scaling == TGC_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return TGC_OK;
}
