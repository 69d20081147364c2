// rope.cu -- tgc_rope, tgc_rope_bwd, tgc_rope_freqs and tgc_kv_append: rotary positions of query and
// key heads, and the new tokens' keys and values on their way into the pages of a cache.
//
//   (a, b) -> s (a cos w - b sin w), s (b cos w + a sin w),  w = pos freq     (backward: -w)
//
// A pair is read, turned and written by one thread, so a call may write over its own input.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "act.cuh"
#include "internal.h"
#include "kv.cuh"
#include "prims.cuh"

namespace tgc {

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
    // the cache that keys and values go to; table == nullptr: none, keys go to out[1]
    KvTable kv;
    const int32_t *table, *seqs;
    int64_t page_s, token_s;
    int tokens, rows;  // of a block
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

// One block: `tokens` tokens, `rows` of their heads.  First the sines and cosines of its tokens (one
// for each token and pair, which the heads share), then the heads, a thread taking V pairs (half
// layout: a vector of V from each half; interleaved: one vector of V / 2 pairs) or a vector of V
// elements to copy at a time.
//
// The angle: pos * freq in fp64 (24 bits of position, 53 of frequency), taken modulo a turn by one
// subtraction, its sine and cosine in fp32.  A thread's share of fp64 is four instructions for a pair
// of a token; with 40 heads they are read 40 times from shared memory.
constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;  // of a block at most

template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    extern __shared__ float2 s_turn[];  // tokens x R/2: scale (cos, sin)
    __shared__ int64_t s_slot[kRopeTokens];
    __shared__ int s_pos[kRopeTokens];
    stream_wait();
    stream_release();
    const int t0 = (int)blockIdx.x * p.tokens, half = p.R / 2;
    const int tokens = p.T - t0 < p.tokens ? p.T - t0 : p.tokens;
    const int all_rows = p.heads[0] + p.heads[1] + p.heads[2];
    const int row0 = (int)blockIdx.y * p.rows, rows = all_rows - row0 < p.rows ? all_rows - row0 : p.rows;
    if ((int)threadIdx.x < tokens) {
        const int t = t0 + (int)threadIdx.x, pos = p.pos[t];
        int64_t slot = -1;
        if (p.table != nullptr && pos >= 0) {
            const int page = p.kv.page_at(p.table, p.seqs != nullptr ? p.seqs[t] : t, pos / p.kv.page_size);
            if (page >= 0) slot = page * p.page_s + pos % p.kv.page_size * p.token_s;
        }
        s_pos[threadIdx.x] = pos;
        s_slot[threadIdx.x] = slot;
    }
    for (int i = (int)threadIdx.x; i < tokens * half; i += kRopeThreads) {
        const int t = i / half;
        double turns = (double)p.pos[t0 + t] * p.freqs[i - t * half] * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= rint(turns);
        float c, s;
        sincospif(2.0f * (float)turns, &s, &c);
        s_turn[i] = make_float2(c * p.scale, s * p.scale * p.sign);
    }
    __syncthreads();
    // Units of a row: those that turn, then those that copy the rest of the head.
    const int turning = (INTERLEAVED && V > 1 ? p.R : half) / V;
    const int units = turning + (p.D - p.R) / V;
    const int n = tokens * rows * units;
    for (int i = (int)threadIdx.x; i < n; i += kRopeThreads) {
        const int unit = i % units, row = i / units % rows + row0, t = i / units / rows;
        const int set = row < p.heads[0] ? 0 : row < p.heads[0] + p.heads[1] ? 1 : 2;
        const int head = row - (set == 0 ? 0 : set == 1 ? p.heads[0] : p.heads[0] + p.heads[1]);
        if (s_pos[t] < 0) continue;
        const T *in = static_cast<const T *>(p.in[set]) + (t0 + t) * p.in_t[set] + head * p.in_h[set];
        T *out = static_cast<T *>(p.out[set]) + head * p.out_h[set];
        if (set > 0 && p.table != nullptr) {
            if (s_slot[t] < 0) continue;
            out += s_slot[t];
        } else {
            out += (t0 + t) * p.out_t[set];
        }
        using W = Vec<T, V>;
        if (unit >= turning) {
            const int e = p.R + (unit - turning) * V;
            *reinterpret_cast<W *>(out + e) = *reinterpret_cast<const W *>(in + e);
        } else if constexpr (INTERLEAVED && V > 1) {
            const int e = unit * V;
            W x = *reinterpret_cast<const W *>(in + e);
            if (set < 2) {
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const float2 w = s_turn[t * half + e / 2 + j];
                    const float a = to_f32(x.v[2 * j]), b = to_f32(x.v[2 * j + 1]);
                    x.v[2 * j] = from_f32<T>(a * w.x - b * w.y);
                    x.v[2 * j + 1] = from_f32<T>(b * w.x + a * w.y);
                }
            }
            *reinterpret_cast<W *>(out + e) = x;
        } else {
            const int ea = unit * V * (INTERLEAVED ? 2 : 1), eb = ea + (INTERLEAVED ? 1 : half);
            W x = *reinterpret_cast<const W *>(in + ea), y = *reinterpret_cast<const W *>(in + eb);
            if (set < 2) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 w = s_turn[t * half + unit * V + j];
                    const float a = to_f32(x.v[j]), b = to_f32(y.v[j]);
                    x.v[j] = from_f32<T>(a * w.x - b * w.y);
                    y.v[j] = from_f32<T>(b * w.x + a * w.y);
                }
            }
            *reinterpret_cast<W *>(out + ea) = x;
            *reinterpret_cast<W *>(out + eb) = y;
        }
    }
}

static int elem_bytes(tgc_dtype t) { return t == TGC_F32 ? 4 : t == TGC_BF16 || t == TGC_F16 ? 2 : 0; }

// The widest vector, in elements, that pointers, strides and the parts of a head all keep: 16 bytes, 2
// elements or 1.
static int rope_vector(const RopeParams &p, bool interleaved, int es, const void *k_pages, const void *v_pages,
                       int64_t head_s) {
    for (const int v : {16 / es, 2}) {
        bool fits = p.D % v == 0 && p.R % v == 0 && (interleaved || p.R / 2 % v == 0);
        auto at = [&](const void *q, int64_t a, int64_t b) {
            fits = fits && reinterpret_cast<uintptr_t>(q) % (v * es) == 0 && a % v == 0 && b % v == 0;
        };
        for (int i = 0; i < 3; ++i)
            if (p.heads[i] > 0) {
                at(p.in[i], p.in_t[i], p.in_h[i]);
                if (p.table == nullptr || i == 0) at(p.out[i], p.out_t[i], p.out_h[i]);
            }
        if (p.table != nullptr) {
            at(k_pages, p.page_s, p.token_s);
            at(v_pages, head_s, 0);
        }
        if (fits) return v;
    }
    return 1;
}

template <typename T, bool INTERLEAVED>
static cudaError_t launch_rope_typed(const RopeParams &p, int v, dim3 grid, size_t smem, cudaStream_t stream) {
    constexpr int W = 16 / sizeof(T);
    return v == W   ? launch_overlapped(rope_kernel<T, W, INTERLEAVED>, grid, dim3(kRopeThreads), smem, 1, stream, p)
           : v == 2 ? launch_overlapped(rope_kernel<T, 2, INTERLEAVED>, grid, dim3(kRopeThreads), smem, 1, stream, p)
                    : launch_overlapped(rope_kernel<T, 1, INTERLEAVED>, grid, dim3(kRopeThreads), smem, 1, stream, p);
}

static int launch_rope(RopeParams &p, bool interleaved, tgc_dtype dtype, int v, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const int sms = sm_count(dev), rows = p.heads[0] + p.heads[1] + p.heads[2];
    const int units = ((interleaved && v > 1 ? p.R : p.R / 2) + p.D - p.R) / v;
    // Many tokens: up to 4 a block, so that its threads each have a sine to take.  Few: one a block, its rows cut
    // so that a thread has one unit.
    p.tokens = 1;
    while (p.tokens < kRopeTokens && 2 * p.tokens * (p.R / 2) <= kRopeThreads && p.T / (2 * p.tokens) >= 8 * sms) p.tokens *= 2;
    p.rows = rows;
    if (p.T < 4 * sms) {
        p.rows = (kRopeThreads + units - 1) / units;
        if (p.rows > rows) p.rows = rows;
        if ((rows + p.rows - 1) / p.rows > 65535) p.rows = (rows + 65534) / 65535;
    }
    const dim3 grid((unsigned)((p.T + p.tokens - 1) / p.tokens), (unsigned)((rows + p.rows - 1) / p.rows));
    const size_t smem = (size_t)p.tokens * (size_t)(p.R / 2) * sizeof(float2);
    auto go = [&](auto type) {
        using T = decltype(type);
        return interleaved ? launch_rope_typed<T, true>(p, v, grid, smem, stream)
                           : launch_rope_typed<T, false>(p, v, grid, smem, stream);
    };
    e = dtype == TGC_BF16 ? go(__nv_bfloat16{}) : dtype == TGC_F16 ? go(__half{}) : go(0.0f);
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
    return launch_rope(p, interleaved, a.dtype, rope_vector(p, interleaved, es, nullptr, nullptr, 0), a.stream);
}

static int append_impl(tgc_kv_append_args a) {
    const int es = elem_bytes(a.dtype);
    if (a.heads_k < 1) return TGC_ERR_INVALID_ARG;
    TGC_TRY(rope_check(a.T, a.heads_q, a.heads_k, a.heads_k, a.D, a.R, a.freqs != nullptr, &a.scale, a.layout, es));
    TGC_TRY(kv_table_check(a.num_pages, a.page_size, a.num_seqs, a.max_pages, &a.table_ld));
    if (a.seqs == nullptr && a.T > a.num_seqs) return TGC_ERR_INVALID_ARG;
    TGC_TRY(kv_pages_check(a.num_pages, a.page_size, a.heads_k, a.D, &a.page_s, &a.token_s, &a.head_s));
    if (a.T == 0) return TGC_OK;
    if (a.pos == nullptr || a.table == nullptr || a.k_pages == nullptr || a.v_pages == nullptr || a.k == nullptr ||
        a.v == nullptr)
        return TGC_ERR_INVALID_ARG;
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
    p.pos = a.pos; p.freqs = a.freqs; p.table = a.table; p.seqs = a.seqs;
    p.T = (int)a.T; p.D = (int)a.D; p.R = (int)a.R;
    p.scale = a.scale; p.sign = 1.0f;
    p.kv = KvTable{(int)a.num_pages, (int)a.page_size, (int)a.num_seqs, (int)a.max_pages, a.table_ld};
    p.page_s = a.page_s; p.token_s = a.token_s;
    const bool interleaved = a.layout == TGC_ROPE_INTERLEAVED;
    return launch_rope(p, interleaved, a.dtype, rope_vector(p, interleaved, es, a.k_pages, a.v_pages, a.head_s), a.stream);
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
