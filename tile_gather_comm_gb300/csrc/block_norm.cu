// block_norm.cu -- tgc_block_norm and tgc_block_norm_bwd: the norms before and after a
// transformer block, fused with the block's gate and residual scale.
//
//   forward   u = post(y), r = a x + c g u, h = pre(r)
//   backward  t = dr + pre'(dh; r), dx = a t, du = c g t, dgate = sum c t u,
//             dy = post'(du; y), and the sums over rows for weights and biases
//   with, for a norm v -> vhat w + b,   q = d w:
//     rms    vhat = v rstd,           dv = rstd (q - vhat mean(q vhat))
//     layer  vhat = (v - mean) rstd,  dv = rstd (q - mean(q) - vhat mean(q vhat))
//
// Bound by memory: every (M, D) tensor is read or written once.  A row is held in the
// registers of its team of threads from the first load to the last store, so the several
// passes a norm needs (mean, deviations, the gradient's two means) touch no memory.  A team
// is a warp (rows of up to 32 vectors; no barrier at all) or a whole block.
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "act.cuh"
#include "internal.h"

namespace tgc {

constexpr int kMaxTeam = 1024;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const void *base, int64_t at) {
    return *reinterpret_cast<const Pack<T, VEC> *>(static_cast<const T *>(base) + at);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(void *base, int64_t at, const float *f) {
    Pack<T, VEC> p;
#pragma unroll
    for (int i = 0; i < VEC; ++i) p.v[i] = from_f32<T>(f[i]);
    *reinterpret_cast<Pack<T, VEC> *>(static_cast<T *>(base) + at) = p;
}

// Sums of N values over the team, the same in every thread and every run: shuffles inside a
// warp, then, for a team of a whole block, one round through shared memory.  `buf` alternates
// between two areas, so one barrier a call suffices.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*smem)[N][32], int *buf) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int d = 16; d > 0; d /= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    if (blockDim.y > 1 || blockDim.x <= 32) return;  // a team is a warp
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) smem[*buf][i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = lane < warps ? smem[*buf][i][lane] : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
        v[i] = s;
    }
    *buf ^= 1;
}

// ---------------------------------------------------------------- forward

struct NormParams {
    const void *y, *x, *gate, *post_w, *post_b, *pre_w, *pre_b;
    void *r, *h;
    int M, D, rows_per_gate;
    int64_t ldy, ldx, ldr, ldh;
    int post, pre;
    float res_scale, branch_scale, eps, inv_d;
};

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxTeam) norm_kernel(const NormParams p) {
    __shared__ float smem[2][1][32];
    int buf = 0;
    const int m = blockIdx.x * blockDim.y + threadIdx.y;
    if (m >= p.M) return;  // whole teams only: a block of one team, or warps that need no barrier
    const int64_t row = m;
    float v[NV][VEC];
    // v := deviations of v from `mean`, and the reciprocal deviation
    auto stats = [&](int kind) -> float {
        if (kind == TGC_NORM_LAYER) {
            float s[1] = {0.0f};
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[0] += v[k][i];
            team_sum(s, smem, &buf);
            const float mean = s[0] * p.inv_d;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if ((k * (int)blockDim.x + (int)threadIdx.x) * VEC < p.D)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[k][i] -= mean;
        }
        float q[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) q[0] += v[k][i] * v[k][i];
        team_sum(q, smem, &buf);
        return rsqrtf(q[0] * p.inv_d + p.eps);
    };
    auto affine = [&](int kind, const void *w, const void *b) {
        const float rstd = stats(kind);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * VEC;
            if (c >= p.D) continue;
            Pack<T, VEC> pw, pb;
            if (w != nullptr) pw = load_pack<T, VEC>(w, c);
            if (b != nullptr) pb = load_pack<T, VEC>(b, c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[k][i] *= rstd;
                if (w != nullptr) v[k][i] *= to_f32(pw.v[i]);
                if (b != nullptr) v[k][i] += to_f32(pb.v[i]);
            }
        }
    };
    Pack<T, VEC> px[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * VEC;
        if (c < p.D) {
            const Pack<T, VEC> py = load_pack<T, VEC>(p.y, row * p.ldy + c);
            if (p.x != nullptr) px[k] = load_pack<T, VEC>(p.x, row * p.ldx + c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[k][i] = to_f32(py.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[k][i] = 0.0f;
        }
    }
    if (p.post != TGC_NORM_NONE) affine(p.post, p.post_w, p.post_b);
    const int64_t gate_row = p.gate != nullptr ? (int64_t)(m / p.rows_per_gate) * p.D : 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * VEC;
        if (c >= p.D) continue;
        Pack<T, VEC> pg;
        if (p.gate != nullptr) pg = load_pack<T, VEC>(p.gate, gate_row + c);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            v[k][i] *= p.branch_scale;
            if (p.gate != nullptr) v[k][i] *= to_f32(pg.v[i]);
            if (p.x != nullptr) v[k][i] += p.res_scale * to_f32(px[k].v[i]);
        }
        if (p.r != nullptr) store_pack<T, VEC>(p.r, row * p.ldr + c, v[k]);
    }
    if (p.pre == TGC_NORM_NONE) return;
    affine(p.pre, p.pre_w, p.pre_b);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * VEC;
        if (c < p.D) store_pack<T, VEC>(p.h, row * p.ldh + c, v[k]);
    }
}

// ---------------------------------------------------------------- backward

// Rows are dealt in units: a unit is up to unit_rows consecutive rows that share a gate
// vector.  A worker (a team) takes units worker, worker + workers, ...; it keeps the sums for
// weights and biases over all its units, and those for the gate over one unit, in registers.
// The sums leave as fp32 partials that norm_sum_kernel adds in a fixed order.
struct NormBwdParams {
    const void *y, *r, *dr, *dh, *gate, *post_w, *post_b, *pre_w;
    void *dx, *dy, *dgate;
    float *partial;       // [4][workers][D]: dpost_w, dpost_b, dpre_w, dpre_b
    float *gate_partial;  // [units][D], or null where a unit is a whole gate segment
    int M, D, rows_per_gate, units_per_gate, unit_rows, units, workers;
    int64_t ldy, ldr, lddr, lddh, lddx, lddy;
    int post, pre;
    bool want[4];
    bool need_y;
    float res_scale, branch_scale, eps, inv_d;
};

// FULL: sums for biases too.
template <typename T, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(kMaxTeam) norm_bwd_kernel(const NormBwdParams p) {
    __shared__ float smem[2][2][32];
    int buf = 0;
    const int worker = blockIdx.x * blockDim.y + threadIdx.y;
    if (worker >= p.workers) return;
    float a_gate[NV][VEC], a_post[NV][VEC], a_pre[NV][VEC], a_postb[FULL ? NV : 1][VEC], a_preb[FULL ? NV : 1][VEC];
    auto clear = [](auto &a) {
#pragma unroll
        for (auto &k : a)
#pragma unroll
            for (float &f : k) f = 0.0f;
    };
    clear(a_post); clear(a_pre); clear(a_postb); clear(a_preb);
    // Deviations of v (in place) and the reciprocal deviation.
    auto stats = [&](float (&v)[NV][VEC], int kind) -> float {
        if (kind == TGC_NORM_LAYER) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[0] += v[k][i];
            team_sum(s, smem, &buf);
            const float mean = s[0] * p.inv_d;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if ((k * (int)blockDim.x + (int)threadIdx.x) * VEC < p.D)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[k][i] -= mean;
        }
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) q[0] += v[k][i] * v[k][i];
        team_sum(q, smem, &buf);
        return rsqrtf(q[0] * p.inv_d + p.eps);
    };
    for (int unit = worker; unit < p.units; unit += p.workers) {
        const int seg = unit / p.units_per_gate, part = unit % p.units_per_gate;
        const int m0 = seg * p.rows_per_gate + part * p.unit_rows;
        const int seg_end = (seg + 1) * p.rows_per_gate;
        const int m1 = m0 + p.unit_rows < seg_end ? m0 + p.unit_rows : seg_end;
        clear(a_gate);
        for (int m = m0; m < m1; ++m) {
            const int64_t row = m;
            float t[NV][VEC];  // dr, then t
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
                for (int i = 0; i < VEC; ++i) t[k][i] = 0.0f;
                if (p.dr != nullptr && c < p.D) {
                    const Pack<T, VEC> pk = load_pack<T, VEC>(p.dr, row * p.lddr + c);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) t[k][i] = to_f32(pk.v[i]);
                }
            }
            if (p.pre != TGC_NORM_NONE) {
                float v[NV][VEC], q[NV][VEC];
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = (k * blockDim.x + threadIdx.x) * VEC;
                    if (c < p.D) {
                        const Pack<T, VEC> pr = load_pack<T, VEC>(p.r, row * p.ldr + c);
                        const Pack<T, VEC> pd = load_pack<T, VEC>(p.dh, row * p.lddh + c);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) { v[k][i] = to_f32(pr.v[i]); q[k][i] = to_f32(pd.v[i]); }
                    } else {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) v[k][i] = q[k][i] = 0.0f;
                    }
                }
                const float rstd = stats(v, p.pre);
                float s[2] = {0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = (k * blockDim.x + threadIdx.x) * VEC;
                    if (c >= p.D) continue;
                    Pack<T, VEC> pw;
                    if (p.pre_w != nullptr) pw = load_pack<T, VEC>(p.pre_w, c);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        v[k][i] *= rstd;
                        a_pre[k][i] += q[k][i] * v[k][i];
                        if (FULL) a_preb[k][i] += q[k][i];
                        if (p.pre_w != nullptr) q[k][i] *= to_f32(pw.v[i]);
                        s[0] += q[k][i] * v[k][i];
                        s[1] += q[k][i];
                    }
                }
                team_sum(s, smem, &buf);
                const float s0 = s[0] * p.inv_d, s1 = p.pre == TGC_NORM_LAYER ? s[1] * p.inv_d : 0.0f;
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) t[k][i] += rstd * (q[k][i] - s1 - v[k][i] * s0);
            }
            if (p.need_y) {
                float v[NV][VEC], q[NV][VEC];
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = (k * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[k][i] = 0.0f;
                    if (c < p.D) {
                        const Pack<T, VEC> py = load_pack<T, VEC>(p.y, row * p.ldy + c);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) v[k][i] = to_f32(py.v[i]);
                    }
                }
                const float rstd = p.post != TGC_NORM_NONE ? stats(v, p.post) : 1.0f;
                float s[2] = {0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = (k * blockDim.x + threadIdx.x) * VEC;
                    if (c >= p.D) continue;
                    Pack<T, VEC> pw, pb, pg;
                    if (p.post_w != nullptr) pw = load_pack<T, VEC>(p.post_w, c);
                    if (p.post_b != nullptr) pb = load_pack<T, VEC>(p.post_b, c);
                    if (p.gate != nullptr) pg = load_pack<T, VEC>(p.gate, (int64_t)seg * p.D + c);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        v[k][i] *= rstd;
                        float u = v[k][i], du = p.branch_scale * t[k][i];
                        if (p.post_w != nullptr) u *= to_f32(pw.v[i]);
                        if (p.post_b != nullptr) u += to_f32(pb.v[i]);
                        a_gate[k][i] += du * u;
                        if (p.gate != nullptr) du *= to_f32(pg.v[i]);
                        a_post[k][i] += du * v[k][i];
                        if (FULL) a_postb[k][i] += du;
                        q[k][i] = p.post_w != nullptr ? du * to_f32(pw.v[i]) : du;
                        s[0] += q[k][i] * v[k][i];
                        s[1] += q[k][i];
                    }
                }
                if (p.post != TGC_NORM_NONE && p.dy != nullptr) team_sum(s, smem, &buf);
                const float s0 = p.post != TGC_NORM_NONE ? s[0] * p.inv_d : 0.0f;
                const float s1 = p.post == TGC_NORM_LAYER ? s[1] * p.inv_d : 0.0f;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = (k * blockDim.x + threadIdx.x) * VEC;
                    if (c >= p.D || p.dy == nullptr) continue;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) q[k][i] = rstd * (q[k][i] - s1 - v[k][i] * s0);
                    store_pack<T, VEC>(p.dy, row * p.lddy + c, q[k]);
                }
            } else if (p.dy != nullptr) {  // no post norm: dy = du
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = (k * blockDim.x + threadIdx.x) * VEC;
                    if (c >= p.D) continue;
                    Pack<T, VEC> pg;
                    if (p.gate != nullptr) pg = load_pack<T, VEC>(p.gate, (int64_t)seg * p.D + c);
                    float q[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        q[i] = p.branch_scale * t[k][i];
                        if (p.gate != nullptr) q[i] *= to_f32(pg.v[i]);
                    }
                    store_pack<T, VEC>(p.dy, row * p.lddy + c, q);
                }
            }
            if (p.dx != nullptr) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = (k * blockDim.x + threadIdx.x) * VEC;
                    if (c >= p.D) continue;
                    float q[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) q[i] = p.res_scale * t[k][i];
                    store_pack<T, VEC>(p.dx, row * p.lddx + c, q);
                }
            }
        }
        if (p.dgate != nullptr) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * blockDim.x + threadIdx.x) * VEC;
                if (c >= p.D) continue;
                if (p.gate_partial == nullptr) store_pack<T, VEC>(p.dgate, (int64_t)seg * p.D + c, a_gate[k]);
                else
#pragma unroll
                    for (int i = 0; i < VEC; ++i) p.gate_partial[(int64_t)unit * p.D + c + i] = a_gate[k][i];
            }
        }
    }
    auto put = [&](int which, const auto &a) {
        if (!p.want[which]) return;
        float *to = p.partial + ((int64_t)which * p.workers + worker) * p.D;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * VEC;
            if (c >= p.D) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) to[c + i] = a[k][i];
        }
    };
    put(0, a_post);
    put(2, a_pre);
    if constexpr (FULL) {
        put(1, a_postb);
        put(3, a_preb);
    }
}

// Adds the partials of one output vector: blockIdx.y 0..3 the parameter vectors, then one a gate.
struct NormSumParams {
    const float *partial, *gate_partial;
    void *out[4];
    void *dgate;
    int D, workers, units_per_gate;
};

template <typename T>
__global__ void __launch_bounds__(256) norm_sum_kernel(const NormSumParams p) {
    __shared__ float part[8][32];
    const int which = blockIdx.y;
    const float *from;
    T *to;
    int n;
    if (which < 4) {
        if (p.out[which] == nullptr) return;
        from = p.partial + (int64_t)which * p.workers * p.D;
        to = static_cast<T *>(p.out[which]);
        n = p.workers;
    } else {
        const int64_t g = which - 4;
        from = p.gate_partial + g * p.units_per_gate * p.D;
        to = static_cast<T *>(p.dgate) + g * p.D;
        n = p.units_per_gate;
    }
    const int c = blockIdx.x * 32 + threadIdx.x % 32, l = threadIdx.x / 32;
    float s = 0.0f;
    if (c < p.D)
        for (int i = l; i < n; i += 8) s += from[(int64_t)i * p.D + c];
    part[l][threadIdx.x % 32] = s;
    __syncthreads();
    if (l == 0 && c < p.D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][threadIdx.x];
        to[c] = from_f32<T>(s);
    }
}

// ---------------------------------------------------------------- host side

static int norm_elem(tgc_dtype dt) { return dt == TGC_BF16 || dt == TGC_F16 ? 2 : dt == TGC_F32 ? 4 : 0; }

// One (rows, D) tensor: resolves its row stride, checks it, and clears *vec where its rows are
// not all 16-byte aligned.
static int norm_matrix(const void *p, int64_t rows, int64_t D, int es, int64_t *ld, bool *vec) {
    if (*ld == 0) *ld = D;
    if (p == nullptr) return TGC_OK;
    if (*ld < D) return TGC_ERR_INVALID_ARG;
    int64_t bytes = 0;
    if (__builtin_mul_overflow(*ld, rows * es, &bytes) || bytes >= (int64_t(1) << 62)) return TGC_ERR_INVALID_ARG;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (at % es != 0) return TGC_ERR_ALIGN;
    if (at % 16 != 0 || (rows > 1 && *ld * es % 16 != 0)) *vec = false;
    return TGC_OK;
}

static bool norm_kind(tgc_norm k) { return k == TGC_NORM_NONE || k == TGC_NORM_RMS || k == TGC_NORM_LAYER; }

// Threads a team and vectors a thread for rows of D: NV 1, 2 or 4 vectors, or 1, 4 or 16 single
// elements, a thread (16384 columns for a team of 1024 at the widest).
struct TeamShape {
    int vec, nv, team, teams;  // teams a block
};
static TeamShape team_shape(int64_t D, int es, bool vec, int prefer) {
    TeamShape s{};
    s.vec = vec && D * es % 16 == 0 ? 16 / es : 1;
    const int64_t n = (D + s.vec - 1) / s.vec;
    const int steps[2][3] = {{1, 4, 16}, {1, 2, 4}};
    for (int i = 0; i < 3; ++i) {
        s.nv = steps[s.vec > 1][i];
        if (n <= (int64_t)s.nv * prefer) break;
    }
    s.team = (int)((n + s.nv - 1) / s.nv + 31) / 32 * 32;
    s.teams = s.team == 32 ? 4 : 1;
    return s;
}

template <typename T>
static void launch_norm(const NormParams &p, const TeamShape &s, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const dim3 block(s.team, s.teams);
    const unsigned grid = (unsigned)((p.M + s.teams - 1) / s.teams);
    if (s.vec > 1) {
        if (s.nv == 1) norm_kernel<T, V, 1><<<grid, block, 0, stream>>>(p);
        else if (s.nv == 2) norm_kernel<T, V, 2><<<grid, block, 0, stream>>>(p);
        else norm_kernel<T, V, 4><<<grid, block, 0, stream>>>(p);
    } else {
        if (s.nv == 1) norm_kernel<T, 1, 1><<<grid, block, 0, stream>>>(p);
        else if (s.nv == 4) norm_kernel<T, 1, 4><<<grid, block, 0, stream>>>(p);
        else norm_kernel<T, 1, 16><<<grid, block, 0, stream>>>(p);
    }
}

#define TGC_TRY(expr)                     \
    do {                                  \
        const int rc_ = (expr);           \
        if (rc_ != TGC_OK) return rc_;    \
    } while (0)

static int norm_impl(tgc_block_norm_args a) {
    const int es = norm_elem(a.dtype);
    if (es == 0) return TGC_ERR_DTYPE;
    if (a.M < 0 || a.M >= (int64_t(1) << 31) || a.D < 1 || a.D > TGC_NORM_MAX_D) return TGC_ERR_INVALID_ARG;
    if (!norm_kind(a.post) || !norm_kind(a.pre)) return TGC_ERR_INVALID_ARG;
    if (a.gate == nullptr ? a.gates != 0 : (a.gates < 1 || a.M % a.gates != 0)) return TGC_ERR_INVALID_ARG;
    if (a.post == TGC_NORM_NONE && (a.post_weight != nullptr || a.post_bias != nullptr)) return TGC_ERR_INVALID_ARG;
    if (a.pre == TGC_NORM_NONE && (a.pre_weight != nullptr || a.pre_bias != nullptr)) return TGC_ERR_INVALID_ARG;
    if ((a.post != TGC_NORM_NONE || a.pre != TGC_NORM_NONE) && !(a.eps > 0.0f)) return TGC_ERR_INVALID_ARG;
    if (a.M == 0) return TGC_OK;
    if ((a.pre != TGC_NORM_NONE) != (a.h != nullptr)) return TGC_ERR_INVALID_ARG;
    if (a.r == nullptr && a.h == nullptr) return TGC_ERR_INVALID_ARG;
    if (a.y == nullptr) return TGC_ERR_INVALID_ARG;
    bool vec = true;
    TGC_TRY(norm_matrix(a.y, a.M, a.D, es, &a.ldy, &vec));
    TGC_TRY(norm_matrix(a.x, a.M, a.D, es, &a.ldx, &vec));
    TGC_TRY(norm_matrix(a.r, a.M, a.D, es, &a.ldr, &vec));
    TGC_TRY(norm_matrix(a.h, a.M, a.D, es, &a.ldh, &vec));
    for (const void *v : {a.gate, a.post_weight, a.post_bias, a.pre_weight, a.pre_bias}) {
        int64_t ld = a.D;
        TGC_TRY(norm_matrix(v, v == a.gate ? a.gates : 1, a.D, es, &ld, &vec));
    }
    const TeamShape s = team_shape(a.D, es, vec, 512);
    NormParams p{};
    p.y = a.y; p.x = a.x; p.gate = a.gate;
    p.post_w = a.post_weight; p.post_b = a.post_bias; p.pre_w = a.pre_weight; p.pre_b = a.pre_bias;
    p.r = a.r; p.h = a.h;
    p.M = (int)a.M; p.D = (int)a.D; p.rows_per_gate = a.gate != nullptr ? (int)(a.M / a.gates) : (int)a.M;
    p.ldy = a.ldy; p.ldx = a.ldx; p.ldr = a.ldr; p.ldh = a.ldh;
    p.post = a.post; p.pre = a.pre;
    p.res_scale = a.res_scale; p.branch_scale = a.branch_scale; p.eps = a.eps; p.inv_d = 1.0f / (float)a.D;
    if (a.dtype == TGC_BF16) launch_norm<__nv_bfloat16>(p, s, a.stream);
    else if (a.dtype == TGC_F16) launch_norm<__half>(p, s, a.stream);
    else launch_norm<float>(p, s, a.stream);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
}

// How the backward pass deals its rows.  About two workers an SM (more for narrow rows, whose
// teams are small), units of at least 4 rows, and whole gate segments where there are enough.
struct NormPlan {
    int segments, rows_per_gate, units_per_gate, unit_rows, units, workers;
    size_t gate_off, total;
};

static NormPlan norm_plan(const tgc_block_norm_bwd_args &a) {
    NormPlan q{};
    const int64_t target = a.D <= 512 ? 1216 : 304;
    q.segments = a.gate != nullptr ? (int)a.gates : 1;
    q.rows_per_gate = (int)(a.M / q.segments);
    int64_t upg = (target + q.segments - 1) / q.segments;
    const int64_t most = (q.rows_per_gate + 3) / 4;
    if (upg > most) upg = most;
    q.unit_rows = (int)((q.rows_per_gate + upg - 1) / upg);
    q.units_per_gate = (q.rows_per_gate + q.unit_rows - 1) / q.unit_rows;
    q.units = q.units_per_gate * q.segments;
    q.workers = q.units < target ? q.units : (int)target;
    auto up = [](size_t v) { return (v + 127) / 128 * 128; };
    const bool sums = a.dpost_weight != nullptr || a.dpost_bias != nullptr || a.dpre_weight != nullptr ||
                      a.dpre_bias != nullptr;
    q.gate_off = sums ? up((size_t)4 * q.workers * (size_t)a.D * 4) : 0;
    q.total = q.gate_off + (a.dgate != nullptr && q.units_per_gate > 1 ? up((size_t)q.units * (size_t)a.D * 4) : 0);
    return q;
}

static int norm_bwd_check(tgc_block_norm_bwd_args &a, bool *vec) {
    const int es = norm_elem(a.dtype);
    if (es == 0) return TGC_ERR_DTYPE;
    if (a.M < 0 || a.M >= (int64_t(1) << 31) || a.D < 1 || a.D > TGC_NORM_MAX_D) return TGC_ERR_INVALID_ARG;
    if (!norm_kind(a.post) || !norm_kind(a.pre)) return TGC_ERR_INVALID_ARG;
    if (a.gate == nullptr ? (a.gates != 0 || a.dgate != nullptr) : (a.gates < 1 || a.M % a.gates != 0))
        return TGC_ERR_INVALID_ARG;
    if (a.post == TGC_NORM_NONE && (a.post_weight != nullptr || a.post_bias != nullptr || a.dpost_weight != nullptr ||
                                    a.dpost_bias != nullptr))
        return TGC_ERR_INVALID_ARG;
    if (a.pre == TGC_NORM_NONE && (a.pre_weight != nullptr || a.dpre_weight != nullptr || a.dpre_bias != nullptr))
        return TGC_ERR_INVALID_ARG;
    if ((a.post != TGC_NORM_NONE || a.pre != TGC_NORM_NONE) && !(a.eps > 0.0f)) return TGC_ERR_INVALID_ARG;
    if (a.M > 0) {
        if ((a.pre != TGC_NORM_NONE) != (a.dh != nullptr)) return TGC_ERR_INVALID_ARG;
        if (a.pre != TGC_NORM_NONE && a.r == nullptr) return TGC_ERR_INVALID_ARG;
        if ((a.post != TGC_NORM_NONE || a.dgate != nullptr) && a.y == nullptr) return TGC_ERR_INVALID_ARG;
    }
    TGC_TRY(norm_matrix(a.y, a.M, a.D, es, &a.ldy, vec));
    TGC_TRY(norm_matrix(a.r, a.M, a.D, es, &a.ldr, vec));
    TGC_TRY(norm_matrix(a.dr, a.M, a.D, es, &a.lddr, vec));
    TGC_TRY(norm_matrix(a.dh, a.M, a.D, es, &a.lddh, vec));
    TGC_TRY(norm_matrix(a.dx, a.M, a.D, es, &a.lddx, vec));
    TGC_TRY(norm_matrix(a.dy, a.M, a.D, es, &a.lddy, vec));
    for (const void *v : {a.gate, (const void *)a.dgate}) {
        int64_t ld = a.D;
        TGC_TRY(norm_matrix(v, a.gates, a.D, es, &ld, vec));
    }
    for (const void *v : {a.post_weight, a.post_bias, a.pre_weight, (const void *)a.dpost_weight, (const void *)a.dpost_bias,
                          (const void *)a.dpre_weight, (const void *)a.dpre_bias}) {
        int64_t ld = a.D;
        TGC_TRY(norm_matrix(v, 1, a.D, es, &ld, vec));
    }
    return TGC_OK;
}

template <typename T, int V, int NV>
static void launch_norm_bwd_nv(const NormBwdParams &p, bool full, dim3 grid, dim3 block, cudaStream_t stream) {
    if (full) norm_bwd_kernel<T, V, NV, true><<<grid, block, 0, stream>>>(p);
    else norm_bwd_kernel<T, V, NV, false><<<grid, block, 0, stream>>>(p);
}

template <typename T>
static void launch_norm_bwd(const NormBwdParams &p, const NormSumParams &q, int nsums, const TeamShape &s, bool full,
                            cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const dim3 block(s.team, s.teams), grid((unsigned)((p.workers + s.teams - 1) / s.teams));
    if (s.vec > 1) {
        if (s.nv == 1) launch_norm_bwd_nv<T, V, 1>(p, full, grid, block, stream);
        else if (s.nv == 2) launch_norm_bwd_nv<T, V, 2>(p, full, grid, block, stream);
        else launch_norm_bwd_nv<T, V, 4>(p, full, grid, block, stream);
    } else {
        if (s.nv == 1) launch_norm_bwd_nv<T, 1, 1>(p, full, grid, block, stream);
        else if (s.nv == 4) launch_norm_bwd_nv<T, 1, 4>(p, full, grid, block, stream);
        else launch_norm_bwd_nv<T, 1, 16>(p, full, grid, block, stream);
    }
    if (nsums > 0) norm_sum_kernel<T><<<dim3((unsigned)((p.D + 31) / 32), (unsigned)nsums), 256, 0, stream>>>(q);
}

static int norm_bwd_impl(tgc_block_norm_bwd_args a) {
    bool vec = true;
    TGC_TRY(norm_bwd_check(a, &vec));
    void *const outs[4] = {a.dpost_weight, a.dpost_bias, a.dpre_weight, a.dpre_bias};
    if (a.M == 0) {
        const size_t es = (size_t)norm_elem(a.dtype);
        cudaError_t e = cudaSuccess;
        for (void *o : outs)
            if (o != nullptr && e == cudaSuccess) e = cudaMemsetAsync(o, 0, (size_t)a.D * es, a.stream);
        if (a.dgate != nullptr && e == cudaSuccess)
            e = cudaMemsetAsync(a.dgate, 0, (size_t)a.gates * (size_t)a.D * es, a.stream);
        return e == cudaSuccess ? TGC_OK : cuda_fail(e);
    }
    const NormPlan q = norm_plan(a);
    if (q.total > 0) {
        if (a.workspace == nullptr || a.workspace_bytes < q.total) return TGC_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(a.workspace) % 128 != 0) return TGC_ERR_ALIGN;
    }
    const TeamShape s = team_shape(a.D, norm_elem(a.dtype), vec, 512);
    NormBwdParams p{};
    p.y = a.y; p.r = a.r; p.dr = a.dr; p.dh = a.dh; p.gate = a.gate;
    p.post_w = a.post_weight; p.post_b = a.post_bias; p.pre_w = a.pre_weight;
    p.dx = a.dx; p.dy = a.dy; p.dgate = a.dgate;
    p.partial = static_cast<float *>(a.workspace);
    if (a.dgate != nullptr && q.units_per_gate > 1)
        p.gate_partial = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + q.gate_off);
    p.M = (int)a.M; p.D = (int)a.D; p.rows_per_gate = q.rows_per_gate; p.units_per_gate = q.units_per_gate;
    p.unit_rows = q.unit_rows; p.units = q.units; p.workers = q.workers;
    p.ldy = a.ldy; p.ldr = a.ldr; p.lddr = a.lddr; p.lddh = a.lddh; p.lddx = a.lddx; p.lddy = a.lddy;
    p.post = a.post; p.pre = a.pre;
    for (int i = 0; i < 4; ++i) p.want[i] = outs[i] != nullptr;
    p.need_y = a.post != TGC_NORM_NONE || a.dgate != nullptr;
    p.res_scale = a.res_scale; p.branch_scale = a.branch_scale; p.eps = a.eps; p.inv_d = 1.0f / (float)a.D;
    NormSumParams n{};
    n.partial = p.partial; n.gate_partial = p.gate_partial; n.dgate = a.dgate;
    for (int i = 0; i < 4; ++i) n.out[i] = outs[i];
    n.D = p.D; n.workers = p.workers; n.units_per_gate = p.units_per_gate;
    const bool sums = outs[0] != nullptr || outs[1] != nullptr || outs[2] != nullptr || outs[3] != nullptr;
    const int nsums = p.gate_partial != nullptr ? 4 + q.segments : sums ? 4 : 0;
    const bool full = outs[1] != nullptr || outs[3] != nullptr;
    if (a.dtype == TGC_BF16) launch_norm_bwd<__nv_bfloat16>(p, n, nsums, s, full, a.stream);
    else if (a.dtype == TGC_F16) launch_norm_bwd<__half>(p, n, nsums, s, full, a.stream);
    else launch_norm_bwd<float>(p, n, nsums, s, full, a.stream);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
}

}  // namespace tgc

extern "C" int tgc_block_norm(const tgc_block_norm_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::norm_impl(*args);
}

extern "C" int tgc_block_norm_bwd(const tgc_block_norm_bwd_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::norm_bwd_impl(*args);
}

extern "C" size_t tgc_block_norm_bwd_workspace_bytes(const tgc_block_norm_bwd_args *args) {
    if (args == nullptr) return 0;
    tgc_block_norm_bwd_args a = *args;
    bool vec = true;
    if (tgc::norm_bwd_check(a, &vec) != TGC_OK || a.M == 0) return 0;
    return tgc::norm_plan(a).total;
}
