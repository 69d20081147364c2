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
// Measured, bf16, 8192 x 4096, rms norms, gate and residual: forward 48.7 us (5.5 TB/s, 67 % of the
// issue slots), backward 85 us and 8 to 10 for the sums over rows (90 together, the launches overlap):
// 4.5 TB/s and 44 % of the issue slots, neither of them full.  A team of 16 warps is all that an SM's
// registers hold, and for each pair of rows all of it waits at one barrier for the sums.
#include <atomic>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include <cuda_runtime.h>

#include "act.cuh"
#include "internal.h"
#include "pairs.cuh"
#include "prims.cuh"

namespace tgc {

// Threads of a block at most, and with them a kernel's register budget.  Forward: 64 a thread where a
// thread holds one vector (two teams of 512 on an SM) or a team may have 1024, 128 elsewhere.
// Backward: 128, and 96 where a thread holds four single elements: more teams then fit an SM
// (2500 x 1191 f16 33 -> 30 us, with layer norms 4096 x 1191 bf16 81 -> 61; 1000 x 777 fp32
// 18.7 -> 19.5).
template <typename T, int VEC, int NV>
constexpr int kFwdMax = (VEC == 1 && NV == 16) || (sizeof(T) == 4 && NV == 4 && VEC > 1) ? 1024 : 512;
template <int VEC, int NV>
constexpr int kBwdMax = VEC == 1 && NV == 4 ? 640 : 512;

// VEC consecutive elements as the words they are loaded in.  Arithmetic goes by L: two elements at
// a time, or one where VEC is 1; get(i) is the i-th such lane in fp32, set(i, f) rounds it back.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    using L = F2;
    uint32_t w[sizeof(T) * VEC / 4];
    __device__ __forceinline__ F2 get(int i) const {
        if constexpr (sizeof(T) == 4) {
            return f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            return f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            return f2(f.x, f.y);
        }
    }
    __device__ __forceinline__ void set(int i, F2 v) {
        const float2 f = split(v);
        if constexpr (sizeof(T) == 4) {
            w[2 * i] = __float_as_uint(f.x);
            w[2 * i + 1] = __float_as_uint(f.y);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f.y), "f"(f.x));
        } else {
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f.y), "f"(f.x));
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t &x : w) x = 0u;
    }
    // Elements used before are converted again after this, not kept in fp32 meanwhile.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (uint32_t &x : w) asm volatile("" : "+r"(x));
    }
};
template <typename T>
struct Pack<T, 1> {
    using L = float;
    T v;
    __device__ __forceinline__ float get(int) const { return to_f32(v); }
    __device__ __forceinline__ void set(int, float f) { v = from_f32<T>(f); }
    __device__ __forceinline__ void clear() { v = from_f32<T>(0.0f); }
    __device__ __forceinline__ void forget() {}
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const void *base, int64_t at) {
    return *reinterpret_cast<const Pack<T, VEC> *>(static_cast<const T *>(base) + at);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(void *base, int64_t at, const typename Pack<T, VEC>::L *f) {
    Pack<T, VEC> p;
#pragma unroll
    for (int i = 0; i < (VEC > 1 ? VEC / 2 : 1); ++i) p.set(i, f[i]);
    *reinterpret_cast<Pack<T, VEC> *>(static_cast<T *>(base) + at) = p;
}
// fp32 in memory <-> lanes
__device__ __forceinline__ void read_lanes(const float *from, float (&to)[1]) { to[0] = from[0]; }
__device__ __forceinline__ void write_lanes(float *to, const float (&from)[1]) { to[0] = from[0]; }
template <int NP>
__device__ __forceinline__ void read_lanes(const float *from, F2 (&to)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; i += 2) {
        const float4 f = *reinterpret_cast<const float4 *>(from + 2 * i);
        to[i] = f2(f.x, f.y);
        to[i + 1] = f2(f.z, f.w);
    }
}
template <int NP>
__device__ __forceinline__ void write_lanes(float *to, const F2 (&from)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; i += 2) {
        const float2 a = split(from[i]), b = split(from[i + 1]);
        *reinterpret_cast<float4 *>(to + 2 * i) = make_float4(a.x, a.y, b.x, b.y);
    }
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

// The same for N = 8 or 16 values at once, with a fraction of the shuffles: in the first steps a
// lane hands half of its values to its partner and keeps the other half, so after log2(N) steps
// each lane holds one value's sum over a few lanes.  smem[value][warp]; unused warps' entries are
// zero from the start (clear_sums).
template <int N>
__device__ __forceinline__ void team_sum_many(float (&v)[N], float (*smem)[N][32], int *buf) {
    static_assert(N == 8 || N == 16, "values");
    const int lane = threadIdx.x % 32;
    int d = 16;
#pragma unroll
    for (int n = N; n > 1; n /= 2, d /= 2) {
        const bool up = (lane & d) != 0;  // keeps the upper half of the n values
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float give = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
        }
    }
    float s = v[0];
#pragma unroll
    for (int e = 32 / N / 2; e > 0; e /= 2) s += __shfl_xor_sync(0xffffffffu, s, e);
    // lanes l * (32 / N) .. hold value l: bit 16 of the lane chose its highest index bit, and so on
    if (blockDim.y == 1 && blockDim.x > 32) {
        constexpr int kPer = 32 / N;  // lanes of a value, each adding 32 / kPer warps
        if (lane % kPer == 0) smem[*buf][lane / kPer][threadIdx.x / 32] = s;
        __syncthreads();
        const float4 *from = reinterpret_cast<const float4 *>(smem[*buf][lane / kPer] + (lane % kPer) * N);
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 f = from[i];
            s += (f.x + f.y) + (f.z + f.w);
        }
#pragma unroll
        for (int e = kPer / 2; e > 0; e /= 2) s += __shfl_xor_sync(0xffffffffu, s, e);
        *buf ^= 1;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, s, i * (32 / N));
}

// Rows arrive through shared memory where a thread's vectors are aligned and a few rows of every
// input fit beside each other: one thread asks for whole rows with bulk copies, two rows ahead.
template <int VEC, int NV>
constexpr bool kStaged = VEC > 1 && NV <= 2;
// The backward pass of wider rows: registers hold a few vectors of its inputs at a time, read where
// they are used and twice a row (the second time from L1 or L2).  Held whole, rows spilled: 4000 x
// 2501 bf16 took 1161 us (139), 2000 x 16384 bf16 422 (142), 2000 x 8192 fp32 692 (107).
template <int VEC, int NV>
constexpr bool kLean = !kStaged<VEC, NV> && VEC * NV > 4;
template <int NV>
constexpr int kFwdRows = NV == 1 ? 2 : 1;  // staged rows the forward kernel works on at a time
template <int NV, bool FULL>
constexpr int kBwdRows = NV == 1 && !FULL ? 2 : 1;  // rows the backward kernel works on at a time

#ifndef TGC_ROW_TIMEOUT_NS
#define TGC_ROW_TIMEOUT_NS 2000000000ull
#endif

// Waits for the rows of a turn.  If they do not land within the limit the fault is marked and *dead set to
// 1 + turn: from then on the team waits no more and asks for no more rows, but goes through those that
// remain, with wrong results.  A barrier of the team lies between the wait of a turn and its ask, so no
// rows beyond the next turn's have been asked for then.  A limit of nothing (tests build the kernels so)
// looks once.
__device__ __forceinline__ void row_wait(uint64_t *bars, uint32_t turn, volatile uint32_t *dead, int *fault) {
    const uint32_t a = smem_addr(&bars[turn & 1u]), parity = (turn >> 1) & 1u;
    constexpr bool kLook = TGC_ROW_TIMEOUT_NS == 0;
    if (kLook ? mbar_test_wait(a, parity) : mbar_try_wait(a, parity)) return;
    if (*dead != 0) return;
    const uint64_t t0 = globaltimer_ns();
    for (uint64_t it = 1; !kLook && it < (1ull << 40); ++it) {
        if (mbar_try_wait(a, parity)) return;
        if ((it & 63) == 0 && (*dead != 0 || globaltimer_ns() - t0 > TGC_ROW_TIMEOUT_NS)) break;
    }
    raise_status(fault, kStatusTimeout);
    *dead = turn + 1;
}

// At a kernel's end: what a dead team asked for has time to land before shared memory is given up.
__device__ __forceinline__ void drain_rows(uint64_t *bars, const volatile uint32_t *dead) {
    const uint32_t d = *dead;
    if (d == 0) return;
    for (uint32_t t = d - 1; t <= d; ++t) mbar_drain_wait(&bars[t & 1u], (t >> 1) & 1u, 200000000ull);
}

// ---------------------------------------------------------------- forward

struct NormParams {
    const void *y, *x, *gate, *post_w, *post_b, *pre_w, *pre_b;
    void *r, *h;
    int M, D, rows_per_gate, workers;
    int64_t ldy, ldx, ldr, ldh;
    int post, pre;
    float res_scale, branch_scale, eps, inv_d;
    int *fault;
};

// A worker (a team) takes a run of consecutive rows, kFwdRows at a time, so that one reduction
// serves them all; the weights stay in its registers.  The next rows are on their way meanwhile:
// to shared memory (staged), or to registers.  BIAS: some norm has a bias.
// STAGED false: also the form for few rows, one a worker, where nothing is to be had ahead.
template <typename T, int VEC, int NV, bool BIAS, bool STAGED>
__global__ void __launch_bounds__(kFwdMax<T, VEC, NV>, NV == 1 ? 2 : 1) norm_kernel(const NormParams p) {
    using P = Pack<T, VEC>;
    using L = typename P::L;
    constexpr int NP = VEC > 1 ? VEC / 2 : 1;
    constexpr int ROWS = STAGED ? kFwdRows<NV> : 1;
    __shared__ float smem[2][ROWS][32];
    __shared__ uint64_t bars[4][2];
    __shared__ uint32_t deads[4];
    extern __shared__ __align__(16) uint8_t staged[];  // a team's own: two stages of ROWS rows of y and x
    int buf = 0;
    const int worker = blockIdx.x * blockDim.y + threadIdx.y;
    uint64_t *const bar = bars[threadIdx.y];
    volatile uint32_t *const dead = &deads[threadIdx.y];
    if (STAGED && threadIdx.x == 0) {
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
        *dead = 0u;
        fence_mbarrier_init();
    }
    if (STAGED && blockDim.y == 1) __syncthreads(); else __syncwarp();
    stream_wait();
    stream_release();
    if (worker >= p.workers) return;  // whole teams only: a block of one team, or warps that need no barrier
    const int m0 = (int)((int64_t)p.M * worker / p.workers), m1 = (int)((int64_t)p.M * (worker + 1) / p.workers);
    const int c0 = threadIdx.x * VEC, step = blockDim.x * VEC;
    const int row_bytes = step * NV * (int)sizeof(T);
    uint8_t *const stages = staged + threadIdx.y * (STAGED ? 4 * ROWS * row_bytes : 0);
    P w1[NV], w2[NV], g[NV], b1[BIAS ? NV : 1], b2[BIAS ? NV : 1];
    P ny[STAGED ? 1 : NV], nx[STAGED ? 1 : NV];  // the next row, where it is not staged
    auto fetch = [&](auto &to, const void *base, int64_t at) {
        if (base == nullptr) return;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (c0 + k * step < p.D) to[k] = load_pack<T, VEC>(base, at + c0 + k * step);
    };
    auto ask = [&](int m, int stage) {
        if (m >= m1) return;
        const int rows = m1 - m < ROWS ? m1 - m : ROWS;
        const uint32_t bytes = (uint32_t)(p.D * (int)sizeof(T));
        mbar_arrive_expect_tx(&bar[stage], bytes * rows * (p.x != nullptr ? 2 : 1));
        for (int r = 0; r < rows; ++r) {
            uint8_t *to = stages + (stage * ROWS + r) * 2 * row_bytes;
            bulk_g2s(to, static_cast<const T *>(p.y) + (m + r) * p.ldy, bytes, &bar[stage]);
            if (p.x != nullptr) bulk_g2s(to + row_bytes, static_cast<const T *>(p.x) + (m + r) * p.ldx, bytes, &bar[stage]);
        }
    };
    if constexpr (STAGED) {
        if (threadIdx.x == 0) {
            ask(m0, 0);
            ask(m0 + ROWS, 1);
        }
    } else {
        fetch(ny, p.y, m0 * p.ldy);
        fetch(nx, p.x, m0 * p.ldx);
    }
    fetch(w1, p.post_w, 0);
    fetch(w2, p.pre_w, 0);
    if constexpr (BIAS) {
        fetch(b1, p.post_b, 0);
        fetch(b2, p.pre_b, 0);
    }
    int seg = -1;
    uint32_t turn = 0;
    for (int m = m0; m < m1; m += ROWS, ++turn) {
        const uint32_t stage = turn & 1u;
        const uint8_t *const here = stages + stage * ROWS * 2 * row_bytes;
        if constexpr (STAGED) row_wait(bar, turn, dead, p.fault);
        L v[ROWS][NV][NP];  // columns past the row's end, and rows past the last, stay zeros
#pragma unroll
        for (int rr = 0; rr < ROWS; ++rr)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                P py;
                const bool in = c0 + k * step < p.D && (ROWS == 1 || m + rr < m1);
                if constexpr (STAGED)
                    py = *reinterpret_cast<const P *>(here + rr * 2 * row_bytes + (c0 + k * step) * (int)sizeof(T));
                else py = ny[k];
#pragma unroll
                for (int i = 0; i < NP; ++i) v[rr][k][i] = in ? py.get(i) : every<L>(0.0f);
            }
        if constexpr (!STAGED)
            if (m + 1 < m1) fetch(ny, p.y, (m + 1) * p.ldy);
        // v := its deviations from the mean (layer); the reciprocal deviations
        auto stats = [&](int kind, float (&rstd)[ROWS]) {
            float s[ROWS];
            if (kind == TGC_NORM_LAYER) {
#pragma unroll
                for (int rr = 0; rr < ROWS; ++rr) {
                    L t = every<L>(0.0f);
#pragma unroll
                    for (int k = 0; k < NV; ++k)
#pragma unroll
                        for (int i = 0; i < NP; ++i) t = add(t, v[rr][k][i]);
                    s[rr] = total(t);
                }
                team_sum(s, smem, &buf);
#pragma unroll
                for (int rr = 0; rr < ROWS; ++rr) {
                    const L mean = every<L>(-s[rr] * p.inv_d);
#pragma unroll
                    for (int k = 0; k < NV; ++k)
                        if (c0 + k * step < p.D)
#pragma unroll
                            for (int i = 0; i < NP; ++i) v[rr][k][i] = add(v[rr][k][i], mean);
                }
            }
#pragma unroll
            for (int rr = 0; rr < ROWS; ++rr) {
                L t = every<L>(0.0f);
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int i = 0; i < NP; ++i) t = fma(v[rr][k][i], v[rr][k][i], t);
                s[rr] = total(t);
            }
            team_sum(s, smem, &buf);
#pragma unroll
            for (int rr = 0; rr < ROWS; ++rr) rstd[rr] = rsqrtf(s[rr] * p.inv_d + p.eps);
        };
        auto affine = [&](L (&x)[NV][NP], float scale, const void *w, const P (&pw)[NV], const void *b, const auto &pb) {
            const L sc = every<L>(scale);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
#pragma unroll
                for (int i = 0; i < NP; ++i) x[k][i] = mul(x[k][i], sc);
                if (w != nullptr)
#pragma unroll
                    for (int i = 0; i < NP; ++i) x[k][i] = mul(x[k][i], pw[k].get(i));
                if constexpr (BIAS) {
                    if (b != nullptr)
#pragma unroll
                        for (int i = 0; i < NP; ++i) x[k][i] = add(x[k][i], pb[k].get(i));
                }
            }
        };
        float rstd[ROWS];
        if (p.post != TGC_NORM_NONE) stats(p.post, rstd);
        const L cs = every<L>(p.branch_scale), rs = every<L>(p.res_scale);
#pragma unroll
        for (int rr = 0; rr < ROWS; ++rr) {
            if (ROWS > 1 && m + rr >= m1) break;
            if (p.gate != nullptr && (m + rr) / p.rows_per_gate != seg) {
                seg = (m + rr) / p.rows_per_gate;
                fetch(g, p.gate, (int64_t)seg * p.D);
            }
            if (p.post != TGC_NORM_NONE) affine(v[rr], rstd[rr], p.post_w, w1, p.post_b, b1);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = c0 + k * step;
#pragma unroll
                for (int i = 0; i < NP; ++i) v[rr][k][i] = mul(v[rr][k][i], cs);
                if (p.gate != nullptr)
#pragma unroll
                    for (int i = 0; i < NP; ++i) v[rr][k][i] = mul(v[rr][k][i], g[k].get(i));
                if (p.x != nullptr) {
                    P px;
                    if constexpr (STAGED)
                        px = *reinterpret_cast<const P *>(here + (rr * 2 + 1) * row_bytes + c * (int)sizeof(T));
                    else px = nx[k];
#pragma unroll
                    for (int i = 0; i < NP; ++i) v[rr][k][i] = fma(px.get(i), rs, v[rr][k][i]);
                }
                if (c >= p.D)
#pragma unroll
                    for (int i = 0; i < NP; ++i) v[rr][k][i] = every<L>(0.0f);
                else if (p.r != nullptr) store_pack<T, VEC>(p.r, (m + rr) * p.ldr + c, v[rr][k]);
            }
        }
        if constexpr (!STAGED)
            if (m + 1 < m1) fetch(nx, p.x, (m + 1) * p.ldx);
        if (p.pre != TGC_NORM_NONE) stats(p.pre, rstd);
        else if (STAGED && blockDim.y == 1) __syncthreads();
        if constexpr (STAGED) {
            // past the sum (or the barrier) every thread has read this stage
            __syncwarp();
            if (threadIdx.x == 0 && *dead == 0) ask(m + 2 * ROWS, (int)stage);
        }
        if (p.pre == TGC_NORM_NONE) continue;
#pragma unroll
        for (int rr = 0; rr < ROWS; ++rr) {
            if (ROWS > 1 && m + rr >= m1) break;
            affine(v[rr], rstd[rr], p.pre_w, w2, p.pre_b, b2);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (c0 + k * step < p.D) store_pack<T, VEC>(p.h, (m + rr) * p.ldh + c0 + k * step, v[rr][k]);
        }
    }
    if (STAGED && threadIdx.x == 0) drain_rows(bar, dead);
}

// ---------------------------------------------------------------- backward

// Rows are dealt in units: a unit is up to unit_rows consecutive rows that share a gate
// vector.  A worker (a team) takes units worker, worker + workers, ... and keeps the sums over a unit's
// rows in registers.  They leave as fp32
// partials that norm_sum_kernel adds in a fixed order.
//
// One reduction a row (two with a layer norm, which takes the means first).  Written out, with
// r and y already without their means, q = dh w_pre, b = c g w_post and t = dr + R (q - s1 - r R s0),
// R and Y the reciprocal deviations, every mean the gradients need is one of
//   r r, y y, q r,  b y dr, b y q, b y r   and for layer norms  q, b y, b dr, b q, b r, b
// summed over the row, so all are taken in one pass and the rest is arithmetic on them:
//   s0 = R mean(q r), s1 = mean(q) (layer)
//   e0 = mean(b t yhat) = Y (mean(b y dr) + R (mean(b y q) - s1 mean(b y) - s0 R mean(b y r)))
//   e1 = mean(b t)      = mean(b dr) + R (mean(b q) - s1 mean(b) - s0 R mean(b r))   (layer)
//   dy = Y (b t - e1 - y Y e0)
// The sums over rows need only S = sum c t yhat and T = sum c t of a unit: dgate = w_post S + b_post T,
// and the unit adds g S and g T to dpost_weight and dpost_bias.
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
    int *fault;
};

// FULL: layer norms or sums for biases.  A thread that holds one vector of a row (NV = 1) keeps
// the columns' factors in registers and, unless FULL, works on two rows at a time: one reduction
// serves both and their arithmetic overlaps.  Wider rows read the factors from shared memory.
template <typename T, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(kBwdMax<VEC, NV>) norm_bwd_kernel(const NormBwdParams p) {
    using P = Pack<T, VEC>;
    using L = typename P::L;
    constexpr int NP = VEC > 1 ? VEC / 2 : 1;
    constexpr bool REGS = NV == 1;
    constexpr int ROWS = kBwdRows<NV, FULL>;
    constexpr int NQ = FULL ? 12 : 6;        // sums a row
    constexpr int NS = FULL || ROWS == 2 ? 16 : 8;
    constexpr bool STAGED = kStaged<VEC, NV>, LEAN = kLean<VEC, NV>;
    // Vectors of each input in registers at a time.
    constexpr int HELD = LEAN ? (VEC == 1 ? 8 : FULL ? 1 : 2) : NV;
    __shared__ alignas(16) float smem[2][NS][32];
    __shared__ float means[2][2][32];
    __shared__ uint64_t bars[4][2];
    __shared__ uint32_t deads[4];
    // A team's own: the columns' factors in fp32 (w_pre, and b of the unit being worked on), unless
    // in registers; then, where rows are staged, two stages of ROWS rows of r, dh, y and dr.
    extern __shared__ __align__(16) float dynamic[];
    int buf = 0, mbuf = 0;
    const int worker = blockIdx.x * blockDim.y + threadIdx.y;
    if (blockDim.y == 1) {
        for (int i = threadIdx.x; i < 2 * NS * 32; i += blockDim.x) (&smem[0][0][0])[i] = 0.0f;
        __syncthreads();
    }
    stream_wait();
    stream_release();
    if (worker >= p.workers) return;
    const int c0 = threadIdx.x * VEC, step = blockDim.x * VEC;
    const int row_bytes = step * NV * (int)sizeof(T);  // of a stage: the row's, rounded up to the team's columns
    float *const fw = dynamic + threadIdx.y * ((REGS ? 0 : 2 * step * NV) + (STAGED ? 2 * ROWS * row_bytes : 0));
    float *const fb = fw + (REGS ? 0 : step * NV);
    uint8_t *const stages = reinterpret_cast<uint8_t *>(fb + (REGS ? 0 : step * NV));
    uint64_t *const bar = bars[threadIdx.y];
    volatile uint32_t *const dead = &deads[threadIdx.y];
    L a_s[NV][NP], a_pre[NV][NP], a_t[FULL ? NV : 1][NP], a_preb[FULL ? NV : 1][NP];
    L rw[NP], rb[NP];  // the factors, where they are in registers
    auto clear = [](auto &a) {
#pragma unroll
        for (auto &k : a)
#pragma unroll
            for (L &f : k) f = every<L>(0.0f);
    };
    clear(a_pre);
    clear(a_preb);
    const bool pre = p.pre != TGC_NORM_NONE, post = p.post != TGC_NORM_NONE;
#pragma unroll
    for (int i = 0; i < NP; ++i) rw[i] = rb[i] = every<L>(0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = c0 + k * step;
        if (c >= p.D) continue;
        P pw;
        L w[NP];
        if (p.pre_w != nullptr) pw = load_pack<T, VEC>(p.pre_w, c);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            w[i] = p.pre_w != nullptr ? pw.get(i) : every<L>(1.0f);
            if constexpr (REGS) rw[i] = w[i];
        }
        if constexpr (!REGS) write_lanes(fw + c, w);
    }
    auto unit_rows = [&](int unit, int *m0, int *m1) {
        const int seg = unit / p.units_per_gate, part = unit % p.units_per_gate;
        *m0 = seg * p.rows_per_gate + part * p.unit_rows;
        const int seg_end = (seg + 1) * p.rows_per_gate;
        *m1 = *m0 + p.unit_rows < seg_end ? *m0 + p.unit_rows : seg_end;
    };
    const void *const in[4] = {pre ? p.r : nullptr, pre ? p.dh : nullptr, p.need_y ? p.y : nullptr, p.dr};
    const int64_t ld[4] = {p.ldr, p.lddh, p.ldy, p.lddr};
    // The rows to ask for, in the order they are worked on (the asking thread's own walk): up to
    // ROWS of one unit at a time.
    int ask_unit = worker, ask_m = 0, ask_end = 0;
    auto ask = [&](int stage) {
        if (ask_unit >= p.units) return;
        const int rows = ask_end - ask_m < ROWS ? ask_end - ask_m : ROWS;
        const uint32_t bytes = (uint32_t)(p.D * (int)sizeof(T));
        uint32_t total = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) total += in[j] != nullptr ? bytes * rows : 0u;
        mbar_arrive_expect_tx(&bar[stage], total);
        for (int r = 0; r < rows; ++r) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in[j] != nullptr)
                    bulk_g2s(stages + ((stage * ROWS + r) * 4 + j) * row_bytes,
                             static_cast<const T *>(in[j]) + (ask_m + r) * ld[j], bytes, &bar[stage]);
        }
        ask_m += rows;
        if (ask_m == ask_end) {
            ask_unit += p.workers;
            if (ask_unit < p.units) unit_rows(ask_unit, &ask_m, &ask_end);
        }
    };
    // Rows that are not staged come from memory, the next ones while the last are worked on where
    // there are registers for them.
    constexpr bool AHEAD = !STAGED && !LEAN;
    P next[4][AHEAD ? ROWS : 1][AHEAD ? NV : 1];
    const T *src[4];  // each input's next row to ask for, at this thread's first column
    bool has[AHEAD ? NV : 1];
    if constexpr (AHEAD) {
#pragma unroll
        for (int k = 0; k < NV; ++k) has[k] = c0 + k * step < p.D;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int rr = 0; rr < ROWS; ++rr)
#pragma unroll
                for (int k = 0; k < NV; ++k) next[j][rr][k].clear();
    }
    auto fetch_next = [&](int left) {  // rows of the unit from src on
        if (left <= 0) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (in[j] == nullptr) continue;
#pragma unroll
            for (int rr = 0; rr < (AHEAD ? ROWS : 1); ++rr) {
                if (rr < left)
#pragma unroll
                    for (int k = 0; k < (AHEAD ? NV : 1); ++k)
                        if (has[k]) next[j][rr][k] = *reinterpret_cast<const P *>(src[j] + k * step);
                src[j] += ld[j];
            }
        }
    };
    if constexpr (STAGED) {
        // an input that is not there reads as zeros
        for (int i = threadIdx.x * 16; i < 8 * ROWS * row_bytes; i += blockDim.x * 16)
            *reinterpret_cast<uint4 *>(stages + i) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_shared();
        if (threadIdx.x == 0) {
            mbar_init(&bar[0], 1);
            mbar_init(&bar[1], 1);
            *dead = 0u;
            fence_mbarrier_init();
        }
        if (blockDim.y == 1) __syncthreads(); else __syncwarp();
        if (threadIdx.x == 0) {
            unit_rows(ask_unit, &ask_m, &ask_end);
            ask(0);
            ask(1);
        }
    }
    uint32_t turn = 0;  // the stage in use and its phase
    for (int unit = worker; unit < p.units; unit += p.workers) {
        const int seg = unit / p.units_per_gate;
        int m0, m1;
        unit_rows(unit, &m0, &m1);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = c0 + k * step;
            if (c >= p.D) continue;
            P pw, pg;
            if (p.post_w != nullptr) pw = load_pack<T, VEC>(p.post_w, c);
            if (p.gate != nullptr) pg = load_pack<T, VEC>(p.gate, (int64_t)seg * p.D + c);
            L f[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                f[i] = every<L>(p.branch_scale);
                if (p.post_w != nullptr) f[i] = mul(f[i], pw.get(i));
                if (p.gate != nullptr) f[i] = mul(f[i], pg.get(i));
                if constexpr (REGS) rb[i] = f[i];
            }
            if constexpr (!REGS) write_lanes(fb + c, f);
        }
        clear(a_s);
        clear(a_t);
        auto factors = [&](int k, L (&w)[NP], L (&b)[NP]) {
            if constexpr (REGS) {
#pragma unroll
                for (int i = 0; i < NP; ++i) { w[i] = rw[i]; b[i] = rb[i]; }
            } else {
                read_lanes(fw + c0 + k * step, w);
                read_lanes(fb + c0 + k * step, b);
            }
        };
        if constexpr (AHEAD) {
#pragma unroll
            for (int j = 0; j < 4; ++j) src[j] = static_cast<const T *>(in[j]) + m0 * ld[j] + c0;
            fetch_next(m1 - m0);
        }
        for (int m = m0; m < m1; m += ROWS) {
            const uint32_t stage = turn & 1u;
            P pr[ROWS][HELD], pd[ROWS][HELD], py[ROWS][HELD], pt[ROWS][HELD];
            if constexpr (STAGED) row_wait(bar, turn, dead, p.fault);
            auto fetch = [&](P (&to)[HELD], int rr, int j, int k0) {
#pragma unroll
                for (int k = 0; k < HELD; ++k) {
                    const int c = c0 + (k0 + k) * step;
                    if constexpr (STAGED)
                        to[k] = *reinterpret_cast<const P *>(stages + ((stage * ROWS + rr) * 4 + j) * row_bytes +
                                                             c * (int)sizeof(T));
                    else if constexpr (AHEAD) to[k] = next[j][rr][k];
                    else if (in[j] != nullptr && c < p.D) to[k] = load_pack<T, VEC>(in[j], (m + rr) * ld[j] + c);
                    else to[k].clear();
                }
            };
#pragma unroll
            for (int rr = 0; rr < ROWS; ++rr) {
                if (LEAN) break;
                fetch(pr[rr], rr, 0, 0);
                fetch(pd[rr], rr, 1, 0);
                fetch(py[rr], rr, 2, 0);
                fetch(pt[rr], rr, 3, 0);
            }
            // LEAN: the next HELD vectors of the row, or of r and y alone
            auto refill = [&](int k, bool all) {
                if (!LEAN || k % HELD != 0) return;
                fetch(pr[0], 0, 0, k);
                fetch(py[0], 0, 2, k);
                if (!all) return;
                fetch(pd[0], 0, 1, k);
                fetch(pt[0], 0, 3, k);
            };
            if constexpr (AHEAD) fetch_next(m1 - m - ROWS);
            L mean_r = every<L>(0.0f), mean_y = every<L>(0.0f);  // negated
            if constexpr (FULL) {
                if (p.pre == TGC_NORM_LAYER || p.post == TGC_NORM_LAYER) {
                    L t0 = every<L>(0.0f), t1 = every<L>(0.0f);
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        refill(k, false);
#pragma unroll
                        for (int i = 0; i < NP; ++i) {
                            t0 = add(t0, pr[0][k % HELD].get(i));
                            t1 = add(t1, py[0][k % HELD].get(i));
                        }
                    }
                    float s[2] = {total(t0), total(t1)};
                    team_sum(s, means, &mbuf);
                    if (p.pre == TGC_NORM_LAYER) mean_r = every<L>(-s[0] * p.inv_d);
                    if (p.post == TGC_NORM_LAYER) mean_y = every<L>(-s[1] * p.inv_d);
                }
            }
            float s[NS] = {};
#pragma unroll
            for (int rr = 0; rr < ROWS; ++rr) {
                L sl[NQ];
#pragma unroll
                for (L &x : sl) x = every<L>(0.0f);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    refill(k, true);
                    if (c0 + k * step >= p.D) continue;
                    L w[NP], b[NP];
                    factors(k, w, b);
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        L r = pr[rr][k % HELD].get(i), y = py[rr][k % HELD].get(i);
                        if (FULL) { r = add(r, mean_r); y = add(y, mean_y); }
                        const L q = mul(pd[rr][k % HELD].get(i), w[i]), d = pt[rr][k % HELD].get(i), by = mul(b[i], y);
                        sl[0] = fma(r, r, sl[0]);
                        sl[1] = fma(y, y, sl[1]);
                        sl[2] = fma(q, r, sl[2]);
                        sl[3] = fma(by, d, sl[3]);
                        sl[4] = fma(by, q, sl[4]);
                        sl[5] = fma(by, r, sl[5]);
                        if constexpr (FULL) {
                            sl[6] = add(sl[6], q);
                            sl[7] = add(sl[7], by);
                            sl[8] = fma(b[i], d, sl[8]);
                            sl[9] = fma(b[i], q, sl[9]);
                            sl[10] = fma(b[i], r, sl[10]);
                            sl[11] = add(sl[11], b[i]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < NQ; ++i) s[rr * (NS / ROWS) + i] = total(sl[i]);
            }
            team_sum_many(s, smem, &buf);
            if constexpr (STAGED) {
                // Past the sum every thread has its part of these rows in registers: the stage is free.
                __syncwarp();
                if (threadIdx.x == 0 && *dead == 0) ask((int)stage);
                ++turn;
            }
#pragma unroll
            for (int rr = 0; rr < ROWS; ++rr) {
                if (ROWS > 1 && m + rr >= m1) break;
                const float *const t0 = s + rr * (NS / ROWS);
                const float R = pre ? rsqrtf(t0[0] * p.inv_d + p.eps) : 0.0f;
                const float Y = post ? rsqrtf(t0[1] * p.inv_d + p.eps) : 1.0f;
                const float s0 = R * t0[2] * p.inv_d;  // mean(q rhat)
                float s1 = 0.0f, e0 = 0.0f, e1 = 0.0f;
                if constexpr (FULL) {
                    if (p.pre == TGC_NORM_LAYER) s1 = t0[6] * p.inv_d;
                    if (post) e0 = Y * p.inv_d * (t0[3] + R * (t0[4] - s1 * t0[7] - s0 * R * t0[5]));
                    if (p.post == TGC_NORM_LAYER) e1 = p.inv_d * (t0[8] + R * (t0[9] - s1 * t0[11] - s0 * R * t0[10]));
                } else {
                    if (post) e0 = Y * p.inv_d * (t0[3] + R * (t0[4] - s0 * R * t0[5]));
                }
                // t = dr + R q - (R s1) - (R s0) rhat;  dy = Y b t - (Y e1) - (Y e0) yhat
                const L lR = every<L>(R), lY = every<L>(Y), k_r = every<L>(-R * s0), k_y = every<L>(-Y * e0);
                const L l1 = every<L>(-R * s1), le = every<L>(-Y * e1), rs = every<L>(p.res_scale);
                // Without a post norm y is no part of dy, not even times zero: it may be infinite.
                auto columns = [&](auto with_post) {
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        if constexpr (!LEAN) {
                            pr[rr][k].forget(); pd[rr][k].forget(); py[rr][k].forget(); pt[rr][k].forget();
                        }
                        refill(k, true);
                        const int c = c0 + k * step;
                        if (c >= p.D) continue;
                        L w[NP], b[NP], ox[NP], oy[NP];
                        factors(k, w, b);
#pragma unroll
                        for (int i = 0; i < NP; ++i) {
                            L r = pr[rr][k % HELD].get(i), y = py[rr][k % HELD].get(i);
                            if (FULL) { r = add(r, mean_r); y = add(y, mean_y); }
                            const L rh = mul(lR, r), yh = mul(lY, y), dh = pd[rr][k % HELD].get(i);
                            L t = fma(lR, mul(dh, w[i]), fma(k_r, rh, pt[rr][k % HELD].get(i)));
                            if (FULL) t = add(t, l1);
                            ox[i] = mul(rs, t);
                            a_s[k][i] = fma(t, yh, a_s[k][i]);
                            a_pre[k][i] = fma(dh, rh, a_pre[k][i]);
                            oy[i] = decltype(with_post)::value ? fma(mul(lY, b[i]), t, mul(k_y, yh)) : mul(b[i], t);
                            if constexpr (FULL) {
                                oy[i] = add(oy[i], le);
                                a_t[k][i] = add(a_t[k][i], t);
                                a_preb[k][i] = add(a_preb[k][i], dh);
                            }
                        }
                        if (p.dx != nullptr) store_pack<T, VEC>(p.dx, (m + rr) * p.lddx + c, ox);
                        if (p.dy != nullptr) store_pack<T, VEC>(p.dy, (m + rr) * p.lddy + c, oy);
                    }
                };
                if (post) columns(std::true_type{}); else columns(std::false_type{});
            }
        }
        // The unit's share of the gate's and the post norm's gradients; the latter gather in the
        // worker's own rows of the partials.
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = c0 + k * step;
            if (c >= p.D) continue;
            P pw, pb, pg;
            if (p.post_w != nullptr) pw = load_pack<T, VEC>(p.post_w, c);
            if (p.post_b != nullptr) pb = load_pack<T, VEC>(p.post_b, c);
            if (p.gate != nullptr) pg = load_pack<T, VEC>(p.gate, (int64_t)seg * p.D + c);
            L dg[NP], gs[NP], gt[NP];
            const L cs = every<L>(p.branch_scale);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const L S = mul(cs, a_s[k][i]);
                dg[i] = p.post_w != nullptr ? mul(S, pw.get(i)) : S;
                gs[i] = p.gate != nullptr ? mul(S, pg.get(i)) : S;
                if constexpr (FULL) {
                    const L t = mul(cs, a_t[k][i]);
                    if (p.post_b != nullptr) dg[i] = fma(t, pb.get(i), dg[i]);
                    gt[i] = p.gate != nullptr ? mul(t, pg.get(i)) : t;
                }
            }
            auto gather = [&](int which, L (&x)[NP]) {
                if (!p.want[which]) return;
                float *to = p.partial + ((int64_t)which * p.workers + worker) * p.D + c;
                if (unit != worker) {
                    L old[NP];
                    read_lanes(to, old);
#pragma unroll
                    for (int i = 0; i < NP; ++i) x[i] = add(x[i], old[i]);
                }
                write_lanes(to, x);
            };
            gather(0, gs);
            if constexpr (FULL) gather(1, gt);
            if (p.dgate != nullptr) {
                if (p.gate_partial == nullptr) store_pack<T, VEC>(p.dgate, (int64_t)seg * p.D + c, dg);
                else write_lanes(p.gate_partial + (int64_t)unit * p.D + c, dg);
            }
        }
    }
    auto put = [&](int which, const auto &a) {
        if (!p.want[which]) return;
        float *to = p.partial + ((int64_t)which * p.workers + worker) * p.D;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (c0 + k * step < p.D) write_lanes(to + c0 + k * step, a[k]);
    };
    put(2, a_pre);
    if constexpr (FULL) put(3, a_preb);
    if (STAGED && threadIdx.x == 0) drain_rows(bar, dead);
}

// Adds the partials of one output vector: blockIdx.y 0..3 the parameter vectors, then one a gate.
struct NormSumParams {
    const float *partial, *gate_partial;
    void *out[4];
    void *dgate;
    int D, workers, units_per_gate;
};

// 32 columns a block: 8 threads of 4 columns x 32 or 64 lanes over the partials, then the lanes in
// a fixed order.
template <typename T>
__global__ void __launch_bounds__(512) norm_sum_kernel(const NormSumParams p) {
    __shared__ alignas(16) float part[64][36];
    stream_wait();
    stream_release();
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
    const int lanes = blockDim.x / 8, warps = blockDim.x / 32;
    const int q = threadIdx.x % 8, l = threadIdx.x / 8, c = blockIdx.x * 32 + q * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (p.D % 4 == 0) {
        if (c < p.D) {
#pragma unroll 8
            for (int i = l; i < n; i += lanes) {
                const float4 f = *reinterpret_cast<const float4 *>(from + (int64_t)i * p.D + c);
                s.x += f.x; s.y += f.y; s.z += f.z; s.w += f.w;
            }
        }
    } else {
#pragma unroll 4
        for (int i = l; i < n; i += lanes) {
            const float *f = from + (int64_t)i * p.D + c;
            if (c < p.D) s.x += f[0];
            if (c + 1 < p.D) s.y += f[1];
            if (c + 2 < p.D) s.z += f[2];
            if (c + 3 < p.D) s.w += f[3];
        }
    }
    *reinterpret_cast<float4 *>(&part[l][q * 4]) = s;
    __syncthreads();
    for (int col = threadIdx.x / 32; col < 32; col += warps) {
        const int lane = threadIdx.x % 32;
        float t = part[lane][col] + (lanes > 32 ? part[lane + 32][col] : 0.0f);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) t += __shfl_xor_sync(0xffffffffu, t, d);
        if (lane == 0 && blockIdx.x * 32 + col < p.D) to[blockIdx.x * 32 + col] = from_f32<T>(t);
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

// Threads a team and vectors a thread for rows of D, the fewest vectors that a team of 512 covers the
// row with.  Forward: 1, 2 or 4 vectors or 1, 4, 8 or 16 single elements, the last of each with
// teams of up to 1024 where 512 do not cover the row.  Backward, whose threads keep sums too: up to
// 8 vectors or 32 elements, no team above 512.
struct TeamShape {
    int vec, nv, team, teams;  // teams a block
    int per_sm;                // teams an SM holds, from the kernel's register budget
};
static TeamShape team_shape(int64_t D, int es, bool vec, bool backward) {
    TeamShape s{};
    s.vec = vec && D * es % 16 == 0 ? 16 / es : 1;
    const int64_t n = (D + s.vec - 1) / s.vec;
    const int steps[2][5] = {{1, 4, 8, 16, 32}, {1, 2, 4, 8, 8}};
    const int last = s.vec > 1 ? (backward ? 8 : 4) : backward ? 32 : 16;
    for (const int nv : steps[s.vec > 1]) {
        s.nv = nv;
        if (nv == last || n <= (int64_t)nv * 512) break;
    }
    s.team = (int)((n + s.nv - 1) / s.nv + 31) / 32 * 32;
    s.teams = s.team == 32 ? 4 : 1;
    int threads;
    if (backward) threads = s.vec == 1 && s.nv == 4 ? 640 : 512;
    else threads = s.nv == 1 || (s.vec == 1 && s.nv == 16) || (es == 4 && s.nv == 4 && s.vec > 1) ? 1024 : 512;
    s.per_sm = threads / s.team;
    return s;
}

constexpr int kMaxTeam = 512;  // threads of a block that has dynamic shared memory, at most

// Lets a kernel have the dynamic shared memory that its widest rows take, once per device.  The limit
// belongs to the kernel, not to a call: were it this call's size, another host thread's narrower rows
// could lower it before this call's launch.
template <auto KERNEL, int BYTES>
static int allow_smem() {
    static std::atomic<bool> done[64];
    if (BYTES <= 40 * 1024) return TGC_OK;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return TGC_OK;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 64) done[dev].store(true, std::memory_order_release);
    return TGC_OK;
}

template <typename T, int V, int NV, bool BIAS, bool STAGED>
static int launch_norm_form(const NormParams &p, dim3 grid, dim3 block, cudaStream_t stream) {
    constexpr int kThread = STAGED ? V * NV * 4 * kFwdRows<NV> * (int)sizeof(T) : 0;  // two stages of y and x
    const int rc = allow_smem<norm_kernel<T, V, NV, BIAS, STAGED>, kMaxTeam * kThread>();
    if (rc != TGC_OK) return rc;
    const cudaError_t e = launch_overlapped(norm_kernel<T, V, NV, BIAS, STAGED>, grid, block,
                                            (size_t)(block.x * block.y) * kThread, 1, stream, p);
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
}

template <typename T, int V, int NV, bool STAGED>
static int launch_norm_nv(const NormParams &p, bool bias, dim3 grid, dim3 block, cudaStream_t stream) {
    if constexpr (STAGED)
        if (p.M <= p.workers) return launch_norm_nv<T, V, NV, false>(p, bias, grid, block, stream);
    return bias ? launch_norm_form<T, V, NV, true, STAGED>(p, grid, block, stream)
                : launch_norm_form<T, V, NV, false, STAGED>(p, grid, block, stream);
}

template <typename T>
static int launch_norm(const NormParams &p, const TeamShape &s, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const dim3 block(s.team, s.teams), grid((unsigned)((p.workers + s.teams - 1) / s.teams));
    const bool bias = p.post_b != nullptr || p.pre_b != nullptr;
    if (s.vec > 1)
        return s.nv == 1   ? launch_norm_nv<T, V, 1, kStaged<V, 1>>(p, bias, grid, block, stream)
               : s.nv == 2 ? launch_norm_nv<T, V, 2, kStaged<V, 2>>(p, bias, grid, block, stream)
                           : launch_norm_nv<T, V, 4, kStaged<V, 4>>(p, bias, grid, block, stream);
    return s.nv == 1   ? launch_norm_nv<T, 1, 1, kStaged<1, 1>>(p, bias, grid, block, stream)
           : s.nv == 4 ? launch_norm_nv<T, 1, 4, kStaged<1, 4>>(p, bias, grid, block, stream)
           : s.nv == 8 ? launch_norm_nv<T, 1, 8, kStaged<1, 8>>(p, bias, grid, block, stream)
                       : launch_norm_nv<T, 1, 16, kStaged<1, 16>>(p, bias, grid, block, stream);
}

#define TGC_TRY(expr)                     \
    do {                                  \
        const int rc_ = (expr);           \
        if (rc_ != TGC_OK) return rc_;    \
    } while (0)

static int norm_impl(tgc_block_norm_args a) {
    const int es = norm_elem(a.dtype);
    if (es == 0) return TGC_ERR_DTYPE;
    if (a.M < 0 || a.M > TGC_MAX_SIZE || a.D < 1 || a.D > TGC_NORM_MAX_D) return TGC_ERR_INVALID_ARG;
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
    const TeamShape s = team_shape(a.D, es, vec, false);
    NormParams p{};
    p.y = a.y; p.x = a.x; p.gate = a.gate;
    p.post_w = a.post_weight; p.post_b = a.post_bias; p.pre_w = a.pre_weight; p.pre_b = a.pre_bias;
    p.r = a.r; p.h = a.h;
    p.M = (int)a.M; p.D = (int)a.D; p.rows_per_gate = a.gate != nullptr ? (int)(a.M / a.gates) : (int)a.M;
    p.ldy = a.ldy; p.ldx = a.ldx; p.ldr = a.ldr; p.ldh = a.ldh;
    p.post = a.post; p.pre = a.pre;
    p.res_scale = a.res_scale; p.branch_scale = a.branch_scale; p.eps = a.eps; p.inv_d = 1.0f / (float)a.D;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const int64_t room = (int64_t)sm_count(dev) * s.per_sm;
    p.workers = (int)(a.M < room ? a.M : room);
    TGC_TRY(device_fault_word(&p.fault));
    return a.dtype == TGC_BF16  ? launch_norm<__nv_bfloat16>(p, s, a.stream)
           : a.dtype == TGC_F16 ? launch_norm<__half>(p, s, a.stream)
                                : launch_norm<float>(p, s, a.stream);
}

// How the backward pass deals its rows: a worker for every team that the card's 152 SMs hold at
// once, units of at least 2 rows, and whole gate segments where there are enough.  It goes by D and
// the type alone, so the workspace's size does not depend on the pointers.  Teams an SM: 16 warps
// where rows come in 16-byte vectors; rows of odd widths, read element by element, take more warps
// and fewer teams fit.
struct NormPlan {
    int segments, rows_per_gate, units_per_gate, unit_rows, units, workers;
    size_t gate_off, total;
};

static NormPlan norm_plan(const tgc_block_norm_bwd_args &a) {
    NormPlan q{};
    const int64_t row = a.D * norm_elem(a.dtype);
    const TeamShape s = team_shape(a.D, norm_elem(a.dtype), true, true);
    const int64_t per_sm = s.vec == 1 ? s.per_sm : row >= 8192 ? 1 : 8192 / row;
    const int64_t target = 152 * (per_sm > 8 ? 8 : per_sm);
    q.segments = a.gate != nullptr ? (int)a.gates : 1;
    q.rows_per_gate = (int)(a.M / q.segments);
    int64_t upg = (target + q.segments - 1) / q.segments;
    const int64_t per_gate = q.rows_per_gate, most = (per_gate + 1) / 2;
    if (upg > most) upg = most;
    q.unit_rows = (int)((per_gate + upg - 1) / upg);
    q.units_per_gate = (int)((per_gate + q.unit_rows - 1) / q.unit_rows);
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
    if (a.M < 0 || a.M > TGC_MAX_SIZE || a.D < 1 || a.D > TGC_NORM_MAX_D) return TGC_ERR_INVALID_ARG;
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

template <typename T, int V, int NV, bool FULL>
static int launch_norm_bwd_form(const NormBwdParams &p, dim3 grid, dim3 block, cudaStream_t stream) {
    // Two fp32 factors a column (128 KiB at the widest row) unless they are in registers, and two
    // stages of four inputs.
    constexpr int kThread = V * NV * ((NV == 1 ? 0 : 8) + (kStaged<V, NV> ? 8 * kBwdRows<NV, FULL> * (int)sizeof(T) : 0));
    const int rc = allow_smem<norm_bwd_kernel<T, V, NV, FULL>, kMaxTeam * kThread>();
    if (rc != TGC_OK) return rc;
    const cudaError_t e = launch_overlapped(norm_bwd_kernel<T, V, NV, FULL>, grid, block,
                                            (size_t)(block.x * block.y) * kThread, 1, stream, p);
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
}

template <typename T, int V, int NV>
static int launch_norm_bwd_nv(const NormBwdParams &p, bool full, dim3 grid, dim3 block, cudaStream_t stream) {
    return full ? launch_norm_bwd_form<T, V, NV, true>(p, grid, block, stream)
                : launch_norm_bwd_form<T, V, NV, false>(p, grid, block, stream);
}

template <typename T>
static int launch_norm_bwd(const NormBwdParams &p, const NormSumParams &q, int nsums, const TeamShape &s, bool full,
                            cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const dim3 block(s.team, s.teams), grid((unsigned)((p.workers + s.teams - 1) / s.teams));
    int rc;
    if (s.vec > 1)
        rc = s.nv == 1 ? launch_norm_bwd_nv<T, V, 1>(p, full, grid, block, stream)
           : s.nv == 2 ? launch_norm_bwd_nv<T, V, 2>(p, full, grid, block, stream)
           : V == 8 || s.nv == 4 ? launch_norm_bwd_nv<T, V, 4>(p, full, grid, block, stream)
                                 : launch_norm_bwd_nv<T, V, V == 8 ? 4 : 8>(p, full, grid, block, stream);
    else
        rc = s.nv == 1 ? launch_norm_bwd_nv<T, 1, 1>(p, full, grid, block, stream)
           : s.nv == 4  ? launch_norm_bwd_nv<T, 1, 4>(p, full, grid, block, stream)
           : s.nv == 8  ? launch_norm_bwd_nv<T, 1, 8>(p, full, grid, block, stream)
           : s.nv == 16 ? launch_norm_bwd_nv<T, 1, 16>(p, full, grid, block, stream)
                        : launch_norm_bwd_nv<T, 1, 32>(p, full, grid, block, stream);
    if (rc != TGC_OK) return rc;
    if (nsums == 0) return TGC_OK;
    const int threads = q.workers > 200 || q.units_per_gate > 200 ? 512 : 256;
    const cudaError_t e = launch_overlapped(norm_sum_kernel<T>, dim3((unsigned)((p.D + 31) / 32), (unsigned)nsums), dim3(threads),
                                            0, 1, stream, q);
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
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
    const TeamShape s = team_shape(a.D, norm_elem(a.dtype), vec, true);
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
    TGC_TRY(device_fault_word(&p.fault));
    NormSumParams n{};
    n.partial = p.partial; n.gate_partial = p.gate_partial; n.dgate = a.dgate;
    for (int i = 0; i < 4; ++i) n.out[i] = outs[i];
    n.D = p.D; n.workers = p.workers; n.units_per_gate = p.units_per_gate;
    const bool sums = outs[0] != nullptr || outs[1] != nullptr || outs[2] != nullptr || outs[3] != nullptr;
    const int nsums = p.gate_partial != nullptr ? 4 + q.segments : sums ? 4 : 0;
    const bool full = outs[1] != nullptr || outs[3] != nullptr || a.post_bias != nullptr || a.post == TGC_NORM_LAYER ||
                      a.pre == TGC_NORM_LAYER;
    return a.dtype == TGC_BF16  ? launch_norm_bwd<__nv_bfloat16>(p, n, nsums, s, full, a.stream)
           : a.dtype == TGC_F16 ? launch_norm_bwd<__half>(p, n, nsums, s, full, a.stream)
                                : launch_norm_bwd<float>(p, n, nsums, s, full, a.stream);
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
