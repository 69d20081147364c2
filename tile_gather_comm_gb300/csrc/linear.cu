// linear.cu -- tgc_linear and tgc_linear_bwd: matrix products with bias, activation and
// residual in the epilogue, dense or grouped by expert, and their gradients.
//
//   forward   z = x w^T + b, y = act(z) + residual
//   backward  dz = dy act'(z), dx = dz w, dw = dz^T x, db = sum of dz over rows
#include <cstdint>

#include <cuda_runtime.h>

#include "act.cuh"
#include "groups.cuh"
#include "internal.h"
#include "linear_gemm.cuh"

namespace tgc {

__device__ int g_async_fault;

int device_fault_word(int **word) {
    void *p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_async_fault);
    if (e != cudaSuccess) return cuda_fail(e);
    *word = static_cast<int *>(p);
    return TGC_OK;
}

static bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---------------------------------------------------------------- dz and the bias gradient

// dz = dy act'(z) and, in the same pass, the column sums of each chunk of kChunk rows (chunks
// never cross a group): a block takes a strip of 32 vectors of 8 columns, 8 row lanes, each lane
// 8 rows a chunk with all its loads under way before the first is used.
// dz is rounded to the operands' 16 bits because the tensor cores take no wider type at their rate: the
// gradients' error against 64 bits goes from 1.7e-3 to 2.3e-3 of the norm in bf16 (2.1e-4 to 2.9e-4 in f16)
// against dz in fp32, which two products of a high and a low part would cost twice the time for.  The
// bias gradient sums the unrounded values.
// Bound by memory: dy and z read once, dz written once, partial sums M/kChunk x N fp32.
// Measured: 8192 x 14336 bf16 gelu 104 us with the bias gradient (705 MB, the copy rate).
constexpr int kChunk = 64;

struct DzParams {
    const void *dy, *z;
    void *dz;        // null: not stored (dy is the products' operand)
    float *partial;  // null: no bias gradient
    int M, N, ngroups;
    int64_t lddy, ldz;
    int act;
    const int32_t *offsets;
};

template <bool F16>
__global__ void __launch_bounds__(256) dz_kernel(const DzParams p) {
    __shared__ float sums[8][32 * 8 + 8];
    __shared__ int s_rows[2];
    stream_wait();
    stream_release();
    const int strips = (p.N + 255) / 256;
    const int strip = (int)(blockIdx.x % (unsigned)strips), chunk = (int)(blockIdx.x / (unsigned)strips);
    const int cv = threadIdx.x % 32, rl = threadIdx.x / 32;
    const int n = (strip * 32 + cv) * 8;
    int r0 = chunk * kChunk, r1 = r0 + kChunk < p.M ? r0 + kChunk : p.M;
    if (p.offsets != nullptr) {
        if (threadIdx.x < 32) {
            int idx = 0;
            const int e = find_group_tile(p.offsets, p.ngroups, p.M, kChunk, chunk, threadIdx.x, &idx);
            if (threadIdx.x == 0) {
                const RowRange g = e >= 0 ? group_range(p.offsets, e, p.M) : RowRange{0, 0};
                const int a = g.begin + idx * kChunk;
                s_rows[0] = a;
                s_rows[1] = a + kChunk < g.end ? a + kChunk : g.end;
            }
        }
        __syncthreads();
        r0 = s_rows[0];
        r1 = s_rows[1];
        if (r0 >= r1) return;
    }
    F2 acc[4];
#pragma unroll
    for (F2 &v : acc) v = every<F2>(0.0f);
    if (n < p.N) {
        constexpr int U = 4;  // rows of a lane in flight
        const uint16_t *dy = static_cast<const uint16_t *>(p.dy) + n, *z = static_cast<const uint16_t *>(p.z) + n;
        uint16_t *dz = static_cast<uint16_t *>(p.dz) + n;
        with_act(p.act, [&](auto act) {
            for (int m = r0 + rl; m < r1; m += 8 * U) {
                uint4 a[U], b[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t row = m + 8 * u;
                    if (row < r1) {
                        a[u] = *reinterpret_cast<const uint4 *>(dy + row * p.lddy);
                        if (decltype(act)::value != TGC_ACT_NONE) b[u] = *reinterpret_cast<const uint4 *>(z + row * p.ldz);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t row = m + 8 * u;
                    if (row >= r1) continue;
                    const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, bw[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        F2 d = unpack16(aw[i], F16);
                        if (decltype(act)::value != TGC_ACT_NONE)
                            d = mul(d, act_grad_of<decltype(act)::value>(unpack16(bw[i], F16)));
                        acc[i] = add(acc[i], d);
                        o[i] = pack16(d, F16);
                    }
                    if (p.dz != nullptr) *reinterpret_cast<uint4 *>(dz + row * p.N) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        });
    }
    if (p.partial == nullptr) return;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float2 f = split(acc[c]);
        sums[rl][cv * 8 + 2 * c] = f.x;
        sums[rl][cv * 8 + 2 * c + 1] = f.y;
    }
    __syncthreads();
    const int col = threadIdx.x, nn = strip * 256 + col;
    if (nn < p.N) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sums[i][col];
        p.partial[(int64_t)chunk * p.N + nn] = s;
    }
}

// Sums each group's chunks in order: 32 columns x 8 chunk lanes a block, then the lanes in order.
// `listed`: chunks that dz_kernel was launched for.
// 4.7 us for the 32 chunks of 2048 x 14336: a launch's length.
template <typename T>
__global__ void __launch_bounds__(256) bias_sum_kernel(const float *partial, T *db, int M, int N, const int32_t *offsets,
                                                       int64_t listed, int early) {
    __shared__ float part[8][32];
    if (!early) stream_wait();
    stream_release();
    const int e = blockIdx.y;
    int64_t first = 0;  // this group's first chunk
    if (offsets != nullptr) {
        unsigned long long mine = 0;  // groups that overlap can have more chunks than 32 bits count
        for (int i = threadIdx.x; i < e; i += 256) {
            const RowRange g = group_range(offsets, i, M);
            mine += (unsigned)((g.end - g.begin + kChunk - 1) / kChunk);
        }
        __shared__ unsigned long long s_first;
        if (threadIdx.x == 0) s_first = 0;
        __syncthreads();
        atomicAdd(&s_first, mine);  // integers: the order does not matter
        __syncthreads();
        first = (int64_t)s_first;
    }
    const RowRange g = group_range(offsets, e, M);
    const int chunks = listed_tiles(first, (g.end - g.begin + kChunk - 1) / kChunk, listed);
    const int c = threadIdx.x % 32, l = threadIdx.x / 32, n = blockIdx.x * 32 + c;
    float s = 0.0f;
    if (n < N)
        for (int k = l; k < chunks; k += 8) s += partial[(first + k) * N + n];
    part[l][c] = s;
    __syncthreads();
    if (l == 0 && n < N) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][c];
        db[(int64_t)e * N + n] = from_f32<T>(s);
    }
    if (early) stream_wait();
}

// ---------------------------------------------------------------- checks

static int check_common(tgc_dtype dtype, tgc_act act, int64_t M, int64_t K, int64_t N, const int32_t *offsets,
                        int ngroups) {
    if (M < 0 || K < 0 || N < 0) return TGC_ERR_INVALID_ARG;
    if (M > TGC_MAX_SIZE || K > TGC_MAX_SIZE || N > TGC_MAX_SIZE) return TGC_ERR_INVALID_ARG;
    if (dtype != TGC_BF16 && dtype != TGC_F16) return TGC_ERR_DTYPE;
    if (act < TGC_ACT_NONE || act > TGC_ACT_SILU) return TGC_ERR_INVALID_ARG;
    if (offsets == nullptr ? ngroups != 0 : (ngroups < 1 || ngroups > TGC_MAX_GROUPS)) return TGC_ERR_INVALID_ARG;
    if (!aligned(offsets, 4)) return TGC_ERR_ALIGN;
    if (K == 0) return TGC_ERR_INVALID_ARG;
    if (K % 8 != 0 || N % 8 != 0) return TGC_ERR_ALIGN;
    if ((int64_t)(ngroups > 0 ? ngroups : 1) * N >= (int64_t(1) << 31)) return TGC_ERR_INVALID_ARG;
    return TGC_OK;
}

// One (rows, cols) operand: resolves its stride and checks it.  null is fine unless `need`.
static int check_matrix(const void *p, bool need, int64_t rows, int64_t cols, int64_t *ld) {
    if (*ld == 0) *ld = cols;
    if (p == nullptr) return need ? TGC_ERR_INVALID_ARG : TGC_OK;
    if (*ld < cols) return TGC_ERR_INVALID_ARG;
    if (*ld % 8 != 0 || !aligned(p, 16)) return TGC_ERR_ALIGN;
    int64_t bytes = 0;
    if (__builtin_mul_overflow(*ld, rows * 2, &bytes) || bytes >= (int64_t(1) << 62)) return TGC_ERR_INVALID_ARG;
    if (*ld >= (int64_t(1) << 39)) return TGC_ERR_INVALID_ARG;  // a tensor map's row stride ends at 2^40 bytes
    return TGC_OK;
}

static int check_weight_stride(int64_t *w_stride, int64_t N, int64_t ldw, int ngroups) {
    if (*w_stride == 0) *w_stride = N * ldw;
    if (ngroups <= 1) return TGC_OK;
    if (*w_stride < (N - 1) * ldw) return TGC_ERR_INVALID_ARG;
    if (*w_stride % 8 != 0) return TGC_ERR_ALIGN;
    if (*w_stride >= (int64_t(1) << 39)) return TGC_ERR_INVALID_ARG;
    return TGC_OK;
}

#define TGC_TRY(expr)                     \
    do {                                  \
        const int rc_ = (expr);           \
        if (rc_ != TGC_OK) return rc_;    \
    } while (0)

// Fills the defaults of `a` in place; TGC_OK when there may be work.
static int linear_check(tgc_linear_args &a) {
    TGC_TRY(check_common(a.dtype, a.act, a.M, a.K, a.N, a.offsets, a.ngroups));
    if (a.M == 0 || a.N == 0) return TGC_OK;
    TGC_TRY(check_matrix(a.x, true, a.M, a.K, &a.ldx));
    TGC_TRY(check_matrix(a.w, true, a.N, a.K, &a.ldw));
    TGC_TRY(check_matrix(a.y, true, a.M, a.N, &a.ldy));
    TGC_TRY(check_matrix(a.z, false, a.M, a.N, &a.ldz));
    TGC_TRY(check_matrix(a.residual, false, a.M, a.N, &a.ldres));
    if (!aligned(a.bias, 16)) return TGC_ERR_ALIGN;
    TGC_TRY(check_weight_stride(&a.w_stride, a.N, a.ldw, a.ngroups));
    if (a.residual == a.y && a.ldres != a.ldy) return TGC_ERR_INVALID_ARG;
    return TGC_OK;
}

static int linear_impl(tgc_linear_args a) {
    TGC_TRY(linear_check(a));
    if (a.M == 0 || a.N == 0) return TGC_OK;
    const int groups = a.offsets != nullptr ? a.ngroups : 1;
    LinearProduct p{};
    p.a = a.x; p.lda = a.ldx;
    p.b = a.w; p.ldb = a.ldw; p.b_stride = a.w_stride;
    p.M = a.M; p.J = a.N; p.R = a.K;
    p.offsets = a.offsets; p.ngroups = groups;
    p.bias = a.bias; p.residual = a.residual; p.y = a.y; p.z = a.z;
    p.ldres = a.ldres; p.ldy = a.ldy; p.ldz = a.ldz;
    p.act = a.act; p.f16 = a.dtype == TGC_F16;
    return launch_linear(p, kFwd, a.stream);
}

// Workspace of the backward pass: dz (M, N) in `dtype` unless dy serves, then the bias gradient's chunk sums.
struct BwdLayout {
    size_t dz, partial, total;
    int64_t chunks;
};
static BwdLayout bwd_layout(const tgc_linear_bwd_args &a) {
    auto up = [](size_t v) { return (v + 127) / 128 * 128; };
    BwdLayout l{};
    l.chunks = (a.M + kChunk - 1) / kChunk + (a.offsets != nullptr ? a.ngroups : 0);
    const bool dz = a.act != TGC_ACT_NONE && (a.dx != nullptr || a.dw != nullptr);
    l.partial = dz ? up((size_t)a.M * (size_t)a.N * 2) : 0;
    l.total = l.partial + (a.dbias != nullptr ? up((size_t)l.chunks * (size_t)a.N * 4) : 0);
    return l;
}

static int linear_bwd_check(tgc_linear_bwd_args &a) {
    TGC_TRY(check_common(a.dtype, a.act, a.M, a.K, a.N, a.offsets, a.ngroups));
    if (a.N == 0) return TGC_ERR_INVALID_ARG;
    const bool some = a.M > 0;
    TGC_TRY(check_matrix(a.dy, some, a.M, a.N, &a.lddy));
    TGC_TRY(check_matrix(a.z, some && a.act != TGC_ACT_NONE, a.M, a.N, &a.ldz));
    TGC_TRY(check_matrix(a.x, some && a.dw != nullptr, a.M, a.K, &a.ldx));
    TGC_TRY(check_matrix(a.w, some && a.dx != nullptr, a.N, a.K, &a.ldw));
    TGC_TRY(check_matrix(a.dx, false, a.M, a.K, &a.lddx));
    if (!aligned(a.dw, 16) || !aligned(a.dbias, 16)) return TGC_ERR_ALIGN;
    TGC_TRY(check_weight_stride(&a.w_stride, a.N, a.ldw, a.ngroups));
    if (a.M * ((a.N + 255) / 256) / kChunk >= (int64_t(1) << 30)) return TGC_ERR_INVALID_ARG;  // the dz pass's blocks
    int64_t bytes = 0;
    const int groups = a.offsets != nullptr ? a.ngroups : 1;
    if (__builtin_mul_overflow(a.N * groups, a.K * 2, &bytes) || bytes >= (int64_t(1) << 62)) return TGC_ERR_INVALID_ARG;
    return TGC_OK;
}

static int linear_bwd_impl(tgc_linear_bwd_args a) {
    TGC_TRY(linear_bwd_check(a));
    const int groups = a.offsets != nullptr ? a.ngroups : 1;
    if (a.M == 0) {
        cudaError_t e = cudaSuccess;
        if (a.dw != nullptr) e = cudaMemsetAsync(a.dw, 0, (size_t)groups * a.N * a.K * 2, a.stream);
        if (e == cudaSuccess && a.dbias != nullptr) e = cudaMemsetAsync(a.dbias, 0, (size_t)groups * a.N * 2, a.stream);
        return e == cudaSuccess ? TGC_OK : cuda_fail(e);
    }
    const BwdLayout l = bwd_layout(a);
    if (l.total > 0) {
        if (a.workspace == nullptr || a.workspace_bytes < l.total) return TGC_ERR_WORKSPACE;
        if (!aligned(a.workspace, 128)) return TGC_ERR_ALIGN;
    }
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const void *dz = a.dy;
    int64_t lddz = a.lddy;
    if (l.total > 0) {
        DzParams d{};
        d.dy = a.dy; d.z = a.z; d.lddy = a.lddy; d.ldz = a.ldz;
        d.M = (int)a.M; d.N = (int)a.N; d.ngroups = a.ngroups; d.act = a.act; d.offsets = a.offsets;
        if (l.partial > 0) {
            d.dz = ws;
            dz = ws;
            lddz = a.N;
        }
        if (a.dbias != nullptr) d.partial = reinterpret_cast<float *>(ws + l.partial);
        const unsigned grid = (unsigned)((a.N + 255) / 256 * l.chunks);
        const cudaError_t e = launch_overlapped(a.dtype == TGC_BF16 ? dz_kernel<false> : dz_kernel<true>, dim3(grid),
                                                dim3(256), 0, 1, a.stream, d);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    // The kernels from here on need only what is complete when the first of them starts, so the
    // later ones need not wait for the earlier: they fill the SMs that those leave.
    int early = 0;
    LinearProduct p{};
    p.a = dz; p.lda = lddz;
    p.M = a.M; p.J = a.K;
    p.offsets = a.offsets; p.ngroups = groups;
    p.f16 = a.dtype == TGC_F16;
    if (a.dx != nullptr) {
        p.b = a.w; p.ldb = a.ldw; p.b_stride = a.w_stride;
        p.R = a.N;
        p.y = a.dx; p.ldy = a.lddx;
        TGC_TRY(launch_linear(p, kDgrad, a.stream));
        early = 1;
    }
    if (a.dw != nullptr) {
        p.b = a.x; p.ldb = a.ldx; p.b_stride = 0;
        p.I = a.N; p.R = 0;
        p.y = a.dw; p.ldy = a.K;
        p.early = early;
        TGC_TRY(launch_linear(p, kWgrad, a.stream));
        early = 1;
    }
    if (a.dbias != nullptr) {
        const float *partial = reinterpret_cast<const float *>(ws + l.partial);
        const dim3 grid((unsigned)((a.N + 31) / 32), (unsigned)groups);
        const cudaError_t e =
            a.dtype == TGC_BF16
                ? launch_overlapped(bias_sum_kernel<__nv_bfloat16>, grid, dim3(256), 0, 1, a.stream, partial,
                                    static_cast<__nv_bfloat16 *>(a.dbias), (int)a.M, (int)a.N, a.offsets, l.chunks, early)
                : launch_overlapped(bias_sum_kernel<__half>, grid, dim3(256), 0, 1, a.stream, partial,
                                    static_cast<__half *>(a.dbias), (int)a.M, (int)a.N, a.offsets, l.chunks, early);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return TGC_OK;
}

}  // namespace tgc

extern "C" int tgc_async_status(cudaStream_t stream) {
    int *word = nullptr, status = 0;
    const int rc = tgc::device_fault_word(&word);
    if (rc != TGC_OK) return rc;
    cudaError_t e = cudaMemcpyAsync(&status, word, sizeof status, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof status, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    return e == cudaSuccess ? status : tgc::cuda_fail(e);
}

extern "C" int tgc_linear(const tgc_linear_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::linear_impl(*args);
}

extern "C" int tgc_linear_bwd(const tgc_linear_bwd_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::linear_bwd_impl(*args);
}

extern "C" size_t tgc_linear_bwd_workspace_bytes(const tgc_linear_bwd_args *args) {
    if (args == nullptr) return 0;
    tgc_linear_bwd_args a = *args;
    if (tgc::linear_bwd_check(a) != TGC_OK || a.M == 0) return 0;
    return tgc::bwd_layout(a).total;
}
