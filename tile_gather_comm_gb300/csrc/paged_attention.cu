// paged_attention.cu -- tgc_paged_attention: one new token of every sequence over its paged cache.
//
//   x_j = scale q.k_j (capped by c tanh(x / c)),  out = sum_j softmax(x)_j v_j,  lse = log sum_j exp(x_j)
//
// Every key and value is read once and used for the G query heads that share it: 4 G flops for 4
// bytes, so HBM is the bound and the design is about keeping loads in flight.
//
// Split: the keys of every (sequence, key head) -- an item -- are cut into units of 64 keys; all units of
// all items lie end to end and every CTA takes an equal run of them, whatever the lengths are.  An
// item that ends up in several CTAs is joined by a second kernel from the parts (maximum, sum,
// unnormalised output) that they leave in the workspace; a CTA leaves two parts at most, so the
// workspace does not grow with the lengths.  The lengths are read on the device.
//
// A CTA's 4 warps work for themselves: of each unit a warp takes 16 keys, copies them with cp.async into
// its own ring of stages, and keeps its own running maximum, sum and output in registers; they
// meet at the item's end.  No barrier in the loop, and a page may end anywhere, as each key finds its
// own page.
//
// Products: mma.sync m16n8k16, the heads that share a key (padded to 16) as rows.  One new token has
// 1 to 16 rows; tcgen05 takes 64 or 128 at least, and its scores would go through TMEM to the
// registers that need them here.  The bound is HBM, not the products.
// The probabilities enter the second product as a high and a low 16-bit part: rounding them to
// 16 bits once would add about as much error as rounding the output does.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "act.cuh"
#include "internal.h"
#include "kv.cuh"
#include "prims.cuh"

namespace tgc {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kStep = 16;                     // keys of a warp's step
constexpr int kUnit = kAttnWarps * kStep;     // keys of a unit
constexpr int kMinUnits = 4;                  // units of a CTA at least: shorter runs cost more in joining than they save
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *table, *lens;
    KvTable kv;
    int heads_q, heads_k, group, D;
    int row_blocks;  // of a group, R rows each
    int64_t q_s, q_h, o_s, o_h, page_s, token_s, head_s;
    float scale;     // times log2(e) unless capped
    float cap, cap_inv;  // cap log2(e), scale / cap; cap 0: none
    int window;
    int adv_pages, adv_tokens;  // kUnit keys on: pages and places
    // workspace: parts (2 a CTA), and for each item the CTAs that share it
    float *part_out;   // (2 grid, R, D)
    float2 *part_ml;   // (2 grid, R): maximum (log2 units), sum
    int2 *shared_by;   // (items): first and last CTA; (-1, -1): one alone
};

// The keys of sequence s in range: [begin, end).
struct KeyRange {
    int begin, end;
};
__device__ __forceinline__ KeyRange key_range(const AttnParams &p, int s) {
    const int end = p.kv.tokens(p.lens[s]);
    return {p.window > 0 && end > p.window ? end - p.window : 0, end};
}
__device__ __forceinline__ int units_of(KeyRange r) { return (r.end - r.begin + kUnit - 1) / kUnit; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    const int bytes = valid ? 16 : 0;  // the rest is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
// c (16 x 8, fp32) += a (16 x 16) b (16 x 8)
template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_approx(float v) {
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v));
    return v;
}

// A 16-byte chunk's place in a row of a stage: rows of DP elements, chunks of 8 rows turned against one another
// so that ldmatrix, which reads one chunk of 8 rows, meets every bank once.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    return (uint32_t)(row * DP * 2 + ((chunk ^ (row & 7)) << 4));
}

template <int DP, int MT>
struct AttnShape {
    static constexpr int kRows = 16 * MT;
    static constexpr int kTile = kStep * DP * 2;      // bytes of a step's keys (or values)
    static constexpr int kStages = DP == 64 ? 6 : DP == 128 ? 3 : 3;
    static constexpr int kQBytes = kRows * DP * 2;
    static constexpr int kRing = kAttnWarps * kStages * 2 * kTile;
    static constexpr int kJoin = kAttnWarps * kRows * (DP + 2) * 4;  // the warps' outputs, in the ring's place
    static constexpr int kSmem = kQBytes + (kRing > kJoin ? kRing : kJoin);
};

// The rows' results: normalised to `out`, or as a part to the workspace.
template <bool F16, int DP, int MT>
__global__ void __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) attention_kernel(const AttnParams p) {
    using S = AttnShape<DP, MT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_scan[kAttnWarps];
    __shared__ int64_t s_before;
    __shared__ int s_seq;
    __shared__ uint32_t s_mask[kAttnWarps][S::kStages];
    const int tid = (int)threadIdx.x, warp = tid / 32, lane = tid % 32;
    uint8_t *q_s = smem, *ring = smem + S::kQBytes;

    // What lies beyond D in the stages stays zero, so it adds nothing to any product.
    if (p.D < DP)
        for (int i = tid; i < S::kRing / 16; i += kAttnThreads) reinterpret_cast<uint4 *>(ring)[i] = make_uint4(0, 0, 0, 0);
    stream_wait();
    stream_release();

    // ---- this CTA's run of units
    const int heads = p.heads_k * p.row_blocks;  // items of a sequence
    const int share = (p.kv.num_seqs + kAttnThreads - 1) / kAttnThreads;
    int64_t mine = 0;
    for (int i = 0; i < share; ++i) {
        const int s = tid * share + i;
        if (s < p.kv.num_seqs) mine += units_of(key_range(p, s));
    }
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    int64_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp) base += s_scan[w];
        total += s_scan[w];
    }
    upto += base;
    total *= heads;
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    if (per < kMinUnits) per = kMinUnits;
    int64_t at = per * blockIdx.x;
    const int64_t stop = at + per < total ? at + per : total;

    // Sequences without keys: zeros.
    for (int s = (int)blockIdx.x; s < p.kv.num_seqs; s += (int)gridDim.x) {
        if (units_of(key_range(p, s)) != 0) continue;
        for (int i = tid; i < p.heads_q * p.D; i += kAttnThreads)
            static_cast<uint16_t *>(p.out)[s * p.o_s + i / p.D * p.o_h + i % p.D] = 0;
        if (p.lse != nullptr)
            for (int i = tid; i < p.heads_q; i += kAttnThreads) p.lse[(int64_t)s * p.heads_q + i] = -INFINITY;
    }
    if (at >= stop) return;

    // The sequence in which the run starts: in the share of the thread whose units hold it.
    if ((upto - mine) * heads <= at && at < upto * heads) {
        int64_t before = upto - mine;
        int s = tid * share;
        for (;; ++s) {
            const int n = units_of(key_range(p, s));
            if (at < (before + n) * heads) break;
            before += n;
        }
        s_seq = s;
        s_before = before * heads;
    }
    __syncthreads();
    int seq = s_seq;
    int64_t seq_begin = s_before;  // global number of the sequence's first unit

    const int chunks = p.D / 8;
    const uint32_t ring_at = smem_addr(ring) + (uint32_t)(warp * S::kStages * 2 * S::kTile);
    const uint32_t q_at = smem_addr(q_s);

    while (at < stop) {
        const KeyRange range = key_range(p, seq);
        const int units = units_of(range);
        if (at >= seq_begin + (int64_t)units * heads) {  // this sequence is done (or has no keys)
            seq_begin += (int64_t)units * heads;
            ++seq;
            continue;
        }
        const int item = (int)((at - seq_begin) / units), unit0 = (int)((at - seq_begin) - (int64_t)item * units);
        const int unit1 = stop - at < units - unit0 ? unit0 + (int)(stop - at) : units;
        const int head_k = item / p.row_blocks, row0 = item % p.row_blocks * S::kRows;
        const int rows = p.group - row0 < S::kRows ? p.group - row0 : S::kRows;
        const int64_t item_begin = seq_begin + (int64_t)item * units;

        // ---- queries to shared memory, rows and columns beyond them zero
        for (int i = tid; i < S::kRows * (DP / 8); i += kAttnThreads) {
            const int r = i / (DP / 8), c = i % (DP / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows && c < chunks)
                v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + seq * p.q_s +
                                                     (int64_t)(head_k * p.group + row0 + r) * p.q_h + c * 8);
            *reinterpret_cast<uint4 *>(q_s + chunk_at<DP>(r, c)) = v;
        }
        __syncthreads();

        // ---- the warp's loads: lane l < 16 finds the page of key l of a step, all lanes copy
        const int steps = unit1 - unit0;
        const uint16_t *kp = static_cast<const uint16_t *>(p.k) + (int64_t)head_k * p.head_s;
        const uint16_t *vp = static_cast<const uint16_t *>(p.v) + (int64_t)head_k * p.head_s;
        int key = range.begin + unit0 * kUnit + warp * kStep + (lane & 15);  // of the step to be issued
        int page_i = key / p.kv.page_size, place = key - page_i * p.kv.page_size;
        auto next_page = [&] { return key < range.end ? p.kv.page_at(p.table, seq, page_i) : -1; };
        int page = next_page();
        auto issue = [&](int step) {
            const int stage = step % S::kStages;
            const int64_t off = page < 0 ? -1 : page * p.page_s + place * p.token_s;
            const uint32_t have = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
            if (lane == 0) s_mask[warp][stage] = have;
            const uint32_t to = ring_at + (uint32_t)(stage * 2 * S::kTile);
#pragma unroll
            for (int i = 0; i < kStep * (DP / 8) / 32; ++i) {
                const int idx = i * 32 + lane, r = idx / (DP / 8), c = idx % (DP / 8);
                const int64_t o = __shfl_sync(0xffffffffu, off, r);
                if (c < chunks) {
                    const int64_t from = o < 0 ? 0 : o + c * 8;
                    cp_async16(to + chunk_at<DP>(r, c), kp + from, o >= 0);
                    cp_async16(to + S::kTile + chunk_at<DP>(r, c), vp + from, o >= 0);
                }
            }
            key += kUnit;
            page_i += p.adv_pages;
            place += p.adv_tokens;
            if (place >= p.kv.page_size) {
                place -= p.kv.page_size;
                ++page_i;
            }
            page = next_page();
        };
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) {
            if (i < steps) issue(i);
            cp_async_commit();
        }

        // ---- the loop
        constexpr bool kQInRegs = DP * MT <= 128;
        uint32_t qf[kQInRegs ? MT : 1][kQInRegs ? DP / 16 : 1][4];
        const uint32_t q_lane = (uint32_t)(lane & 15);
        if constexpr (kQInRegs)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk)
                    ldmatrix4(qf[m][kk], q_at + chunk_at<DP>(m * 16 + (int)q_lane, kk * 2 + (lane >> 4)));
        float acc[MT][DP / 8][4];
        float top[MT][2], sum[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int j = 0; j < DP / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
            top[m][0] = top[m][1] = -INFINITY;
            sum[m][0] = sum[m][1] = 0.0f;
        }
        for (int step = 0; step < steps; ++step) {
            cp_async_wait<S::kStages - 2>();
            __syncwarp();
            const int stage = step % S::kStages;
            const uint32_t k_at = ring_at + (uint32_t)(stage * 2 * S::kTile), v_at = k_at + S::kTile;
            const uint32_t have = s_mask[warp][stage];
            if (step + S::kStages - 1 < steps) issue(step + S::kStages - 1);
            cp_async_commit();

            // scores: two tiles of 16 rows x 8 keys
            float x[MT][2][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[m][j][e] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                uint32_t b[4];  // keys 0-7 and 8-15, each the two halves of 16 elements
                ldmatrix4(b, k_at + chunk_at<DP>((lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if constexpr (kQInRegs) {
                        mma16<F16>(x[m][0], qf[m][kk], b[0], b[1]);
                        mma16<F16>(x[m][1], qf[m][kk], b[2], b[3]);
                    } else {
                        uint32_t a[4];
                        ldmatrix4(a, q_at + chunk_at<DP>(m * 16 + (int)q_lane, kk * 2 + (lane >> 4)));
                        mma16<F16>(x[m][0], a, b[0], b[1]);
                        mma16<F16>(x[m][1], a, b[2], b[3]);
                    }
                }
            }
            // softmax, in powers of two
            uint32_t ph[MT][4], pl[MT][4];  // probabilities as the next product's operand: high and low parts
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (p.cap > 0.0f) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[m][j][e] = p.cap * tanhf(x[m][j][e] * p.cap_inv);
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[m][j][e] *= p.scale;
                }
                if (have != 0xffffu) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(have >> (j * 8 + (lane & 3) * 2 + (e & 1)) & 1u)) x[m][j][e] = -INFINITY;
                }
                float big[2];
                bool rescale = false;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    big[h] = fmaxf(fmaxf(x[m][0][2 * h], x[m][0][2 * h + 1]), fmaxf(x[m][1][2 * h], x[m][1][2 * h + 1]));
                    big[h] = fmaxf(big[h], __shfl_xor_sync(0xffffffffu, big[h], 1));
                    big[h] = fmaxf(big[h], __shfl_xor_sync(0xffffffffu, big[h], 2));
                    rescale = rescale || big[h] > top[m][h];
                }
                if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float now = fmaxf(top[m][h], big[h]);
                        const float f = now == -INFINITY ? 1.0f : exp2_approx(top[m][h] - now);
                        top[m][h] = now;
                        sum[m][h] *= f;
#pragma unroll
                        for (int j = 0; j < DP / 8; ++j) {
                            acc[m][j][2 * h] *= f;
                            acc[m][j][2 * h + 1] *= f;
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float off = top[m][h] == -INFINITY ? 0.0f : top[m][h];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float a = exp2_approx(x[m][j][2 * h] - off), b = exp2_approx(x[m][j][2 * h + 1] - off);
                        sum[m][h] += a + b;
                        const F2 both = f2(a, b);
                        const uint32_t hi = pack16(both, F16);
                        const float2 r = split(unpack16(hi, F16));
                        ph[m][j * 2 + h] = hi;
                        pl[m][j * 2 + h] = pack16(f2(a - r.x, b - r.y), F16);
                    }
                }
            }
            // outputs: 16 keys deep, tiles of 16 rows x 8 elements
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) {
                uint32_t b[4];
                ldmatrix4_trans(b, v_at + chunk_at<DP>(lane & 15, j * 2 + (lane >> 4)));
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mma16<F16>(acc[m][2 * j], ph[m], b[0], b[1]);
                    mma16<F16>(acc[m][2 * j + 1], ph[m], b[2], b[3]);
                    mma16<F16>(acc[m][2 * j], pl[m], b[0], b[1]);
                    mma16<F16>(acc[m][2 * j + 1], pl[m], b[2], b[3]);
                }
            }
        }

        // ---- the warps' parts meet in the ring's place
        cp_async_wait<0>();
        __syncthreads();
        float *w_out = reinterpret_cast<float *>(ring);                         // (warps, rows, DP)
        float2 *w_ml = reinterpret_cast<float2 *>(w_out + kAttnWarps * S::kRows * DP);  // (warps, rows)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float l = sum[m][h];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                const int r = m * 16 + h * 8 + (lane >> 2);
                if ((lane & 3) == 0) w_ml[warp * S::kRows + r] = make_float2(top[m][h], l);
                if (r < rows)
#pragma unroll
                    for (int j = 0; j < DP / 8; ++j)
                        *reinterpret_cast<float2 *>(w_out + (warp * S::kRows + r) * DP + j * 8 + (lane & 3) * 2) =
                            make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
            }
        __syncthreads();
        const int64_t first = item_begin / per, last = (item_begin + units - 1) / per;
        const bool whole = first == last;
        const int part = 2 * (int)blockIdx.x + (item_begin < per * blockIdx.x ? 0 : 1);
        if (tid == 0 && unit0 == 0)
            p.shared_by[(int64_t)seq * heads + item] = whole ? make_int2(-1, -1) : make_int2((int)first, (int)last);
        for (int i = tid; i < rows * (p.D / 2); i += kAttnThreads) {
            const int r = i / (p.D / 2), c = i % (p.D / 2) * 2;
            float2 ml[kAttnWarps];
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                ml[w] = w_ml[w * S::kRows + r];
                m = fmaxf(m, ml[w].x);
            }
            const float off = m == -INFINITY ? 0.0f : m;
            float l = 0.0f;
            float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float f = exp2_approx(ml[w].x - off);
                const float2 v = *reinterpret_cast<const float2 *>(w_out + (w * S::kRows + r) * DP + c);
                l += ml[w].y * f;
                o.x += v.x * f;
                o.y += v.y * f;
            }
            const int head = head_k * p.group + row0 + r;
            if (whole) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + seq * p.o_s + head * p.o_h + c) =
                    pack16(f2(o.x * inv, o.y * inv), F16);
                if (c == 0 && p.lse != nullptr)
                    p.lse[(int64_t)seq * p.heads_q + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float2 *>(p.part_out + ((int64_t)part * S::kRows + r) * p.D + c) = o;
                if (c == 0) p.part_ml[part * S::kRows + r] = make_float2(m, l);
            }
        }
        __syncthreads();
        if (p.D < DP && at + (unit1 - unit0) < stop) {  // zeros again where the parts lay
            for (int i = tid; i < S::kRing / 16; i += kAttnThreads)
                reinterpret_cast<uint4 *>(ring)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
        }
        at += unit1 - unit0;
    }
}

// One block a row (sequence, query head) joins the parts of an item that several CTAs share.
constexpr int kJoinThreads = 128;

template <bool F16>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnParams p, const int part_rows) {
    __shared__ float s_ml[2][kJoinThreads / 32];
    __shared__ float2 s_out[kJoinThreads / 32][TGC_ATTENTION_MAX_D / 2];
    stream_wait();
    stream_release();
    const int head = (int)(blockIdx.x % (unsigned)p.heads_q), seq = (int)(blockIdx.x / (unsigned)p.heads_q);
    const KeyRange range = key_range(p, seq);
    if (range.end == range.begin) return;
    const int heads = p.heads_k * p.row_blocks, in_group = head % p.group;
    const int item = head / p.group * p.row_blocks + in_group / part_rows, row = in_group % part_rows;
    const int2 by = p.shared_by[(int64_t)seq * heads + item];
    if (by.x < 0) return;
    // the first CTA's part is its second place unless the item began in an earlier one, so never here
    const int n = by.y - by.x + 1, tid = (int)threadIdx.x, warp = tid / 32, lane = tid % 32;
    auto part_at = [&](int i) { return (int64_t)(2 * (by.x + i) + (i == 0 ? 1 : 0)) * part_rows + row; };
    float m = -INFINITY;
    for (int i = tid; i < n; i += kJoinThreads) m = fmaxf(m, p.part_ml[part_at(i)].x);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) s_ml[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, s_ml[0][w]);
    const float off = m == -INFINITY ? 0.0f : m;
    // a warp takes every fourth part; a lane pairs of elements 32 apart
    float l = 0.0f;
    float2 o[TGC_ATTENTION_MAX_D / 64];
#pragma unroll
    for (float2 &v : o) v = make_float2(0.0f, 0.0f);
    for (int i = warp; i < n; i += kJoinThreads / 32) {
        const float2 ml = p.part_ml[part_at(i)];
        const float f = exp2_approx(ml.x - off);
        const float *from = p.part_out + part_at(i) * p.D;
        l += ml.y * f;
#pragma unroll
        for (int j = 0; j < TGC_ATTENTION_MAX_D / 64; ++j) {
            const int c = (j * 32 + lane) * 2;
            if (c < p.D) {
                const float2 v = *reinterpret_cast<const float2 *>(from + c);
                o[j].x += v.x * f;
                o[j].y += v.y * f;
            }
        }
    }
    if (lane == 0) s_ml[1][warp] = l;
#pragma unroll
    for (int j = 0; j < TGC_ATTENTION_MAX_D / 64; ++j) s_out[warp][j * 32 + lane] = o[j];
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) l += s_ml[1][w];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int c = tid; c < p.D / 2; c += kJoinThreads) {
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) {
            v.x += s_out[w][c].x;
            v.y += s_out[w][c].y;
        }
        *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + seq * p.o_s + head * p.o_h + 2 * c) =
            pack16(f2(v.x * inv, v.y * inv), F16);
    }
    if (tid == 0 && p.lse != nullptr)
        p.lse[(int64_t)seq * p.heads_q + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- host

#define TGC_TRY(expr)                     \
    do {                                  \
        const int rc_ = (expr);           \
        if (rc_ != TGC_OK) return rc_;    \
    } while (0)

static int attn_check(tgc_paged_attention_args &a) {
    if (a.dtype != TGC_BF16 && a.dtype != TGC_F16) return TGC_ERR_DTYPE;
    if (a.num_seqs < 0 || a.heads_q < 1 || a.heads_k < 1 || a.heads_q % a.heads_k != 0 || a.D < 1 ||
        a.D > TGC_ATTENTION_MAX_D)
        return TGC_ERR_INVALID_ARG;
    if (a.heads_q > TGC_MAX_SIZE || (a.num_seqs > 0 && a.heads_q > TGC_MAX_SIZE / a.num_seqs)) return TGC_ERR_INVALID_ARG;
    if (a.window < 0 || !std::isfinite(a.scale) || !std::isfinite(a.softcap) || a.softcap < 0.0f) return TGC_ERR_INVALID_ARG;
    TGC_TRY(kv_table_check(a.num_pages, a.page_size, a.num_seqs, a.max_pages, &a.table_ld));
    TGC_TRY(kv_pages_check(a.num_pages, a.page_size, a.heads_k, a.D, &a.page_s, &a.token_s, &a.head_s));
    TGC_TRY(heads_check(a.num_seqs, a.heads_q, a.D, &a.q_s, &a.q_h));
    TGC_TRY(heads_check(a.num_seqs, a.heads_q, a.D, &a.o_s, &a.o_h));
    return TGC_OK;
}

struct AttnPlan {
    int dp, mt, row_blocks, grid;
    int64_t items;
    bool join;
    size_t ml_off, shared_off, total;
};

// Rows of an MMA: 16 for up to 16 heads a key head, 32 for more where the registers hold their outputs (D <= 128).
// Grid: two CTAs an SM (one for D > 128), no more than there can be runs of kMinUnits units.
static AttnPlan attn_plan(const tgc_paged_attention_args &a, int sms) {
    AttnPlan q{};
    const int64_t group = a.heads_q / a.heads_k;
    q.dp = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
    q.mt = group > 16 && q.dp <= 128 ? 2 : 1;
    q.row_blocks = (int)((group + 16 * q.mt - 1) / (16 * q.mt));
    q.items = a.num_seqs * a.heads_k * q.row_blocks;
    int64_t most = a.max_pages * a.page_size;
    if (a.window > 0 && most > a.window) most = a.window;
    const int64_t units = (most + kUnit - 1) / kUnit, room = (int64_t)sms * (q.dp <= 128 ? 2 : 1);
    const int64_t runs = units > 0 ? (q.items * units + kMinUnits - 1) / kMinUnits : 1;
    q.grid = (int)(runs < 1 ? 1 : runs < room ? runs : room);
    q.join = q.grid > 1 && units > 1;  // items of one unit are never split
    auto up = [](size_t v) { return (v + 127) / 128 * 128; };
    const size_t rows = (size_t)2 * q.grid * 16 * q.mt;
    q.ml_off = up(rows * (size_t)a.D * 4);
    q.shared_off = q.ml_off + up(rows * 8);
    q.total = q.shared_off + up((size_t)q.items * 8);
    return q;
}

template <bool F16, int DP, int MT>
static int launch_attention(const AttnParams &p, const AttnPlan &q, cudaStream_t stream) {
    using S = AttnShape<DP, MT>;
    TGC_TRY((allow_smem<attention_kernel<F16, DP, MT>, S::kSmem>()));
    cudaError_t e = launch_overlapped(attention_kernel<F16, DP, MT>, dim3((unsigned)q.grid), dim3(kAttnThreads),
                                      (size_t)S::kSmem, 1, stream, p);
    if (e == cudaSuccess && q.join)
        e = launch_overlapped(attention_join_kernel<F16>, dim3((unsigned)(p.kv.num_seqs * p.heads_q)), dim3(kJoinThreads), 0, 1,
                              stream, p, S::kRows);
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
}

static int attn_impl(tgc_paged_attention_args a) {
    TGC_TRY(attn_check(a));
    if (a.num_seqs == 0) return TGC_OK;
    if (a.q == nullptr || a.out == nullptr || a.lens == nullptr) return TGC_ERR_INVALID_ARG;
    if (a.max_pages > 0 && a.num_pages > 0 && (a.table == nullptr || a.k_pages == nullptr || a.v_pages == nullptr))
        return TGC_ERR_INVALID_ARG;
    if (a.q == a.out && ((a.num_seqs > 1 && a.q_s != a.o_s) || (a.heads_q > 1 && a.q_h != a.o_h))) return TGC_ERR_INVALID_ARG;
    uintptr_t bits = 0;
    for (const void *v : {a.q, (const void *)a.out, a.k_pages, a.v_pages}) bits |= reinterpret_cast<uintptr_t>(v);
    for (const int64_t v : {a.D, a.q_s, a.q_h, a.o_s, a.o_h, a.page_s, a.token_s, a.head_s}) bits |= (uintptr_t)v * 2;
    if (bits % 16 != 0) return TGC_ERR_ALIGN;
    bits = 0;
    for (const void *v : {(const void *)a.lse, (const void *)a.table, (const void *)a.lens}) bits |= reinterpret_cast<uintptr_t>(v);
    if (bits % 4 != 0) return TGC_ERR_ALIGN;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const AttnPlan q = attn_plan(a, sm_count(dev));
    if (a.workspace == nullptr || a.workspace_bytes < q.total) return TGC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(a.workspace) % 128 != 0) return TGC_ERR_ALIGN;
    AttnParams p{};
    p.q = a.q; p.k = a.k_pages; p.v = a.v_pages; p.out = a.out; p.lse = a.lse; p.table = a.table; p.lens = a.lens;
    p.kv = KvTable{(int)a.num_pages, (int)a.page_size, (int)a.num_seqs, (int)a.max_pages, a.table_ld};
    p.heads_q = (int)a.heads_q; p.heads_k = (int)a.heads_k; p.group = (int)(a.heads_q / a.heads_k); p.D = (int)a.D;
    p.row_blocks = q.row_blocks;
    p.q_s = a.q_s; p.q_h = a.q_h; p.o_s = a.o_s; p.o_h = a.o_h;
    p.page_s = a.page_s; p.token_s = a.token_s; p.head_s = a.head_s;
    const float scale = a.scale != 0.0f ? a.scale : 1.0f / std::sqrt((float)a.D);
    p.scale = scale * kLog2e;
    if (a.softcap > 0.0f) {
        p.cap = a.softcap * kLog2e;
        p.cap_inv = scale / a.softcap;
    }
    p.window = a.window > TGC_MAX_SIZE ? 0 : (int)a.window;
    p.adv_pages = kUnit / (int)a.page_size;
    p.adv_tokens = kUnit % (int)a.page_size;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    p.part_out = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + q.ml_off);
    p.shared_by = reinterpret_cast<int2 *>(ws + q.shared_off);
    auto go = [&](auto f16) {
        constexpr bool F16 = decltype(f16)::value;
        return q.dp == 64    ? (q.mt == 1 ? launch_attention<F16, 64, 1>(p, q, a.stream) : launch_attention<F16, 64, 2>(p, q, a.stream))
               : q.dp == 128 ? (q.mt == 1 ? launch_attention<F16, 128, 1>(p, q, a.stream) : launch_attention<F16, 128, 2>(p, q, a.stream))
                             : launch_attention<F16, 256, 1>(p, q, a.stream);
    };
    return a.dtype == TGC_F16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace tgc

extern "C" int tgc_paged_attention(const tgc_paged_attention_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::attn_impl(*args);
}

extern "C" size_t tgc_paged_attention_workspace_bytes(const tgc_paged_attention_args *args) {
    if (args == nullptr) return 0;
    tgc_paged_attention_args a = *args;
    if (tgc::attn_check(a) != TGC_OK || a.num_seqs == 0) return 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    return tgc::attn_plan(a, tgc::sm_count(dev)).total;
}
