// paged_attention.cu -- tgc_paged_attention: one new token of every sequence over its paged cache.
//
//   x_j = scale q.k_j (capped by c tanh(x / c)),  out = sum_j softmax(x)_j v_j,  lse = log sum_j exp(x_j)
//
// Every key and value is read once and used for the G query heads that share it (once for every 32 of them, 16 with
// more than 128 elements, where G is larger): 4 G flops for 4 bytes, so HBM is the bound up to 8 heads and the design is
// about keeping loads in flight.
//
// A CTA's 4 warps work for themselves: of each unit of keys a warp takes its quarter, or all of its own
// head (a step), copies it with cp.async into its own ring of slots, and keeps its own reference, sum and
// output in registers; where they share an item, they meet at its end.  No barrier in the loop; a page may end anywhere, as each key
// finds its own page.  The copies run ahead of the products across the end of an item, so they do not
// pause while the warps meet.
//
// Products: mma.sync m16n8k16 with keys (then elements of the values) as rows and the heads that share a key
// as columns, padded to 8: scores^T = K Q^T, out^T = V^T P^T.  The scores come out with a key a lane group,
// and movmatrix turns 8 x 8 of them into the second product's operand.  A quarter of an SM takes 8 clocks for one of
// them (21 where the next one needs its sums): 192 for 16 keys of up to 8 heads x 128, whose bytes take HBM 1400 a quarter.
// With 16 and 32 heads neither products nor bytes are the bound, but the chain of scores, softmax and outputs in each of the
// two warps that a quarter has: 64 x up to 4000 tokens, 2 x 16 heads x 128, 42 us (bytes 23): tensor pipe 19 % busy, HBM 49 %,
// issue slots 36 %, and of 5.2 warp cycles an instruction 2.0 for fixed latencies, 1.0 for shared memory, 0.4 for loads; 1 x
// 32 heads 42 us (bytes 11), 2 x 16 x 256 84 (45), where registers run out as well (192 and 124 bytes of spills read).
// The same on tcgen05 -- 128 keys or elements as rows, heads as columns, scores and outputs in TMEM, warps of
// their own for copies, products and softmax -- was built and measured: 66 us there, 98 against 83 with 256
// elements a head, 220 against 126 for 170 sequences of 70 tokens.  A product of 128 rows took 130 clocks there at 16 to 64
// columns, more than the unit needs, so that form was not at its best; it is not kept.
// The probabilities enter the second product as a high and a low 16-bit part: rounding them to
// 16 bits once would add about as much error as rounding the output does.  Both parts lose 2^-17 of a probability at most in
// bf16, 2^-23 in fp16.  A third one leaves the outputs' distance from 64 bits as it is (64 x 8192 tokens: 1.664e-3 of their size with
// two, three and in plain fp32) and costs 1 to 14 % (192.7 -> 194.2 us, 1 x 32 heads 42.4 -> 48.3).
// Probabilities are taken relative to a reference that follows the running maximum by steps (Slack): until the next one
// they grow by up to kOver - kLift powers of two, which costs no bits, and no lane needs another's maximum.  In
// bf16 the reference lies above the maximum, so that no probability passes 1: larger ones take values near fp32's end
// past it.  fp16 has few exponents, so there it stays kLift powers of two below the maximum: what is lost
// beneath fp16's smallest number is then at most 2^-36 of the largest key's weight a key, not 2^-25.
//
// Two ways to deal the work:
//  - runs: the keys of every (sequence, key head) -- an item -- are cut into units; all units of all items
//    lie end to end and every CTA takes an equal run of them, whatever the lengths are.  An item that ends up
//    in several runs is joined by a second kernel from the parts (reference, sum, unnormalised output) that
//    they leave in the workspace; a run leaves two parts at most, so the workspace does not grow with the
//    lengths.
//    An item is a key head, whose keys the 4 warps share, or (own runs) 4 key heads side by side, one a warp: rows 4 times as
//    long for the copies, no meeting of warps, no barrier at all, but 4 times the parts where items are split.
//  - clusters: an item is a cluster's, cut evenly over its CTAs, which join through distributed shared
//    memory: one launch and no workspace, for calls with few and short items (attn_plan says which).
// Both read the lengths on the device.
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

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kMaxCluster = 8;
constexpr float kLn2 = 0.6931471805599453f;

// The item that begins in a run and ends in a later one, `last`; -1: there is none.
struct SplitItem {
    int seq, item, last;
};

struct AttnParams {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *table, *lens;
    KvTable kv;
    int heads_q, heads_k, group, D;
    int row_blocks;  // of a group, R heads each
    int64_t q_s, q_h, o_s, o_h, page_s, token_s, head_s;
    float scale;     // times log2(e) unless capped
    float cap, cap_inv;  // cap log2(e), scale / cap; cap 0: none
    int window;
    int cluster;  // CTAs of a cluster
    int adv_pages, adv_tokens;  // a unit on: pages and places
    // workspace: parts (2 a run, of 4 heads with own runs), and for each item the runs that share it
    float *part_out;   // (2 runs, 1 or 4, R, D)
    float2 *part_ml;   // (2 runs, 1 or 4, R): reference (log2 units), sum
    SplitItem *split;  // (runs)
};

// The keys of sequence s in range: [begin, end).
struct KeyRange {
    int begin, end;
};
__device__ __forceinline__ KeyRange range_of(const AttnParams &p, int len) {
    const int end = p.kv.tokens(len);
    return {p.window > 0 && end > p.window ? end - p.window : 0, end};
}
__device__ __forceinline__ KeyRange key_range(const AttnParams &p, int s) { return range_of(p, p.lens[s]); }
// a / b in 32 bits where both fit: 64-bit divisions take a few hundred cycles each, at every item's start and end.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
template <int UNIT>
__device__ __forceinline__ int units_of(KeyRange r) { return (r.end - r.begin + UNIT - 1) / UNIT; }

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

// An 8 x 8 matrix of 16-bit elements, two in a row a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// A 16-byte chunk's place in a row of a slot: rows of DP elements, chunks of 8 rows turned against one another
// so that ldmatrix, which reads one chunk of 8 rows, meets every bank once.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    return (uint32_t)(row * DP * 2 + ((chunk ^ (row & 7)) << 4));
}

// Powers of two: the reference is set kLift below the maximum, and again when a score passes it by kOver (probabilities up
// to 2^kOver then; fp16 ends at 2^16; bf16 has fp32's exponents below 1, and fp32's sums want 1 above).
template <bool F16>
struct Slack {
    static constexpr float kLift = F16 ? 11.0f : -8.0f, kOver = F16 ? 15.0f : 0.0f;
};

// DP: elements of a head, padded to 64, 128 or 256.  NT: query heads of an item, in eights.
template <int DP, int NT>
struct AttnShape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kKeys = DP == 64 ? 32 : 16;  // of a warp's step
    static constexpr int kUnit = kAttnWarps * kKeys;
    static constexpr int kTile = kKeys * DP * 2;      // bytes of a step's keys (or values)
    // A warp's ring: three slots, of a step's keys and values; with wide heads of either alone (keys, values, keys, ...), so
    // that two CTAs fit an SM: alone, its one warp a quarter waits for each of its own products.
    static constexpr bool kAlone = DP == 256;
    static constexpr int kStages = 3;
    static constexpr int kSlot = kAlone ? kTile : 2 * kTile;
    static constexpr int kWarpRing = kStages * kSlot;
    __device__ static int keys_at(int step) { return (kAlone ? 2 * step : step) % kStages * kSlot; }
    __device__ static int values_at(int step) { return kAlone ? (2 * step + 1) % kStages * kSlot : keys_at(step) + kTile; }
    // The slot that the last of `steps` steps left last: no copy has reached it again.
    __device__ static int last_slot(int steps) { return (kAlone ? 2 * steps + 2 : steps + 2) % kStages; }
    static constexpr int kRings = kAttnWarps * kWarpRing;
    // The queries of three items: one in work, two that the copies may have entered.  They come with the copies, as
    // loads of their own would queue behind those at every item's start (0: no room beside the rings, loads).
    static constexpr int kQueries = (DP == 128 && NT == 4) || (DP == 256 && NT == 2) ? 0 : kRows * DP * 2;
    static constexpr int kSmem = kRings + 3 * kQueries;
    // With a key head a warp: the queries of two items of each warp, as those of the one in work are in registers.
    static constexpr int kOwnSmem = kRings + 2 * kAttnWarps * kRows * DP * 2;
    // Outputs of so many heads fit a slot; more take turns.
    static constexpr int kRound = kRows * DP * 4 <= kSlot ? kRows : kSlot / (DP * 4);
    // Where a CTA of a cluster that took `steps` steps leaves its part of the heads from r0 on: not in the slot where its
    // warps' parts meet.
    __device__ static int cta_part(int steps, int r0) {
        return r0 / kRound * kWarpRing + (last_slot(steps) + 1) % kStages * kSlot;
    }
};

// How the work is dealt: see the top.
enum AttnForm { kRuns, kOwnRuns, kClusters };
// Shapes whose queries fit beside the rings, two CTAs an SM.  Those of 64 elements x 16 heads would: 200 x 1000 tokens of 4 x 16
// heads take 40.3 us so and 40.4, 64 x 4000 38.5 both, 200 x 1000 of 8 x 9 61.2 and 66.7; no instances for it.
template <int DP, int NT>
constexpr bool kOwnFits = DP <= 128 && NT == 1;
static_assert(AttnShape<128, 1>::kOwnSmem <= 112 * 1024 && AttnShape<64, 1>::kOwnSmem <= 112 * 1024, "two CTAs an SM");

static_assert(AttnShape<128, 4>::kRound == 16 && AttnShape<64, 4>::kRound == 32 && AttnShape<256, 2>::kRound == 8, "whole eights");

// Where a run stands: its place in the row of all units, and the item there.
struct RunAt {
    int64_t at, seq_begin;  // units before it; units before its sequence
    int seq, item, unit, units;  // item of the sequence; unit of the item, of so many
    int begin, end;              // keys of the sequence in range
};

// Warp-collective: the sequence that holds unit `at`, looked for from the first on (r is zeroed), then the item and unit.
// False only where the lengths change under the call.
template <int UNIT>
__device__ __forceinline__ bool seek(const AttnParams &p, RunAt &r, int64_t at, int heads, int lane) {
    for (; r.seq < p.kv.num_seqs; r.seq += 32) {
        const int mine = r.seq + lane < p.kv.num_seqs ? units_of<UNIT>(key_range(p, r.seq + lane)) : 0;
        int64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, r.seq_begin + upto * heads > at);
        if (past != 0) {
            const int l = __ffs(past) - 1;
            r.seq += l;
            r.seq_begin += __shfl_sync(0xffffffffu, upto - mine, l) * heads;
            break;
        }
        r.seq_begin += __shfl_sync(0xffffffffu, upto, 31) * heads;
    }
    if (r.seq >= p.kv.num_seqs) return false;
    const KeyRange k = key_range(p, r.seq);
    r.begin = k.begin;
    r.end = k.end;
    r.units = units_of<UNIT>(k);
    r.at = at;
    const int64_t in_seq = at - r.seq_begin;
    if (r.units == 0) return false;
    const int64_t item = quotient(in_seq, r.units);
    if (item >= heads) return false;
    r.item = (int)item;
    r.unit = (int)(in_seq - (int64_t)r.item * r.units);
    return true;
}

// The pair at `local`'s place in CTA `rank` of this cluster.
__device__ __forceinline__ float2 load_cluster(const void *local, int rank) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y) : "r"(mapa_shared(smem_addr(local), (uint32_t)rank)) : "memory");
    return v;
}

__device__ __forceinline__ void store_lse(const AttnParams &p, int seq, int head, float m, float l) {
    if (p.lse != nullptr) p.lse[(int64_t)seq * p.heads_q + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}
template <bool F16>
__device__ __forceinline__ void store_four(const AttnParams &p, int seq, int head, int c, F2 a, F2 b) {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + seq * p.o_s + head * p.o_h + c) =
        make_uint2(pack16(a, F16), pack16(b, F16));
}
// Normalises a row's two neighbouring outputs and stores them.
template <bool F16>
__device__ __forceinline__ void store_out(const AttnParams &p, int seq, int head, int c, float m, float l, float2 o) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + seq * p.o_s + head * p.o_h + c) =
        pack16(f2(o.x * inv, o.y * inv), F16);
    if (c == 0) store_lse(p, seq, head, m, l);
}

template <bool F16, int DP, int NT, AttnForm FORM>
__global__ void __launch_bounds__(kAttnThreads, 2) attention_kernel(const AttnParams p) {
    using S = AttnShape<DP, NT>;
    constexpr bool CLUSTER = FORM == kClusters, OWN = FORM == kOwnRuns;
    constexpr int UNIT = OWN ? S::kKeys : S::kUnit, ITEMS = OWN ? kAttnWarps : 1;  // keys of a unit; key heads (or parts of their groups) of an item
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_sum[kAttnWarps];
    __shared__ uint32_t s_mask[kAttnWarps][S::kStages];
    __shared__ float2 s_ml[kAttnWarps][S::kRows];
    __shared__ float2 s_cta_ml[S::kRows];
    // Sequence, item and units of the items entered last: the products read them at an item's start, when six are at most.
    // Warps that share items all read warp 0's, so that they meet at the same ones.
    constexpr int kItemRing = 8;
    __shared__ int3 s_items[kAttnWarps][kItemRing];
    const int tid = (int)threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t4 = lane & 3;
    uint8_t *const ring = smem + warp * S::kWarpRing;
    const uint32_t ring_at = smem_addr(ring);
    const int chunks = p.D / 8;

    // Products are 16 deep: where D ends inside 16, the rest of the keys' rows has to be zero.
    auto clear_tail = [&](int slot) {
        if (chunks % 2 != 0 && lane < S::kKeys)
            *reinterpret_cast<uint4 *>(ring + slot * S::kSlot + chunk_at<DP>(lane, chunks)) = make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) clear_tail(i);
    stream_wait();
    stream_release();

    // ---- this CTA's run
    const int heads = p.heads_k * p.row_blocks / ITEMS;  // items of a sequence
    int64_t stop = 0, per = 0;                   // end of the run; units of a run
    RunAt r{};                                   // where the copies stand
    int rank = 0, ranks = 1;
    if constexpr (CLUSTER) {
        rank = (int)cluster_ctarank();
        ranks = p.cluster;
        const int all = (int)blockIdx.x / ranks;
        r.seq = all / heads;
        r.item = all % heads;
        const KeyRange k = key_range(p, r.seq);
        r.begin = k.begin;
        r.end = k.end;
        r.units = units_of<UNIT>(k);
        const int each = (r.units + ranks - 1) / ranks;
        r.unit = each * rank < r.units ? each * rank : r.units;
        r.at = r.unit;
        stop = r.unit + each < r.units ? r.unit + each : r.units;
    } else {
        int64_t mine = 0, total = 0;
        for (int s = tid; s < p.kv.num_seqs; s += kAttnThreads) mine += units_of<UNIT>(key_range(p, s));
#pragma unroll
        for (int d = 16; d > 0; d /= 2) mine += __shfl_xor_sync(0xffffffffu, mine, d);
        if (lane == 0) s_sum[warp] = mine;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) total += s_sum[w];
        total *= heads;
        per = quotient(total + gridDim.x - 1, gridDim.x);
        // Sequences without keys: zeros.
        for (int s = (int)blockIdx.x; s < p.kv.num_seqs; s += (int)gridDim.x) {
            if (units_of<UNIT>(key_range(p, s)) != 0) continue;
            for (int i = tid; i < p.heads_q * (p.D / 2); i += kAttnThreads)
                store_out<F16>(p, s, i / (p.D / 2), i % (p.D / 2) * 2, 0.0f, 0.0f, make_float2(0.0f, 0.0f));
        }
        if (tid == 0) p.split[blockIdx.x].last = -1;
        const int run = (int)blockIdx.x;
        if (per * run >= total) return;
        stop = per * (run + 1) < total ? per * (run + 1) : total;
        if (!seek<UNIT>(p, r, per * run, heads, lane)) r.at = stop;
    }

    // ---- the warp's copies: a lane finds the page of a key of the step, all lanes copy.  r runs kAhead units before the
    // copies, across the ends of items, and looks the pages up: a load queues behind the copies under way, about two units'
    // worth.  With wide heads, or 32, a unit's products take longer than that, and there are no registers for more.
    constexpr int kAhead = S::kAlone || NT == 4 ? 1 : 3;
    const int my_key = (OWN ? 0 : warp * S::kKeys) + lane % S::kKeys;
    int key = 0, page_i = 0, look = 0, key_head = 0;  // of the unit to be looked up next, with its place in the page
    int page[kAhead], place[kAhead], head[kAhead];    // of the units to be copied next; head is ~ its number where an item begins
    int entered = 0;     // items that r has entered
    if (lane < kItemRing) s_items[warp][lane] = make_int3(0, 0, 1);
    __syncwarp();
    bool fresh = false;  // nothing of the last one is looked up yet
    auto past = [&](int &at) {
        at += p.adv_tokens;
        const bool over = at >= p.kv.page_size;
        if (over) at -= p.kv.page_size;
        return over;
    };
    auto enter_item = [&] {
        if (lane == 0) s_items[warp][entered % kItemRing] = make_int3(r.seq, r.item, r.units);
        ++entered;
        key = r.begin + r.unit * UNIT + my_key;
        page_i = key / p.kv.page_size;
        look = key - page_i * p.kv.page_size;
        key_head = (OWN ? r.item * ITEMS + warp : r.item) / p.row_blocks;
        fresh = true;
    };
    // The next sequence that has keys; none only where the lengths change under the call.  A lane has the length of one of
    // the next 32: a load here would wait behind the copies.
    int lens_from = r.seq + 1, its_len = 0;
    auto load_lens = [&] { its_len = lens_from + lane < p.kv.num_seqs ? p.lens[lens_from + lane] : 0; };
    if (!CLUSTER) load_lens();
    auto next_seq = [&] {
        while (++r.seq < p.kv.num_seqs) {
            if (r.seq == lens_from + 32) {
                lens_from = r.seq;
                load_lens();
            }
            const KeyRange k = range_of(p, __shfl_sync(0xffffffffu, its_len, r.seq - lens_from));
            r.begin = k.begin;
            r.end = k.end;
            r.units = units_of<UNIT>(k);
            if (r.units > 0) return true;
        }
        return false;
    };
    auto look_up = [&] {
#pragma unroll
        for (int i = 1; i < kAhead; ++i) {
            page[i - 1] = page[i];
            place[i - 1] = place[i];
            head[i - 1] = head[i];
        }
        page[kAhead - 1] = r.at < stop && key < r.end ? p.kv.entry_at(p.table, r.seq, page_i) : -1;  // looked at when it is used: the load is not waited for
        place[kAhead - 1] = look;
        head[kAhead - 1] = fresh ? ~key_head : key_head;
        if (r.at >= stop) return;
        fresh = false;
        key += UNIT;
        page_i += p.adv_pages + (past(look) ? 1 : 0);
        ++r.at;
        if (++r.unit == r.units && !CLUSTER && r.at < stop) {
            r.unit = 0;
            if (++r.item == heads) {
                r.item = 0;
                if (!next_seq()) {
                    r.at = stop;
                    return;
                }
            }
            enter_item();
        }
    };
    RunAt c = r;            // where the products stand
    int64_t copied = r.at;  // units before the one to be copied next
    if (r.at < stop) enter_item();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) look_up();
    if (FORM == kRuns) __syncthreads();
    // An item's queries, a share a warp, with the copies of its first unit: two units ahead of the products, so in the
    // place of an item that all warps are done with.
    constexpr int kQueries = OWN ? S::kRows * DP * 2 : S::kQueries;
    auto queries_of = [&](int item) {  // the item's number in the run
        return smem_addr(smem + S::kRings) + (uint32_t)((OWN ? warp * 2 + item % 2 : item % 3) * kQueries);
    };
    int items = 0;  // whose queries are copied
    auto copy_queries = [&] {
        __syncwarp();
        const int3 it = s_items[warp][items % kItemRing];
        const int item = OWN ? it.y * ITEMS + warp : it.y, head_k = item / p.row_blocks, row0 = item % p.row_blocks * S::kRows;
        const uint32_t to = queries_of(items);
        for (int i = OWN ? lane : tid; i < S::kRows * (DP / 8); i += OWN ? 32 : kAttnThreads) {
            const int row = i / (DP / 8), ch = i % (DP / 8);
            const bool there = row0 + row < p.group && ch < chunks;
            cp_async16(to + chunk_at<DP>(row, ch),
                       static_cast<const uint16_t *>(p.q) + (there ? it.x * p.q_s + (int64_t)(head_k * p.group + row0 + row) * p.q_h + ch * 8 : 0),
                       there);
        }
        ++items;
    };
    int64_t off = -1;  // of this lane's key in the pools, of the unit in work
    auto copy_rows = [&](const void *pool, int to) {
#pragma unroll
        for (int i = 0; i < S::kKeys * (DP / 8) / 32; ++i) {
            const int idx = i * 32 + lane, row = idx / (DP / 8), ch = idx % (DP / 8);
            const int64_t o = __shfl_sync(0xffffffffu, off, row);
            if (ch < chunks)
                cp_async16(ring_at + (uint32_t)to + chunk_at<DP>(row, ch), static_cast<const uint16_t *>(pool) + (o < 0 ? 0 : o + ch * 8), o >= 0);
        }
    };
    auto copy_keys = [&](int unit) {  // the unit's number in the run
        off = -1;
        if (copied < stop) {
            const bool first = head[0] < 0;
            if (kQueries > 0 && first) copy_queries();
            if (p.kv.is_page(page[0])) off = page[0] * p.page_s + place[0] * p.token_s + (first ? ~head[0] : head[0]) * p.head_s;
            const uint32_t have = __ballot_sync(0xffffffffu, off >= 0);
            if (lane == 0) s_mask[warp][unit % S::kStages] = have;
            copy_rows(p.k, S::keys_at(unit));
        }
    };
    auto copy_values = [&](int unit) {  // and on to the next unit
        if (copied >= stop) return;
        copy_rows(p.v, S::values_at(unit));
        ++copied;
        look_up();
    };
    // The copies stay two units ahead (kAlone: a unit's keys and another's values, and the keys after them).
    copy_keys(0);
    if (S::kAlone) cp_async_commit();
    copy_values(0);
    cp_async_commit();
    copy_keys(1);
    if (!S::kAlone) copy_values(1);
    cp_async_commit();
    constexpr int kBehind = S::kAlone ? 2 : 1;  // groups that may be under way while the next one's data are used

    int step = 0, done = 0;  // steps, items
    while (CLUSTER || c.at < stop) {
        if constexpr (!CLUSTER) {
            __syncwarp();
            const int3 it = s_items[OWN ? warp : 0][done % kItemRing];
            c.seq = it.x;
            c.item = it.y;
            c.units = it.z;
        }
        const int my_item = OWN ? c.item * ITEMS + warp : c.item;
        const int head_k = my_item / p.row_blocks, row0 = my_item % p.row_blocks * S::kRows;
        const int rows = p.group - row0 < S::kRows ? p.group - row0 : S::kRows;
        const int head0 = head_k * p.group + row0;
        const int todo = (int)(stop - c.at < c.units - c.unit ? stop - c.at : c.units - c.unit);

        // queries as the first product's right operand: lane (g, t4) has elements 2 t4, 2 t4 + 1 of every 8 of head g
        uint32_t qf[NT][DP / 16][2];
        if constexpr (kQueries > 0) {
            if (CLUSTER && todo <= 0) cp_async_wait<0>();
            else cp_async_wait<kBehind>();
            if constexpr (OWN) __syncwarp();
            else __syncthreads();
            const uint32_t q_at = queries_of(done);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < DP / 32; ++i) {
                    uint32_t a[4];
                    ldmatrix4(a, q_at + chunk_at<DP>(n * 8 + (lane & 7), i * 4 + (lane >> 3)));
                    qf[n][2 * i][0] = a[0];
                    qf[n][2 * i][1] = a[1];
                    qf[n][2 * i + 1][0] = a[2];
                    qf[n][2 * i + 1][1] = a[3];
                }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint16_t *from = static_cast<const uint16_t *>(p.q) + c.seq * p.q_s + (int64_t)(head0 + n * 8 + g) * p.q_h + t4 * 2;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i)
                    qf[n][i / 2][i % 2] = n * 8 + g < rows && i < chunks ? *reinterpret_cast<const uint32_t *>(from + i * 8) : 0u;
            }
        }
        ++done;
        float acc[DP / 16][NT][4];  // elements g and g + 8 of every 16, heads 2 t4 and 2 t4 + 1 of every 8
        float top[NT][2], sum[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < DP / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][n][e] = 0.0f;
            top[n][0] = top[n][1] = -INFINITY;
            sum[n][0] = sum[n][1] = 0.0f;
        }
        for (int left = todo; left > 0; --left, ++step) {
            cp_async_wait<kBehind>();
            __syncwarp();
            const uint32_t k_at = ring_at + (uint32_t)S::keys_at(step), v_at = ring_at + (uint32_t)S::values_at(step);
            const uint32_t have = s_mask[warp][step % S::kStages];
            if (!S::kAlone) {
                copy_keys(step + 2);
                copy_values(step + 2);
                cp_async_commit();
            }

            constexpr int MK = S::kKeys / 16;
            float x[MK][NT][4];  // keys g and g + 8 of every 16
#pragma unroll
            for (int m = 0; m < MK; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[m][n][e] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                if (kk * 2 >= chunks) break;
#pragma unroll
                for (int m = 0; m < MK; ++m) {
                    uint32_t a[4];
                    ldmatrix4(a, k_at + chunk_at<DP>(m * 16 + (lane & 15), kk * 2 + (lane >> 4)));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16<F16>(x[m][n], a, qf[n][kk][0], qf[n][kk][1]);
                }
            }
            if (S::kAlone) {  // the next values in place of these keys
                __syncwarp();
                copy_values(step + 1);
                cp_async_commit();
            }
            if (p.cap > 0.0f) {
#pragma unroll
                for (int m = 0; m < MK; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[m][n][e] = p.cap * tanhf(x[m][n][e] * p.cap_inv);
            } else {
#pragma unroll
                for (int m = 0; m < MK; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[m][n][e] *= p.scale;
            }
            if (have != 0xffffffffu) {
#pragma unroll
                for (int m = 0; m < MK; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (!(have >> (m * 16 + h * 8 + g) & 1u))
#pragma unroll
                            for (int n = 0; n < NT; ++n) x[m][n][2 * h] = x[m][n][2 * h + 1] = -INFINITY;
            }
            // softmax in powers of two
            float big[NT][2];
            bool past = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(x[0][n][e], x[0][n][2 + e]);
                    if (MK == 2) v = fmaxf(v, fmaxf(x[MK - 1][n][e], x[MK - 1][n][2 + e]));
                    big[n][e] = v;
                    past = past || v > top[n][e] + Slack<F16>::kOver;
                }
            if (__any_sync(0xffffffffu, past)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = big[n][e];
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                        v = fmaxf(top[n][e], v - Slack<F16>::kLift);
                        const float f = v == -INFINITY ? 1.0f : exp2_approx(top[n][e] - v);
                        top[n][e] = v;
                        sum[n][e] *= f;
#pragma unroll
                        for (int j = 0; j < DP / 16; ++j) {
                            acc[j][n][e] *= f;
                            acc[j][n][2 + e] *= f;
                        }
                    }
            }
            uint32_t hi[MK][NT][2], lo[MK][NT][2];  // probabilities: keys 0-7 and 8-15 of every 16
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float off0 = top[n][0] == -INFINITY ? 0.0f : top[n][0], off1 = top[n][1] == -INFINITY ? 0.0f : top[n][1];
#pragma unroll
                for (int m = 0; m < MK; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float a = exp2_approx(x[m][n][2 * h] - off0), b = exp2_approx(x[m][n][2 * h + 1] - off1);
                        sum[n][0] += a;
                        sum[n][1] += b;
                        const uint32_t w = pack16(f2(a, b), F16);
                        const float2 back = split(unpack16(w, F16));
                        hi[m][n][h] = transpose8(w);
                        lo[m][n][h] = transpose8(pack16(f2(a - back.x, b - back.y), F16));
                    }
            }
            if (S::kAlone) {
                cp_async_wait<kBehind>();
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) {
                if (j * 2 >= chunks) break;
#pragma unroll
                for (int m = 0; m < MK; ++m) {
                    uint32_t a[4];
                    ldmatrix4_trans(a, v_at + chunk_at<DP>(m * 16 + (lane & 7) + ((lane >> 4) << 3), j * 2 + ((lane >> 3) & 1)));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16<F16>(acc[j][n], a, hi[m][n][0], hi[m][n][1]);
                        mma16<F16>(acc[j][n], a, lo[m][n][0], lo[m][n][1]);
                    }
                }
            }
            if (S::kAlone && left > 1) {  // keys in place of these values; after the item's end, where it is this
                __syncwarp();
                copy_keys(step + 2);
                cp_async_commit();
            }
        }

        // ---- the item's end, in the slot that each warp used last, which its copies have not reached again
        const int last = S::last_slot(step);
        auto part_of = [&](int w) { return reinterpret_cast<float *>(smem + w * S::kWarpRing + last * S::kSlot); };
        // heads' rows of DP; pairs of heads turned against one another, so that a warp's stores meet every bank once
        auto place_of = [](int row, int d) { return row * DP + (d ^ (((row >> 1) & 3) << 3)); };
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = sum[n][e];
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
                if (g == 0) s_ml[warp][n * 8 + t4 * 2 + e] = make_float2(top[n][e], l);
            }
        const int64_t item_begin = c.at - c.unit;  // OWN: a warp's output is whole, and only stored by rows
        const bool whole = CLUSTER ? ranks == 1 : c.unit == 0 && todo == c.units;
        const int part = 2 * (int)blockIdx.x + (c.unit > 0 ? 0 : 1);
        if (!CLUSTER && tid == 0 && c.unit == 0 && !whole)  // the item begins here and goes on in later runs
            p.split[blockIdx.x] = SplitItem{c.seq, c.item, min((int)quotient(item_begin + c.units - 1, per), (int)gridDim.x - 1)};
        if constexpr (OWN) {
            __syncwarp();
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n * 8 + t4 * 2 + (e & 1) < rows)
#pragma unroll
                        for (int j = 0; j < DP / 16; ++j)
                            part_of(warp)[place_of(n * 8 + t4 * 2 + (e & 1), j * 16 + g + (e >> 1) * 8)] = acc[j][n][e];
            __syncwarp();
            for (int i = lane; i < rows * (DP / 4); i += 32) {
                const int row = i / (DP / 4), d = i % (DP / 4) * 4;
                if (d >= p.D) continue;
                const float2 ml = s_ml[warp][row];
                const float4 v = *reinterpret_cast<const float4 *>(part_of(warp) + place_of(row, d));
                if (whole) {
                    const F2 inv = every<F2>(ml.y == 0.0f ? 0.0f : 1.0f / ml.y);
                    if (d == 0) store_lse(p, c.seq, head0 + row, ml.x, ml.y);
                    store_four<F16>(p, c.seq, head0 + row, d, mul(f2(v.x, v.y), inv), mul(f2(v.z, v.w), inv));
                } else {
                    const int64_t at = (int64_t)(part * ITEMS + warp) * S::kRows + row;
                    if (d == 0) p.part_ml[at] = ml;
                    *reinterpret_cast<float4 *>(p.part_out + at * p.D + d) = v;
                }
            }
            __syncwarp();
            clear_tail(last);
            c.at += todo;
            c.unit = 0;
            continue;
        }
#pragma unroll
        for (int r0 = 0; r0 < S::kRows; r0 += S::kRound) {
            __syncwarp();
#pragma unroll
            for (int n = r0 / 8; n < (r0 + S::kRound) / 8; ++n)
#pragma unroll
                for (int j = 0; j < DP / 16; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        part_of(warp)[place_of(n * 8 - r0 + t4 * 2 + (e & 1), j * 16 + g + (e >> 1) * 8)] = acc[j][n][e];
            __syncthreads();
            // a thread takes every kSpan-th four elements of a row: the warps' factors are computed once
            constexpr int kSpan = kAttnThreads / S::kRound;
            const int row = tid / kSpan;
            if (r0 + row < rows) {
                float f[kAttnWarps], m = -INFINITY, l = 0.0f;
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, s_ml[w][r0 + row].x);
                const float off = m == -INFINITY ? 0.0f : m;
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) {
                    const float2 ml = s_ml[w][r0 + row];
                    f[w] = exp2_approx(ml.x - off);
                    l += ml.y * f[w];
                }
                const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
                if (tid % kSpan == 0) {
                    if (whole) store_lse(p, c.seq, head0 + r0 + row, m, l);
                    else if (CLUSTER) s_cta_ml[r0 + row] = make_float2(m, l);
                    else p.part_ml[part * S::kRows + r0 + row] = make_float2(m, l);
                }
#pragma unroll
                for (int d = tid % kSpan * 4; d < DP; d += kSpan * 4) {
                    if (d >= p.D) break;
                    F2 o[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
#pragma unroll
                    for (int w = 0; w < kAttnWarps; ++w) {
                        const float4 v = *reinterpret_cast<const float4 *>(part_of(w) + place_of(row, d));
                        o[0] = fma(f2(v.x, v.y), every<F2>(f[w]), o[0]);
                        o[1] = fma(f2(v.z, v.w), every<F2>(f[w]), o[1]);
                    }
                    if (whole) {
                        store_four<F16>(p, c.seq, head0 + r0 + row, d, mul(o[0], every<F2>(inv)), mul(o[1], every<F2>(inv)));
                    } else {
                        const float2 a = split(o[0]), b = split(o[1]);
                        float *to = CLUSTER ? reinterpret_cast<float *>(smem + S::cta_part(step, r0)) + row * DP + d
                                            : p.part_out + ((int64_t)part * S::kRows + r0 + row) * p.D + d;
                        *reinterpret_cast<float4 *>(to) = make_float4(a.x, a.y, b.x, b.y);
                    }
                }
            }
            __syncthreads();
        }
        if constexpr (CLUSTER) {
            if (ranks > 1) {
                // the CTAs' parts meet: every CTA takes some of the outputs and reads all parts of them
                cluster_sync();
                const int each = (c.units + ranks - 1) / ranks;
                for (int i = rank * kAttnThreads + tid; i < rows * (p.D / 2); i += ranks * kAttnThreads) {
                    const int row = i / (p.D / 2), d = i % (p.D / 2) * 2, r0 = row / S::kRound * S::kRound;
                    float2 ml[kMaxCluster], v[kMaxCluster];
                    float m = -INFINITY;
#pragma unroll
                    for (int q = 0; q < kMaxCluster; ++q) {
                        if (q >= ranks) break;
                        const int before = each * q < c.units ? each * q : c.units;
                        const int steps = c.units - before < each ? c.units - before : each;
                        ml[q] = load_cluster(&s_cta_ml[row], q);
                        v[q] = load_cluster(smem + S::cta_part(steps, r0) + ((row - r0) * DP + d) * 4, q);
                        m = fmaxf(m, ml[q].x);
                    }
                    const float off = m == -INFINITY ? 0.0f : m;
                    float l = 0.0f;
                    float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int q = 0; q < kMaxCluster; ++q) {
                        if (q >= ranks) break;
                        const float f = exp2_approx(ml[q].x - off);
                        l += ml[q].y * f;
                        o.x += v[q].x * f;
                        o.y += v[q].y * f;
                    }
                    store_out<F16>(p, c.seq, head0 + row, d, m, l, o);
                }
                cluster_sync();  // no CTA ends while another may still read its part
            }
            return;
        }
        clear_tail(last);
        if (S::kAlone) {
            __syncwarp();
            copy_keys(step + 1);
            cp_async_commit();
        }
        c.at += todo;
        c.unit = 0;
    }
    cp_async_wait<0>();
}

// Joins the items that several runs share: a block for each run that such an item begins in (at most one does) and
// kJoinRows of its heads.  kJoinWarps warps a head take parts in turn, kJoinDeep at a time, with a maximum of their own,
// and meet in shared memory.
constexpr int kJoinRows = 2;
constexpr int kJoinWarps = 4;
constexpr int kJoinThreads = kJoinRows * kJoinWarps * 32;
constexpr int kJoinDeep = 4;

template <bool F16, int VEC>  // VEC: float2 a lane, 1, 2 or 4 for D up to 64, 128 or 256
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnParams p, const int part_rows, const int own) {
    __shared__ float2 s_ml[kJoinRows][kJoinWarps];
    __shared__ float2 s_out[kJoinRows][kJoinWarps][VEC * 32];
    stream_wait();
    stream_release();
    const SplitItem it = p.split[blockIdx.x];
    if (it.last < 0) return;
    const int first = (int)blockIdx.x, last = it.last;
    const int mine = (int)threadIdx.x / (kJoinWarps * 32), tid = (int)threadIdx.x % (kJoinWarps * 32);
    const int warp = tid / 32, lane = tid % 32;
    // kOwnRuns: an item is `own` of what is one elsewhere
    const int item = it.item * own + (int)blockIdx.z;
    const int row0 = item % p.row_blocks * part_rows, row = (int)blockIdx.y * kJoinRows + mine;
    const bool live = row < part_rows && row0 + row < p.group;
    const int seq = it.seq, head = item / p.row_blocks * p.group + row0 + row;
    float m = -INFINITY, l = 0.0f;
    float2 o[VEC];
#pragma unroll
    for (float2 &v : o) v = make_float2(0.0f, 0.0f);
    for (int i = first + warp; i <= last && live; i += kJoinWarps * kJoinDeep) {
        float2 ml[kJoinDeep], v[kJoinDeep][VEC];
#pragma unroll
        for (int u = 0; u < kJoinDeep; ++u) {
            const int run = i + u * kJoinWarps;
            ml[u] = make_float2(-INFINITY, 0.0f);
            if (run > last) continue;
            // the first run's part is in its second place, the others' in their first
            const int64_t at = ((int64_t)(2 * run + (run == first ? 1 : 0)) * own + (int)blockIdx.z) * part_rows + row;
            ml[u] = p.part_ml[at];
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if ((j * 32 + lane) * 2 < p.D) v[u][j] = *reinterpret_cast<const float2 *>(p.part_out + at * p.D + (j * 32 + lane) * 2);
        }
        float now = m;
#pragma unroll
        for (int u = 0; u < kJoinDeep; ++u) now = fmaxf(now, ml[u].x);
        const float off = now == -INFINITY ? 0.0f : now, f = exp2_approx(m - off);
        m = now;
        l *= f;
#pragma unroll
        for (float2 &w : o) w.x *= f, w.y *= f;
#pragma unroll
        for (int u = 0; u < kJoinDeep; ++u) {
            if (i + u * kJoinWarps > last) continue;
            const float g = exp2_approx(ml[u].x - off);
            l += ml[u].y * g;
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if ((j * 32 + lane) * 2 < p.D) o[j].x += v[u][j].x * g, o[j].y += v[u][j].y * g;
        }
    }
    if (lane == 0) s_ml[mine][warp] = make_float2(m, l);
#pragma unroll
    for (int j = 0; j < VEC; ++j) s_out[mine][warp][j * 32 + lane] = o[j];
    __syncthreads();
    if (!live || tid * 2 >= p.D) return;
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_ml[mine][w].x);
    const float off = m == -INFINITY ? 0.0f : m;
    float2 sum = make_float2(0.0f, 0.0f);
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = exp2_approx(s_ml[mine][w].x - off);
        l += s_ml[mine][w].y * f;
        sum.x += s_out[mine][w][tid].x * f;
        sum.y += s_out[mine][w][tid].y * f;
    }
    store_out<F16>(p, seq, head, 2 * tid, m, l, sum);
}

// ---------------------------------------------------------------- host

#define TGC_TRY(expr)                     \
    do {                                  \
        const int rc_ = (expr);           \
        if (rc_ != TGC_OK) return rc_;    \
    } while (0)

static float attn_scale(const tgc_paged_attention_args &a) { return a.scale != 0.0f ? a.scale : 1.0f / std::sqrt((float)a.D); }

static int attn_check(tgc_paged_attention_args &a) {
    if (a.dtype != TGC_BF16 && a.dtype != TGC_F16) return TGC_ERR_DTYPE;
    if (a.num_seqs < 0 || a.heads_q < 1 || a.heads_k < 1 || a.heads_q % a.heads_k != 0 || a.D < 1 ||
        a.D > TGC_ATTENTION_MAX_D)
        return TGC_ERR_INVALID_ARG;
    if (a.heads_q > TGC_ATTENTION_MAX_HEADS || (a.num_seqs > 0 && a.heads_q > TGC_MAX_SIZE / a.num_seqs)) return TGC_ERR_INVALID_ARG;
    if (a.window < 0 || !std::isfinite(a.scale) || !std::isfinite(a.softcap) || a.softcap < 0.0f) return TGC_ERR_INVALID_ARG;
    // The kernel's factors: an infinite one meets zeros, and a ratio below fp32's normal range has lost bits.
    if (!std::isfinite(attn_scale(a) * kLog2e)) return TGC_ERR_INVALID_ARG;
    if (a.softcap > 0.0f && (!std::isfinite(a.softcap * kLog2e) || !std::isnormal(attn_scale(a) / a.softcap))) return TGC_ERR_INVALID_ARG;
    TGC_TRY(kv_table_check(a.num_pages, a.page_size, a.num_seqs, a.max_pages, &a.table_ld));
    TGC_TRY(kv_pages_check(a.num_pages, a.page_size, a.heads_k, a.D, &a.page_s, &a.token_s, &a.head_s));
    TGC_TRY(heads_check(a.num_seqs, a.heads_q, a.D, &a.q_s, &a.q_h));
    TGC_TRY(heads_check(a.num_seqs, a.heads_q, a.D, &a.o_s, &a.o_h));
    return TGC_OK;
}

struct AttnPlan {
    int dp, nt, row_blocks, unit, grid, cluster;  // cluster: 0 where the work is dealt in runs
    int own;                                      // key heads of an item of kOwnRuns, 1 otherwise
    int64_t items;
    size_t ml_off, split_off, total;
};

// Heads of an item, in eights: as many as share a key, up to 32 (16 for D > 128, whose outputs take twice the
// registers).
// Clusters where the items' CTAs are all resident at once, a CTA has at most kClusterUnits units of its item and not many
// more than a run would have; runs otherwise.  With 8 heads of 128 x 4 a key, clusters and runs take 5.8 and 7.7 us for
// 200 tokens, 7.6 and 8.4 for 900, 9.6 and 9.3 for 2000, 13.6 and 11.6 for 4000 (8 units where a run has 2), 13.9 and 15.7 for
// 16 x 1000 (8 and 7), 12.0 and 18.3 for 32 x 500.  Runs: one for each of two CTAs an SM, no more than there can be units.
// Own runs where what the four times longer rows and the meetings saved give is more than their four times as many parts
// cost, which grow with the heads that share a key: where items * (most keys + kOwnEnd) is at least kOwnKeys a run and such
// head.  1578 sizes (64 to 128 elements, 1 to 8 heads a key, 16 to 8192 items of up to 200 to 30000 keys, uneven), own against
// shared: 1.06 of the time within a quarter below the line, 0.99 within a third above it, 1.09 under half of it, 0.89 from
// four times it on; 384 items x 200 keys x 8 heads x 128 21.9 us and 15.6, 96 x 3000 x 8 x 64 20.7 and 16.3 (below), 512 x 1500 x 1 x 128
// 43.4 and 48.1, 256 x 24000 x 8 x 64 138 and 149 (above).  Keys past kOwnMost do not count: a table that is much wider
// than its lengths would pass with any.
constexpr int kClusterUnits = 16, kClusterBehind = 3;
constexpr int64_t kOwnEnd = 1500, kOwnMost = 16384, kOwnKeys = 900;

static AttnPlan attn_plan(const tgc_paged_attention_args &a, int sms) {
    AttnPlan q{};
    q.own = 1;
    const int64_t group = a.heads_q / a.heads_k;
    q.dp = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
    q.unit = q.dp == 64 ? AttnShape<64, 1>::kUnit : AttnShape<128, 1>::kUnit;
    q.nt = group <= 8 ? 1 : group <= 16 || q.dp == 256 ? 2 : 4;
    q.row_blocks = (int)((group + 8 * q.nt - 1) / (8 * q.nt));
    q.items = a.num_seqs * a.heads_k * q.row_blocks;
    int64_t most = a.max_pages * a.page_size;
    if (a.window > 0 && most > a.window) most = a.window;
    const int64_t units = (most + q.unit - 1) / q.unit, room = (int64_t)sms * 2;
    int c = 1;
    while (c < kMaxCluster && 2 * c * q.items <= room && c < units) c *= 2;
    const int64_t each = (units + c - 1) / c;
    if (c * q.items <= room && each <= kClusterUnits && each - (q.items * units + room - 1) / room <= kClusterBehind) {
        q.cluster = c;
        q.grid = (int)(c * q.items);
        return q;
    }
    const int64_t runs = q.items * units;
    q.grid = (int)(runs < 1 ? 1 : runs < room ? runs : room);
    if (q.dp <= 128 && q.nt == 1 && a.heads_k % kAttnWarps == 0 &&
        q.items * (std::min(most, kOwnMost) + kOwnEnd) >= room * kOwnKeys * group) {
        q.own = kAttnWarps;
        q.unit /= kAttnWarps;
    }
    auto up = [](size_t v) { return (v + 127) / 128 * 128; };
    const size_t rows = (size_t)2 * q.grid * q.own * 8 * q.nt;
    q.ml_off = up(rows * (size_t)a.D * 4);
    q.split_off = q.ml_off + up(rows * 8);
    q.total = q.split_off + up((size_t)q.grid * sizeof(SplitItem));
    return q;
}

template <bool F16, int DP, int NT, AttnForm FORM>
static int launch_attention_form(const AttnParams &p, const AttnPlan &q, cudaStream_t stream) {
    using S = AttnShape<DP, NT>;
    constexpr int kSmem = FORM == kOwnRuns ? S::kOwnSmem : S::kSmem;
    TGC_TRY((allow_smem<attention_kernel<F16, DP, NT, FORM>, kSmem>()));
    cudaError_t e = launch_overlapped(attention_kernel<F16, DP, NT, FORM>, dim3((unsigned)q.grid), dim3(kAttnThreads),
                                      (size_t)kSmem, FORM == kClusters ? q.cluster : 1, stream, p);
    if (e == cudaSuccess && FORM != kClusters)
        e = launch_overlapped(attention_join_kernel<F16, DP / 64>,
                              dim3((unsigned)q.grid, (unsigned)((std::min(p.group, S::kRows) + kJoinRows - 1) / kJoinRows), (unsigned)q.own),
                              dim3(kJoinThreads), 0, 1, stream, p, S::kRows, q.own);
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
}

template <bool F16, int DP, int NT>
static int launch_attention(const AttnParams &p, const AttnPlan &q, cudaStream_t stream) {
    if (q.cluster > 0) return launch_attention_form<F16, DP, NT, kClusters>(p, q, stream);
    if constexpr (kOwnFits<DP, NT>)
        if (q.own > 1) return launch_attention_form<F16, DP, NT, kOwnRuns>(p, q, stream);
    return launch_attention_form<F16, DP, NT, kRuns>(p, q, stream);
}

static int attn_impl(tgc_paged_attention_args a) {
    TGC_TRY(attn_check(a));
    if (a.num_seqs == 0) return TGC_OK;
    if (a.q == nullptr || a.out == nullptr || a.lens == nullptr) return TGC_ERR_INVALID_ARG;
    if (a.max_pages > 0 && a.table == nullptr) return TGC_ERR_INVALID_ARG;  // read whatever the pool holds
    if (a.max_pages > 0 && a.num_pages > 0 && (a.k_pages == nullptr || a.v_pages == nullptr)) return TGC_ERR_INVALID_ARG;
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
    if (q.total > 0) {
        if (a.workspace == nullptr || a.workspace_bytes < q.total) return TGC_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(a.workspace) % 128 != 0) return TGC_ERR_ALIGN;
    }
    AttnParams p{};
    p.q = a.q; p.k = a.k_pages; p.v = a.v_pages; p.out = a.out; p.lse = a.lse; p.table = a.table; p.lens = a.lens;
    p.kv = KvTable{(int)a.num_pages, (int)a.page_size, (int)a.num_seqs, (int)a.max_pages, a.table_ld};
    p.heads_q = (int)a.heads_q; p.heads_k = (int)a.heads_k; p.group = (int)(a.heads_q / a.heads_k); p.D = (int)a.D;
    p.row_blocks = q.row_blocks;
    p.q_s = a.q_s; p.q_h = a.q_h; p.o_s = a.o_s; p.o_h = a.o_h;
    p.page_s = a.page_s; p.token_s = a.token_s; p.head_s = a.head_s;
    const float scale = attn_scale(a);
    p.scale = scale * kLog2e;
    if (a.softcap > 0.0f) {
        p.cap = a.softcap * kLog2e;
        p.cap_inv = scale / a.softcap;
    }
    p.window = a.window > TGC_MAX_SIZE ? 0 : (int)a.window;
    p.cluster = q.cluster;
    p.adv_pages = q.unit / (int)a.page_size;
    p.adv_tokens = q.unit % (int)a.page_size;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    p.part_out = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + q.ml_off);
    p.split = reinterpret_cast<SplitItem *>(ws + q.split_off);
    auto go = [&](auto f16) {
        constexpr bool F16 = decltype(f16)::value;
        auto heads = [&](auto dp) {
            constexpr int DP = decltype(dp)::value;
            if (q.nt == 1) return launch_attention<F16, DP, 1>(p, q, a.stream);
            if constexpr (DP < 256)
                if (q.nt == 4) return launch_attention<F16, DP, 4>(p, q, a.stream);
            return launch_attention<F16, DP, 2>(p, q, a.stream);
        };
        return q.dp == 64    ? heads(std::integral_constant<int, 64>{})
               : q.dp == 128 ? heads(std::integral_constant<int, 128>{})
                             : heads(std::integral_constant<int, 256>{});
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
