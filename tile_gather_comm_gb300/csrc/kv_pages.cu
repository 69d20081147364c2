// kv_pages.cu -- upkeep of the paged cache on the device: tgc_kv_copy, tgc_kv_reserve, tgc_kv_fork,
// tgc_kv_free, tgc_kv_compact.
//
// Pages are given out and moved by number, lowest first, so results do not depend on timing: a
// count of each segment of kSegment pages, then every segment ranks its own pages behind the
// counts before it.  No list of free pages is kept between calls: refs says which they are.
#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"
#include "kv.cuh"
#include "prims.cuh"

namespace tgc {

constexpr int kSegment = 2048;     // pages of a block
constexpr int kSegThreads = 256;
constexpr int kSegEach = kSegment / kSegThreads;
constexpr int kListThreads = 1024;

// Workspace, in this order.
struct KvSpace {
    int *count;        // per segment: free pages (reserve, fork) or pages in use (compact)
    int *from, *to;    // pages to copy: per entry (fork) or move (compact); -1: none
    int *have, *len;   // per entry: pages held before, tokens afterwards
    int *flag;         // per entry: 1 where it can be
    int64_t *upto;     // per entry: pages asked for up to and with it
    int *claim;        // per sequence: the first entry that names it
    int *map;          // per page: its move (compact), -1: stays
    int *sums;         // compact: moves, pages in use
    size_t total;
};

static KvSpace kv_space(void *base, int64_t n, int64_t num_pages, int64_t num_seqs) {
    KvSpace w{};
    size_t at = 0;
    auto take = [&](int64_t count, size_t each) {
        uint8_t *p = base == nullptr ? nullptr : static_cast<uint8_t *>(base) + at;
        at += ((size_t)count * each + 127) / 128 * 128;
        return p;
    };
    const int64_t list = n > num_pages / 2 + 1 ? n : num_pages / 2 + 1;
    w.upto = reinterpret_cast<int64_t *>(take(n, 8));
    w.count = reinterpret_cast<int *>(take((num_pages + kSegment - 1) / kSegment, 4));
    w.from = reinterpret_cast<int *>(take(list, 4));
    w.to = reinterpret_cast<int *>(take(list, 4));
    w.have = reinterpret_cast<int *>(take(n, 4));
    w.len = reinterpret_cast<int *>(take(n, 4));
    w.flag = reinterpret_cast<int *>(take(n, 4));
    w.claim = reinterpret_cast<int *>(take(num_seqs, 4));
    w.map = reinterpret_cast<int *>(take(num_pages, 4));
    w.sums = reinterpret_cast<int *>(take(2, 4));
    w.total = at;
    return w;
}

struct KvParams {
    int32_t *refs, *table, *lens;
    KvTable kv;
    const int32_t *src, *dst, *add;
    int32_t *ok, *used;
    int n, segments;
    KvSpace w;
};

// Sum over the block of `v`; every thread gets it.  s: one place a warp.
template <int THREADS>
__device__ __forceinline__ int block_sum(int v, int *s) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();  // the places may still be read from the sum before
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) sum += s[w];
    return sum;
}

// Sum of `v` over the threads before this one; *total over all.
template <int THREADS, typename V>
__device__ __forceinline__ V block_before(V v, V *s, V *total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    V upto = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const V o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    __syncthreads();
    if (lane == 31) s[warp] = upto;
    __syncthreads();
    V base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += s[w];
        all += s[w];
    }
    *total = all;
    return base + upto - v;
}

// The pages of this thread in segment `seg`: bit i set where page seg * kSegment + threadIdx.x * kSegEach + i is in use.
__device__ __forceinline__ unsigned pages_in_use(const KvParams &p, int seg, int *valid) {
    const int first = seg * kSegment + (int)threadIdx.x * kSegEach;
    unsigned bits = 0;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kSegEach; ++i)
        if (first + i < p.kv.num_pages) {
            ++n;
            if (p.refs[first + i] > 0) bits |= 1u << i;
        }
    *valid = n;
    return bits;
}

// The number at `local`'s place in CTA `rank` of this cluster.
__device__ __forceinline__ int read_cluster_int(const int *local, int rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_addr(local), (uint32_t)rank)) : "memory");
    return v;
}

// What each entry of a reserve (FORK = false) or fork asks for.  One block: the first entry that names a
// sequence gets it, whatever the order in which threads run.
template <bool FORK>
__device__ void list_entries(const KvParams &p) {
    __shared__ int64_t s[kListThreads / 32];
    __shared__ int64_t s_base;
    for (int e = threadIdx.x; e < p.n; e += kListThreads)
        if (p.kv.is_seq(p.dst[e])) p.w.claim[p.dst[e]] = p.n;
    if (threadIdx.x == 0) s_base = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < p.n; e += kListThreads)
        if (p.kv.is_seq(p.dst[e])) atomicMin(&p.w.claim[p.dst[e]], e);
    __syncthreads();
    for (int e0 = 0; e0 < p.n; e0 += kListThreads) {
        const int e = e0 + (int)threadIdx.x;
        int64_t need = 0;
        if (e < p.n) {
            const int d = p.dst[e];
            int flag = p.kv.is_seq(d) && *(volatile int *)&p.w.claim[d] == e;
            int have = 0, len = 0;
            if (FORK) {
                const int from = p.src[e];
                flag = flag && p.kv.is_seq(from) && from != d && p.lens[d] == 0;
                if (flag) {
                    len = p.kv.tokens(p.lens[from]);
                    have = len / p.kv.page_size;
                    need = len % p.kv.page_size != 0;
                }
                p.w.from[e] = flag && need ? p.kv.page_at(p.table, from, have) : -1;
                p.w.to[e] = -1;
            } else if (flag) {
                const int add = p.add[e], old = p.kv.tokens(p.lens[d]);
                const int64_t grown = (int64_t)old + add;
                flag = add >= 0 && grown <= (int64_t)p.kv.max_pages * p.kv.page_size;
                if (flag) {
                    len = (int)grown;
                    have = p.kv.pages_of(old);
                    need = p.kv.pages_of(len) - have;
                }
            }
            p.w.flag[e] = flag;
            p.w.have[e] = have;
            p.w.len[e] = len;
        }
        int64_t all = 0;
        const int64_t before = block_before<kListThreads, int64_t>(need, s, &all);
        const int64_t base = s_base;
        if (e < p.n) p.w.upto[e] = base + before + need;
        __syncthreads();
        if (threadIdx.x == 0) s_base = base + all;
        __syncthreads();
    }
}

// One block lists the entries, the others count the free pages of their segments.
template <bool FORK>
__global__ void __launch_bounds__(kListThreads) list_kernel(const KvParams p) {
    __shared__ int s[kListThreads / 32];
    stream_wait();
    stream_release();
    if (blockIdx.x == 0) {
        list_entries<FORK>(p);
        return;
    }
    const int seg = (int)blockIdx.x - 1;
    int free = 0;
    for (int i = (int)threadIdx.x; i < kSegment; i += kListThreads) {
        const int page = seg * kSegment + i;
        free += page < p.kv.num_pages && p.refs[page] <= 0;
    }
    free = block_sum<kListThreads>(free, s);
    if (threadIdx.x == 0) p.w.count[seg] = free;
}

// Hands the free pages out: page of rank r (among the free) is entry e's where e is the first with upto > r.
// Entries are dealt to the blocks for what does not need a page.
template <bool FORK>
__global__ void __launch_bounds__(kSegThreads) grant_kernel(const KvParams p) {
    __shared__ int s[kSegThreads / 32];
    __shared__ int64_t s64[kSegThreads / 32];
    stream_wait();
    stream_release();
    int64_t before = 0, free = 0;
    for (int i = (int)threadIdx.x; i < p.segments; i += kSegThreads) {
        const int c = p.w.count[i];
        free += c;
        if (i < (int)blockIdx.x) before += c;
    }
    int64_t sum = 0;
    block_before<kSegThreads, int64_t>(before, s64, &sum);
    before = sum;
    block_before<kSegThreads, int64_t>(free, s64, &sum);
    free = sum;
    const int64_t asked = p.w.upto[p.n - 1];
    if (before < asked && (int)blockIdx.x < p.segments) {
        int valid = 0, total = 0;
        const unsigned used = pages_in_use(p, (int)blockIdx.x, &valid);
        int64_t rank = before + block_before<kSegThreads, int>(valid - __popc(used), s, &total);
        for (int i = 0; i < valid && rank < asked; ++i) {
            if (used >> i & 1u) continue;
            int lo = 0, hi = p.n - 1;  // the first entry with upto > rank
            while (lo < hi) {
                const int mid = lo + (hi - lo) / 2;
                if (p.w.upto[mid] > rank) hi = mid;
                else lo = mid + 1;
            }
            const int64_t first = lo > 0 ? p.w.upto[lo - 1] : 0;
            if (p.w.upto[lo] <= free) {
                const int page = (int)blockIdx.x * kSegment + (int)threadIdx.x * kSegEach + i;
                p.table[p.dst[lo] * p.kv.ld + p.w.have[lo] + (rank - first)] = page;
                p.refs[page] = 1;
                if (FORK) p.w.to[lo] = page;
            }
            ++rank;
        }
    }
    // a warp an entry
    const int warps = (int)gridDim.x * (kSegThreads / 32), lane = (int)threadIdx.x % 32;
    for (int64_t e = (int64_t)blockIdx.x * (kSegThreads / 32) + threadIdx.x / 32; e < p.n; e += warps) {
        const bool good = p.w.flag[e] != 0 && p.w.upto[e] <= free;
        if (lane == 0 && p.ok != nullptr) p.ok[e] = good;
        if (!good) continue;
        const int d = p.dst[e];
        if (FORK)
            for (int i = lane; i < p.w.have[e]; i += 32) {
                const int page = p.table[p.src[e] * p.kv.ld + i];
                p.table[d * p.kv.ld + i] = page;
                if (p.kv.is_page(page)) atomicAdd(&p.refs[page], 1);
            }
        if (lane == 0) p.lens[d] = p.w.len[e];
    }
}

// The same for lists of up to kGrowEntries in one launch of one cluster: every CTA works the list out for itself in
// shared memory, counts the free pages of its share of all, and after a cluster barrier gives its own out.  A
// launch and the trip of the list through memory are saved: 48 forks and their reserve 27 -> 23 us (the two kernels above are for longer lists).
constexpr int kGrowCtas = 8, kGrowThreads = 1024, kGrowEntries = 1024;
constexpr int kGrowEach = 8;  // pages of a thread at a time

template <bool FORK>
__global__ void __launch_bounds__(kGrowThreads) grow_kernel(const KvParams p) {
    __shared__ __align__(16) int s_dst[kGrowEntries];
    __shared__ int s_have[kGrowEntries], s_len[kGrowEntries];
    __shared__ int64_t s_upto[kGrowEntries];
    __shared__ bool s_can[kGrowEntries];
    __shared__ int s[kGrowThreads / 32];
    __shared__ int64_t s64[kGrowThreads / 32];
    __shared__ int s_free;
    stream_wait();
    stream_release();
    const int tid = (int)threadIdx.x, rank = (int)cluster_ctarank(), lane = tid % 32;
    // the list: entry tid
    const int e = tid, d = e < p.n ? p.dst[e] : -1;
    const int src = FORK && e < p.n ? p.src[e] : -1, add = !FORK && e < p.n ? p.add[e] : 0;
    if (e < kGrowEntries) s_dst[e] = d;
    bool can = e < p.n && p.kv.is_seq(d);
    int old = 0, mine = 0;
    if (can) {
        mine = p.lens[d];
        if (FORK && p.kv.is_seq(src)) old = p.kv.tokens(p.lens[src]);
    }
    // this CTA's pages: those free
    const int share = (p.kv.num_pages + kGrowCtas - 1) / kGrowCtas;
    const int page0 = min(share * rank, p.kv.num_pages), page1 = min(page0 + share, p.kv.num_pages);
    int free = 0;
    for (int i = page0 + tid; i < page1; i += kGrowThreads) free += p.refs[i] <= 0;
    free = block_sum<kGrowThreads>(free, s);
    if (tid == 0) s_free = free;
    int have = 0, len = 0;
    int64_t need = 0;
    if (can) {
        // named earlier?  Four at a time; the last ones from e on do not count
        int same = 0;
        for (int i = 0; i < e; i += 4) {
            const int4 v = *reinterpret_cast<const int4 *>(s_dst + i);
            same |= (v.x == d) | (i + 1 < e & v.y == d) | (i + 2 < e & v.z == d) | (i + 3 < e & v.w == d);
        }
        can = same == 0;
        if (FORK) {
            can = can && p.kv.is_seq(src) && src != d && mine == 0;
            if (can) {
                len = old;
                have = len / p.kv.page_size;
                need = len % p.kv.page_size != 0;
            }
        } else if (can) {
            const int before = p.kv.tokens(mine);
            const int64_t grown = (int64_t)before + add;
            can = add >= 0 && grown <= (int64_t)p.kv.max_pages * p.kv.page_size;
            if (can) {
                len = (int)grown;
                have = p.kv.pages_of(before);
                need = p.kv.pages_of(len) - have;
            }
        }
    }
    int64_t asked = 0;
    const int64_t upto = block_before<kGrowThreads, int64_t>(need, s64, &asked) + need;
    s_have[e] = have;
    s_len[e] = len;
    s_upto[e] = upto;
    s_can[e] = can;
    cluster_sync();  // the counts are there, and all lengths have been read
    int64_t before = 0, total = 0;
    for (int r = 0; r < kGrowCtas; ++r) {
        const int c = read_cluster_int(&s_free, r);
        if (r < rank) before += c;
        total += c;
    }
    // 64 bits: the step past the last pages of the largest pool leaves 32
    for (int64_t base = page0; base < page1 && before < asked; base += kGrowThreads * kGrowEach) {
        const int64_t first = base + tid * kGrowEach;
        unsigned bits = 0;
#pragma unroll
        for (int i = 0; i < kGrowEach; ++i)
            if (first + i < page1 && p.refs[first + i] <= 0) bits |= 1u << i;
        int here = 0;
        int64_t order = before + block_before<kGrowThreads, int>(__popc(bits), s, &here);
        before += here;
        for (; bits != 0 && order < asked; bits &= bits - 1, ++order) {
            int lo = 0, hi = p.n - 1;  // the first entry with upto > order
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (s_upto[mid] > order) hi = mid;
                else lo = mid + 1;
            }
            if (s_upto[lo] > total) continue;
            const int page = (int)first + __ffs(bits) - 1;
            p.table[s_dst[lo] * p.kv.ld + s_have[lo] + (order - (lo > 0 ? s_upto[lo - 1] : 0))] = page;
            p.refs[page] = 1;
            if (FORK) p.w.to[lo] = page;
        }
    }
    // a warp an entry
    for (int i = rank * (kGrowThreads / 32) + tid / 32; i < p.n; i += kGrowCtas * (kGrowThreads / 32)) {
        const bool good = s_can[i] && s_upto[i] <= total;
        if (lane == 0 && p.ok != nullptr) p.ok[i] = good;
        if (FORK) {
            const int from = p.src[i], whole = s_have[i];
            const bool part = good && s_len[i] % p.kv.page_size != 0;
            if (lane == 0) p.w.from[i] = part ? p.kv.page_at(p.table, from, whole) : -1;
            if (!good) continue;
            for (int j = lane; j < whole; j += 32) {
                const int page = p.table[from * p.kv.ld + j];
                p.table[s_dst[i] * p.kv.ld + j] = page;
                if (p.kv.is_page(page)) atomicAdd(&p.refs[page], 1);
            }
        }
        if (good && lane == 0) p.lens[s_dst[i]] = s_len[i];
    }
    cluster_sync();  // no CTA ends while another may still read its count
}

// ---------------------------------------------------------------- copying

struct CopyParams {
    const uint8_t *from[TGC_KV_MAX_POOLS];
    uint8_t *to[TGC_KV_MAX_POOLS];
    const int32_t *src, *dst;
    int64_t n, page_bytes;
    int pools, from_pages, to_pages, pieces;  // pieces a page
};

// A warp copies a piece of up to kPiece bytes of a page: all its loads under way before the first store.
// Bound by HBM: every byte once each way.
constexpr int kPiece = 4096;
constexpr int kCopyThreads = 256;

__device__ __forceinline__ void copy_pages(const CopyParams &p, int64_t n) {
    const int lane = (int)threadIdx.x % 32;
    const int64_t warps = (int64_t)gridDim.x * (kCopyThreads / 32), items = n * p.pools * p.pieces;
    for (int64_t w = (int64_t)blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32; w < items; w += warps) {
        const int64_t i = w / (p.pools * p.pieces);
        const int rest = (int)(w - i * (p.pools * p.pieces)), pool = rest / p.pieces, piece = rest - pool * p.pieces;
        const int a = p.src[i], b = p.dst[i];
        if (a < 0 || a >= p.from_pages || b < 0 || b >= p.to_pages) continue;
        const int64_t at = (int64_t)piece * kPiece + lane * 16;
        const uint8_t *from = p.from[pool] + a * p.page_bytes + at;
        uint8_t *to = p.to[pool] + b * p.page_bytes + at;
        uint4 v[kPiece / 512];
#pragma unroll
        for (int j = 0; j < kPiece / 512; ++j)
            if (at + j * 512 < p.page_bytes) v[j] = *reinterpret_cast<const uint4 *>(from + j * 512);
#pragma unroll
        for (int j = 0; j < kPiece / 512; ++j)
            if (at + j * 512 < p.page_bytes) *reinterpret_cast<uint4 *>(to + j * 512) = v[j];
    }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
    stream_wait();
    stream_release();
    copy_pages(p, p.n);
}

// ---------------------------------------------------------------- free, compact

__global__ void __launch_bounds__(kSegThreads) free_kernel(const KvParams p) {
    stream_wait();
    stream_release();
    const int64_t threads = (int64_t)gridDim.x * kSegThreads, items = (int64_t)p.n * p.kv.max_pages;
    for (int64_t i = (int64_t)blockIdx.x * kSegThreads + threadIdx.x; i < items; i += threads) {
        const int e = (int)(i / p.kv.max_pages), d = p.dst[e];
        if (!p.kv.is_seq(d)) continue;
        int32_t *entry = p.table + d * p.kv.ld + (i - (int64_t)e * p.kv.max_pages);
        if (*(volatile int32_t *)entry < 0) continue;
        const int page = atomicExch(entry, -1);  // a sequence listed twice gives its pages back once
        if (p.kv.is_page(page)) atomicSub(&p.refs[page], 1);
    }
    for (int64_t e = (int64_t)blockIdx.x * kSegThreads + threadIdx.x; e < p.n; e += threads)
        if (p.kv.is_seq(p.dst[e])) p.lens[p.dst[e]] = 0;
}

__global__ void __launch_bounds__(kSegThreads) count_used_kernel(const KvParams p) {
    __shared__ int s[kSegThreads / 32];
    stream_wait();
    stream_release();
    int valid = 0;
    const int used = block_sum<kSegThreads>(__popc(pages_in_use(p, (int)blockIdx.x, &valid)), s);
    if (threadIdx.x == 0) p.w.count[blockIdx.x] = used;
}

// Movers (in use, at or above the number in use) and holes (free, below it), both in order: the j-th goes to the j-th.
__global__ void __launch_bounds__(kSegThreads) plan_moves_kernel(const KvParams p) {
    __shared__ int s[kSegThreads / 32];
    stream_wait();
    stream_release();
    int before = 0, all = 0;
    for (int i = (int)threadIdx.x; i < p.segments; i += kSegThreads) {
        const int c = p.w.count[i];
        all += c;
        if (i < (int)blockIdx.x) before += c;
    }
    before = block_sum<kSegThreads>(before, s);
    all = block_sum<kSegThreads>(all, s);
    // pages in use below `all`: whole segments, and the one that `all` falls into
    const int edge = all / kSegment;
    int low = 0;
    for (int i = (int)threadIdx.x; i < edge; i += kSegThreads) low += p.w.count[i];
    for (int i = edge * kSegment + (int)threadIdx.x; i < all; i += kSegThreads) low += p.refs[i] > 0;
    low = block_sum<kSegThreads>(low, s);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.w.sums[0] = all - low;
        p.w.sums[1] = all;
        if (p.used != nullptr) *p.used = all;
    }
    int valid = 0, total = 0;
    const unsigned used = pages_in_use(p, (int)blockIdx.x, &valid);
    int rank = before + block_before<kSegThreads, int>(__popc(used), s, &total);  // pages in use before this one
    const int first = (int)blockIdx.x * kSegment + (int)threadIdx.x * kSegEach;
    for (int i = 0; i < valid; ++i) {
        const int page = first + i;
        const bool in_use = used >> i & 1u;
        if (page >= all) p.w.map[page] = in_use ? rank - low : -1;
        if (page >= all && in_use) p.w.from[rank - low] = page;
        if (page < all && !in_use) p.w.to[page - rank] = page;
        rank += in_use;
    }
}

// The moves: bytes, references, the table.
__global__ void __launch_bounds__(kCopyThreads) move_kernel(const KvParams p, const __grid_constant__ CopyParams c) {
    stream_wait();
    stream_release();
    const int n = p.w.sums[0], all = p.w.sums[1];
    if (n == 0) return;
    const int64_t threads = (int64_t)gridDim.x * kCopyThreads, me = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
    for (int64_t j = me; j < n; j += threads) {
        const int a = p.w.from[j], b = p.w.to[j];
        p.refs[b] = p.refs[a];
        p.refs[a] = 0;
    }
    const int64_t entries = (int64_t)p.kv.num_seqs * p.kv.max_pages;
    for (int64_t i = me; i < entries; i += threads) {
        const int64_t row = i / p.kv.max_pages;
        int32_t *entry = p.table + row * p.kv.ld + (i - row * p.kv.max_pages);
        const int page = *entry;
        if (page < all || !p.kv.is_page(page)) continue;
        const int move = p.w.map[page];
        if (move >= 0) *entry = p.w.to[move];
    }
    copy_pages(c, n);
}

// ---------------------------------------------------------------- host

#define TGC_TRY(expr)                     \
    do {                                  \
        const int rc_ = (expr);           \
        if (rc_ != TGC_OK) return rc_;    \
    } while (0)

static int done(cudaError_t e) { return e == cudaSuccess ? TGC_OK : cuda_fail(e); }

static bool off4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }

// The bookkeeping that every call but copy has.
static int kv_check(tgc_kv_args &a) {
    if (a.n < 0 || a.n > TGC_MAX_SIZE) return TGC_ERR_INVALID_ARG;
    return kv_table_check(a.num_pages, a.page_size, a.num_seqs, a.max_pages, &a.table_ld);
}

static int kv_params(const tgc_kv_args &a, bool space, KvParams *out) {
    if ((a.num_pages > 0 && a.refs == nullptr) || (a.num_seqs > 0 && a.max_pages > 0 && a.table == nullptr))
        return TGC_ERR_INVALID_ARG;
    if (off4(a.refs) || off4(a.table) || off4(a.lens) || off4(a.src) || off4(a.dst) || off4(a.add) || off4(a.ok) || off4(a.used))
        return TGC_ERR_ALIGN;
    KvParams p{};
    p.refs = a.refs; p.table = a.table; p.lens = a.lens;
    p.kv = KvTable{(int)a.num_pages, (int)a.page_size, (int)a.num_seqs, (int)a.max_pages, a.table_ld};
    p.src = a.src; p.dst = a.dst; p.add = a.add; p.ok = a.ok; p.used = a.used;
    p.n = (int)a.n;
    p.segments = (int)((a.num_pages + kSegment - 1) / kSegment);
    if (space) {
        p.w = kv_space(a.workspace, a.n, a.num_pages, a.num_seqs);
        if (a.workspace == nullptr || a.workspace_bytes < p.w.total) return TGC_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(a.workspace) % 128 != 0) return TGC_ERR_ALIGN;
    }
    *out = p;
    return TGC_OK;
}

static int kv_pools(const tgc_kv_args &a, const void *const *from, int64_t from_pages, CopyParams *out) {
    if (a.npools < 0 || a.npools > TGC_KV_MAX_POOLS || (a.npools > 0 && (a.pools == nullptr || from == nullptr)))
        return TGC_ERR_INVALID_ARG;
    if (a.num_pages < 0 || a.num_pages > TGC_MAX_SIZE || from_pages < 0 || from_pages > TGC_MAX_SIZE) return TGC_ERR_INVALID_ARG;
    *out = CopyParams{};
    if (a.npools == 0) return TGC_OK;  // nothing to copy: page_bytes is not looked at
    // a pool ends below 2^59 bytes, the pieces of all pools below 2^31
    const int64_t most = a.num_pages > from_pages ? a.num_pages : from_pages;
    if (a.page_bytes < 1 || a.page_bytes > (int64_t(1) << 34) || most > (int64_t(1) << 59) / a.page_bytes) return TGC_ERR_INVALID_ARG;
    if (a.page_bytes % 16 != 0) return TGC_ERR_ALIGN;
    CopyParams c{};
    for (int i = 0; i < a.npools; ++i) {
        c.to[i] = static_cast<uint8_t *>(a.pools[i]);
        c.from[i] = static_cast<const uint8_t *>(from[i]);
        if (c.to[i] == nullptr || c.from[i] == nullptr) return TGC_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(c.to[i]) % 16 != 0 || reinterpret_cast<uintptr_t>(c.from[i]) % 16 != 0) return TGC_ERR_ALIGN;
    }
    c.page_bytes = a.page_bytes;
    c.pools = a.npools;
    c.from_pages = (int)from_pages;
    c.to_pages = (int)a.num_pages;
    c.pieces = (int)((a.page_bytes + kPiece - 1) / kPiece);
    *out = c;
    return TGC_OK;
}

// Blocks that copy: 8 warps each, up to 8 an SM.
static int copy_grid(int64_t pages, const CopyParams &c, dim3 *grid) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const int64_t each = (int64_t)c.pools * c.pieces, room = (int64_t)sm_count(dev) * 8;
    const int64_t blocks = pages > room * 8 ? room : (pages * each + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    *grid = dim3((unsigned)(blocks < 1 ? 1 : blocks < room ? blocks : room));
    return TGC_OK;
}

static int copy_impl(const tgc_kv_args &a) {
    if (a.n < 0 || a.n > TGC_MAX_SIZE) return TGC_ERR_INVALID_ARG;
    CopyParams c{};
    TGC_TRY(kv_pools(a, a.from, a.from_pages, &c));
    if (a.n == 0 || a.npools == 0) return TGC_OK;
    if (a.src == nullptr || a.dst == nullptr) return TGC_ERR_INVALID_ARG;
    if (off4(a.src) || off4(a.dst)) return TGC_ERR_ALIGN;
    c.src = a.src; c.dst = a.dst; c.n = a.n;
    dim3 grid;
    TGC_TRY(copy_grid(a.n, c, &grid));
    return done(launch_overlapped(copy_kernel, grid, dim3(kCopyThreads), 0, 1, a.stream, c));
}

template <bool FORK>
static int grow_impl(tgc_kv_args a) {
    TGC_TRY(kv_check(a));
    CopyParams c{};
    if (FORK) TGC_TRY(kv_pools(a, const_cast<const void *const *>(a.pools), a.num_pages, &c));
    if (a.n == 0) return TGC_OK;
    if (a.dst == nullptr || (FORK ? a.src : a.add) == nullptr || (a.num_seqs > 0 && a.lens == nullptr)) return TGC_ERR_INVALID_ARG;
    KvParams p{};
    TGC_TRY(kv_params(a, true, &p));
    cudaError_t e;
    if (a.n <= kGrowEntries) {
        e = launch_overlapped(grow_kernel<FORK>, dim3(kGrowCtas), dim3(kGrowThreads), 0, kGrowCtas, a.stream, p);
    } else {
        e = launch_overlapped(list_kernel<FORK>, dim3((unsigned)p.segments + 1), dim3(kListThreads), 0, 1, a.stream, p);
        if (e != cudaSuccess) return cuda_fail(e);
        const int64_t warps = (a.n + kSegThreads / 32 - 1) / (kSegThreads / 32), blocks = warps < 1024 ? warps : 1024;
        e = launch_overlapped(grant_kernel<FORK>, dim3((unsigned)(blocks > p.segments ? blocks : p.segments)), dim3(kSegThreads), 0, 1,
                              a.stream, p);
    }
    if (e != cudaSuccess || !FORK || a.npools == 0) return done(e);
    c.src = p.w.from; c.dst = p.w.to; c.n = a.n;
    dim3 grid;
    TGC_TRY(copy_grid(a.n, c, &grid));
    return done(launch_overlapped(copy_kernel, grid, dim3(kCopyThreads), 0, 1, a.stream, c));
}

static int free_impl(tgc_kv_args a) {
    TGC_TRY(kv_check(a));
    if (a.n == 0) return TGC_OK;
    if (a.dst == nullptr || (a.num_seqs > 0 && a.lens == nullptr)) return TGC_ERR_INVALID_ARG;
    KvParams p{};
    TGC_TRY(kv_params(a, false, &p));
    int64_t blocks = (a.n * (a.max_pages > 0 ? a.max_pages : 1) + kSegThreads - 1) / kSegThreads;
    if (blocks > 2048) blocks = 2048;
    return done(launch_overlapped(free_kernel, dim3((unsigned)blocks), dim3(kSegThreads), 0, 1, a.stream, p));
}

static int compact_impl(tgc_kv_args a) {
    a.n = 0;
    TGC_TRY(kv_check(a));
    CopyParams c{};
    TGC_TRY(kv_pools(a, const_cast<const void *const *>(a.pools), a.num_pages, &c));
    if (a.num_pages == 0) return a.used == nullptr ? TGC_OK : done(cudaMemsetAsync(a.used, 0, 4, a.stream));
    KvParams p{};
    TGC_TRY(kv_params(a, true, &p));
    cudaError_t e = launch_overlapped(count_used_kernel, dim3((unsigned)p.segments), dim3(kSegThreads), 0, 1, a.stream, p);
    if (e == cudaSuccess) e = launch_overlapped(plan_moves_kernel, dim3((unsigned)p.segments), dim3(kSegThreads), 0, 1, a.stream, p);
    if (e != cudaSuccess) return cuda_fail(e);
    c.src = p.w.from; c.dst = p.w.to;
    dim3 grid;
    TGC_TRY(copy_grid(a.num_pages / 2 + 1, c, &grid));
    return done(launch_overlapped(move_kernel, grid, dim3(kCopyThreads), 0, 1, a.stream, p, c));
}

}  // namespace tgc

extern "C" int tgc_kv_copy(const tgc_kv_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::copy_impl(*args);
}

extern "C" int tgc_kv_reserve(const tgc_kv_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::grow_impl<false>(*args);
}

extern "C" int tgc_kv_fork(const tgc_kv_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::grow_impl<true>(*args);
}

extern "C" int tgc_kv_free(const tgc_kv_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::free_impl(*args);
}

extern "C" int tgc_kv_compact(const tgc_kv_args *args) {
    if (args == nullptr) return TGC_ERR_INVALID_ARG;
    return tgc::compact_impl(*args);
}

extern "C" size_t tgc_kv_workspace_bytes(const tgc_kv_args *args) {
    if (args == nullptr) return 0;
    tgc_kv_args a = *args;
    if (tgc::kv_check(a) != TGC_OK) return 0;
    return tgc::kv_space(nullptr, a.n, a.num_pages, a.num_seqs).total;
}
