// linear_gemm.cuh -- what the linear operator's matrix product kernels share: the three products,
// their parameters, the operand tiles in shared memory and the walk over groups.
//
// One product kernel serves the three products, out(i, j) = sum_r A(i, r) B(j, r):
//   kFwd    y  = x  w^T    A = x  (rows, r contiguous)   B = w (r contiguous)
//   kDgrad  dx = dz w      A = dz (rows, r contiguous)   B = w (j contiguous)
//   kWgrad  dw = dz^T x    A = dz (i contiguous)         B = x (j contiguous)
// kFwd and kDgrad tile the rows of each group; kWgrad reduces over them.  An operand whose r axis
// is contiguous is K-major, the other kind MN-major; tcgen05 takes either from shared memory, so no
// operand is ever transposed by a kernel of its own.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "groups.cuh"
#include "internal.h"
#include "prims.cuh"
#include "schedule.h"

namespace tgc {

enum : int { kFwd = 0, kDgrad = 1, kWgrad = 2 };

// A wait inside the products ends without success after this long; where it is for a whole reduction,
// which may take longer than that, after this long without a step of it.  0 (for tests): after one look.
#ifndef TGC_LINEAR_TIMEOUT_NS
#define TGC_LINEAR_TIMEOUT_NS 4000000000ull
#endif

// At a kernel's end after such a wait: what a stage that was asked for has to land, or a product to end.
constexpr uint64_t kLinDrainNs = 200ull * 1000 * 1000;

constexpr int kRowBox = 32;  // rows of the small boxes that load a partial tile of rows

struct LinearParams {
    int M;           // rows of the grouped axis
    int I, J, R;     // output rows (kWgrad only), output columns, reduction length (not kWgrad)
    int num_m;       // tile rows of one group (kWgrad)
    int listed;      // tile rows of all groups at most (not kWgrad)
    int num_n;       // tile columns
    int ngroups;
    int group_m;     // tile rows of a group of the raster
    const int32_t *offsets;
    // epilogue
    const void *bias, *residual;
    void *y, *z;
    int64_t ldres, ldy, ldz;
    int act;
    int f16;
    int early;            // inputs complete before the kernel before this one started
    int *fault;           // set when a wait expired
    uint64_t timeout_ns;
};

// One product as the entry points ask for it (arguments checked).
struct LinearProduct {
    const void *a, *b;
    int64_t lda, ldb, b_stride;
    int64_t M, I, J, R;  // grouped axis; output rows of kWgrad; output columns; reduction (not kWgrad)
    const int32_t *offsets;
    int ngroups;         // 1 without offsets
    const void *bias, *residual;
    void *y, *z;
    int64_t ldres, ldy, ldz;
    int act;
    int f16;
    int early;           // see launch_overlapped
};
int launch_linear(const LinearProduct &q, int mode, cudaStream_t stream);

// Operand maps: A and B as 3-D (inner, rows, matrix) tensors; a_small the same A with boxes of
// few rows; y and z for the TMA stores.
struct LinearMaps {
    CUtensorMap a, a_small, b, y, z;
};

// Fills the maps for B boxes of b_rows rows (K-major) or 64 columns (MN-major); what q.z == null
// leaves out is not set.  lin_params sets everything but num_m and listed.
constexpr int kLinMaxDevices = 64;
bool lin_maps(LinearMaps *maps, const LinearProduct &q, int mode, int b_rows, int row_box);
int lin_params(LinearParams *p, const LinearProduct &q, int tile_n);
constexpr int kMaxSplit = 8;  // parts: a portable cluster
// (linear_split.cu) The product with the reduction of each 128 x tn tile split over `parts` CTAs.
int launch_linear_split(const LinearProduct &q, int mode, int tn, int parts, cudaStream_t stream);
// room[c]: clusters of c CTAs of the split kernel that the device holds at once.
int split_room(int mode, int device, int (&room)[kMaxSplit + 1]);
// Stages of its ring for tiles of so many rows of A and columns.
int split_stages(int64_t a_rows, int64_t tn);
// Rows of the boxes that the split kernel loads A in: TMA spends its time by box rows, whether
// they exist or not, so a few tokens load 8 at a time.
inline int split_row_box(int64_t M) { return M <= 8 ? 8 : M <= 16 ? 16 : kRowBox; }
// Tile rows of 128 that the split kernel launches: with groups, no more than one partial one each.
inline int64_t split_tiles(const LinearProduct &q, int mode) {
    const int64_t rows = mode == kWgrad ? q.I : q.M;
    if (mode == kWgrad || q.offsets == nullptr) return (rows + 127) / 128;
    return rows / 128 + (q.ngroups < rows ? q.ngroups : rows);
}

struct Tile {
    int e;             // group
    int m0;            // first output row (in y / dx: a row of the whole tensor; in dw: inside the group's matrix)
    int n0;            // first output column
    int rows;          // output rows of the tile that exist (may exceed the tile)
    int red0, red;     // kWgrad: first row and number of rows of the reduction
    int num_kb;        // 64-deep steps of the reduction, at least one
};

// Waits for the phase of `bar` with this parity; false, and the fault marked, when the limit passed.
// progress != 0: address (shared::cluster) of a count of steps that starts the limit anew whenever it moves.
template <bool CLUSTER = false>
__device__ __forceinline__ bool lin_wait(uint64_t *bar, uint32_t parity, const LinearParams &p, uint32_t progress = 0) {
    const uint32_t a = smem_addr(bar);
    constexpr bool kLook = TGC_LINEAR_TIMEOUT_NS == 0;
    auto ready = [&] {
        if (kLook) return mbar_test_wait(a, parity);
        return CLUSTER ? mbar_try_wait_cluster(a, parity) : mbar_try_wait(a, parity);
    };
    if (ready()) return true;
    uint64_t t0 = globaltimer_ns();
    uint32_t seen = progress != 0 ? read_progress(progress) : 0u;
    for (uint64_t it = 1; !kLook && it < (1ull << 40); ++it) {
        if (ready()) return true;
        if ((it & 63) != 0) continue;
        const uint64_t now = globaltimer_ns();
        const uint32_t steps = progress != 0 ? read_progress(progress) : 0u;
        if (steps != seen) {
            seen = steps;
            t0 = now;
        }
        if (now - t0 > p.timeout_ns) break;
    }
    raise_status(p.fault, kStatusTimeout);
    return false;
}

// Cumulative tile rows of the groups, built by one warp at kernel start: tile0[e] is the first
// tile row of group e, tile0[ngroups] their number (p.listed where groups overlap and have more).
__device__ __forceinline__ void build_tile_table(const LinearParams &p, int tile_m, int *tile0, int lane) {
    int base = 0;
    for (int e0 = 0; e0 < p.ngroups; e0 += 32) {
        int n = 0;
        if (e0 + lane < p.ngroups) {
            const RowRange r = group_range(p.offsets, e0 + lane, p.M);
            n = (r.end - r.begin + tile_m - 1) / tile_m;
        }
        int upto = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        if (e0 + lane < p.ngroups) tile0[e0 + lane] = listed_place(base, upto - n, p.listed);
        base = listed_place(base, __shfl_sync(0xffffffffu, upto, 31), p.listed);
    }
    if (lane == 0) tile0[p.ngroups] = base;
}

template <int MODE>
__device__ __forceinline__ int num_tiles(const LinearParams &p, const int *tile0) {
    return MODE == kWgrad ? p.ngroups * p.num_m * p.num_n : tile0[p.ngroups] * p.num_n;
}

template <int MODE, int TM, int TN>
__device__ __forceinline__ Tile get_tile(const LinearParams &p, const int *tile0, int t) {
    Tile r;
    TileSchedule s;
    s.num_pid_n = p.num_n;
    s.group_m = p.group_m;
    s.pivot_off = 0;
    s.band_n = 0;
    int pm, pn;
    if (MODE == kWgrad) {
        const int per = p.num_m * p.num_n;
        r.e = t / per;
        s.num_pid_m = p.num_m;
        s.tile(t - r.e * per, pm, pn);
        const RowRange g = group_range(p.offsets, r.e, p.M);
        r.red0 = g.begin;
        r.red = g.end - g.begin;
        r.m0 = pm * TM;
        r.rows = p.I - r.m0;
        r.num_kb = r.red > 0 ? (r.red + kBK - 1) / kBK : 1;
    } else {
        const int row = t / p.num_n;  // the last group whose first tile row is <= row
        int lo = 0, hi = p.ngroups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (tile0[mid] <= row) lo = mid; else hi = mid;
        }
        r.e = lo;
        s.num_pid_m = tile0[lo + 1] - tile0[lo];
        s.tile(t - tile0[lo] * p.num_n, pm, pn);
        const RowRange g = group_range(p.offsets, lo, p.M);
        r.m0 = g.begin + pm * TM;
        r.rows = g.end - r.m0;
        r.red0 = 0;
        r.red = p.R;
        r.num_kb = (p.R + kBK - 1) / kBK;
    }
    r.n0 = pn * TN;
    return r;
}

// Four words of 16-bit pairs added to eight fp32 values.
__device__ __forceinline__ void add16(F2 (&v)[4], const uint4 &w, bool f16) {
    v[0] = add(v[0], unpack16(w.x, f16));
    v[1] = add(v[1], unpack16(w.y, f16));
    v[2] = add(v[2], unpack16(w.z, f16));
    v[3] = add(v[3], unpack16(w.w, f16));
}

}  // namespace tgc
