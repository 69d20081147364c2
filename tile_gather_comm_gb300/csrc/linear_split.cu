// linear_split.cu -- the linear operator's products when there are few tiles: the reduction of a
// tile of 128 rows and up to 128 columns is split over the CTAs of a cluster, which add their
// partial sums through distributed shared memory.
//
// With few rows the product streams the weight once and is bound by HBM (one row: 1 flop a byte);
// what matters is that the SMs load, with enough bytes in flight.  So: small tiles, CTAs of about
// 110 KiB, all of it stages, of which two fit an SM, the reduction cut into parts where there are
// few tiles, and A's stage no larger than the rows there are (the MMA reads 128 rows of shared memory
// whatever they hold; what it computes from rows that do not exist is never stored).  No partial
// sum goes to memory and nothing is added atomically: every output is summed over the parts in
// order by one thread, so the result is the same in every run.
// Measured, with the forms that lin_choose takes: 1 x 4096 x 14336 bf16 23.7 to 24.4 us a call among others
// (4.8 TB/s; 29 alone from a cold L2) on 112 CTAs, a tile of 128 columns each and its whole reduction; 48 x
// 14336 x 4096 f16 with a residual 29 us on 32 tiles of 4 parts; 48 rows over 16 experts of 4096 x 14336
// 218 to 224 us (6.9 TB/s) on 1792 CTAs.  Their bytes take 17.6, 17.9 and 228 at the copy rate.
#include <cstdint>
#include <cstring>
#include <mutex>

#include "linear_gemm.cuh"

namespace tgc {

constexpr int kSplitThreads = 256;
constexpr int kSplitSmem = 110 * 1024;             // two CTAs an SM, with what the system and static data take
constexpr int kSplitRing = kSplitSmem - 1024 - 512;  // less alignment slack and barriers
constexpr int kSplitMaxStages = 12;

struct SplitShape {
    int a_bytes, stages;  // A's stage and their number
    int parts;            // CTAs of a cluster
    int tn;               // columns of a tile: a multiple of 16, of 64 where B is MN-major
    int row_box;          // rows of the boxes A is loaded in
};

constexpr uint32_t kSplitTmemCols = 128;

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int MODE>
__global__ void __launch_bounds__(kSplitThreads, 2)
    linear_split_kernel(const __grid_constant__ LinearMaps maps, const LinearParams p, const SplitShape q) {
    constexpr bool kAMn = MODE == kWgrad, kBMn = MODE != kFwd;
    constexpr uint32_t kBoxMn = 64 * kBK * 2;
    const int TN = q.tn, kBBytes = TN * kBK * 2;
    const int kPitch = TN + 4;  // floats from one row of the partial tile to the next: no bank conflicts
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *sA = ring, *sB = ring + q.stages * q.a_bytes;
    float *part = reinterpret_cast<float *>(ring);  // after the last product the ring holds the partial tile
    uint64_t *full = reinterpret_cast<uint64_t *>(ring + kSplitRing);
    uint64_t *empty = full + kSplitMaxStages;
    uint64_t *done = empty + kSplitMaxStages;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(done + 1);
    __shared__ Tile s_tile;
    __shared__ uint32_t s_steps;  // whose products have been issued

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part_id = (int)(blockIdx.x % (unsigned)q.parts), t = (int)(blockIdx.x / (unsigned)q.parts);
    if (threadIdx.x == 0) {
        for (int s = 0; s < q.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        s_steps = 0u;
        fence_mbarrier_init();
        fence_proxy_async_shared();
        prefetch_tensormap(MODE == kWgrad ? &maps.a : &maps.a_small);
        prefetch_tensormap(&maps.b);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, kSplitTmemCols);
        tmem_relinquish();
    }
    if (MODE != kWgrad && p.offsets == nullptr && !p.early && threadIdx.x == 96) {
        // The weight's first stages come into L2 while the kernel before this one ends.  L2 is where
        // all SMs' writes meet, so this is right even if that kernel writes the weight.  Not beside a main
        // part (early), which reads the same weight now: 777 x 4104 x 5000 39.9 -> 39.4 us without it.
        const int steps = (p.R + kBK - 1) / kBK, n0 = t % p.num_n * TN;
        const int b0 = (int)((int64_t)steps * part_id / q.parts), b1 = (int)((int64_t)steps * (part_id + 1) / q.parts);
        for (int kb = b0; kb < b1 && kb < b0 + q.stages; ++kb) {
            if (kBMn) {
                for (int c = 0; c < TN / 64; ++c) tma_prefetch_3d(&maps.b, n0 + c * 64, kb * kBK, 0);
            } else {
                tma_prefetch_3d(&maps.b, kb * kBK, n0, 0);
            }
        }
    }
    if (!p.early) stream_wait();
    if (warp == 2) {  // which tile
        Tile tl;
        int pm, pn = t % p.num_n;
        if (MODE == kWgrad || p.offsets == nullptr) {  // (kWgrad with groups does not come here)
            pm = t / p.num_n;
            tl.e = 0;
            tl.m0 = pm * 128;
            tl.rows = (MODE == kWgrad ? p.I : p.M) - tl.m0;
        } else {
            tl.e = find_group_tile(p.offsets, p.ngroups, p.M, 128, t / p.num_n, lane, &pm);
            const RowRange g = tl.e >= 0 ? group_range(p.offsets, tl.e, p.M) : RowRange{0, 0};
            tl.m0 = g.begin + pm * 128;
            tl.rows = tl.e >= 0 ? g.end - tl.m0 : 0;
        }
        tl.n0 = pn * TN;
        tl.red0 = 0;
        tl.red = MODE == kWgrad ? p.M : p.R;
        tl.num_kb = (tl.red + kBK - 1) / kBK;
        if (lane == 0) s_tile = tl;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const Tile tl = s_tile;
    const int rows = tl.rows < 128 ? tl.rows : 128;
    // this CTA's share of the steps; every part has one (parts <= num_kb)
    const int kb0 = (int)((int64_t)tl.num_kb * part_id / q.parts), kb1 = (int)((int64_t)tl.num_kb * (part_id + 1) / q.parts);
    bool ok = true;
    if (rows > 0) {  // the same for the whole cluster
        if (warp == 0 && lane == 0) {
            const int box_bytes = kAMn ? (int)kBoxMn : q.row_box * kBK * 2;
            const int boxes = kAMn ? 2 : (rows + q.row_box - 1) / q.row_box;
            const uint32_t tx = (uint32_t)(boxes * box_bytes + kBBytes);
            int s = 0;
            uint32_t ph = 1;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!lin_wait(&empty[s], ph, p)) break;
                mbar_arrive_expect_tx(&full[s], tx);
                uint8_t *a = sA + s * q.a_bytes, *b = sB + s * kBBytes;
                const int r0 = kb * kBK;
                if (kBMn) {
                    for (int c = 0; c < TN / 64; ++c)
                        tma_load_3d(b + c * kBoxMn, &maps.b, &full[s], tl.n0 + c * 64, r0, MODE == kWgrad ? 0 : tl.e);
                } else {
                    tma_load_3d(b, &maps.b, &full[s], r0, tl.n0, tl.e);
                }
                if (kAMn) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_3d(a + c * kBoxMn, &maps.a, &full[s], tl.m0 + c * 64, r0, 0);
                } else {
                    for (int c = 0; c < boxes; ++c)
                        tma_load_3d(a + c * box_bytes, &maps.a_small, &full[s], r0, tl.m0 + c * q.row_box, 0);
                }
                if (++s == q.stages) { s = 0; ph ^= 1u; }
            }
            // Only now: a successor that started with this kernel would take HBM from it.
            stream_release();
        } else if (warp == 1 && lane == 0) {
            const uint32_t idesc = make_idesc_16_f32(p.f16 != 0, kAMn, kBMn, 128, TN);
            const uint32_t a0 = smem_addr(sA), b0 = smem_addr(sB);
            int s = 0;
            uint32_t ph = 0;
            bool fed = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                fed = lin_wait(&full[s], ph, p);
                if (!fed) break;
                tc_fence_after();
                const uint64_t ad = kAMn ? make_sw128_mnmajor_desc(a0 + s * q.a_bytes, kBoxMn)
                                         : make_sw128_kmajor_desc(a0 + s * q.a_bytes);
                const uint64_t bd = kBMn ? make_sw128_mnmajor_desc(b0 + s * kBBytes, kBoxMn)
                                         : make_sw128_kmajor_desc(b0 + s * kBBytes);
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                    mma_bf16_ss(tmem, ad + (uint64_t)(k * (kAMn ? 2048 >> 4 : 32 >> 4)),
                                bd + (uint64_t)(k * (kBMn ? 2048 >> 4 : 32 >> 4)), idesc, kb > kb0 || k > 0 ? 1u : 0u);
                mma_commit(&empty[s]);
                if ((kb & 15) == 0) publish_progress(&s_steps, (uint32_t)(kb - kb0 + 1));
                if (++s == q.stages) { s = 0; ph ^= 1u; }
            }
            mma_commit(done);
            if (!fed) {  // what is under way has time to end before the ring and TMEM are used otherwise
                mbar_drain_wait(done, 0, kLinDrainNs);
                for (int n = 0; n < q.stages; ++n) {
                    mbar_drain_wait(&full[s], ph, kLinDrainNs);
                    if (++s == q.stages) { s = 0; ph ^= 1u; }
                }
            }
        }
        __syncwarp();
        // Every load this CTA issued has landed once the MMAs that read it have completed, so the
        // ring is free.  TMEM lane = row of the tile.
        if (lane == 0) ok = lin_wait(done, 0, p, smem_addr(&s_steps));
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        tc_fence_after();
        const int qrow = (warp & 3) * 32, row = qrow + lane;
        if (ok && qrow < rows) {  // warps 0..3 take the even 32-column chunks, 4..7 the odd ones
#pragma unroll 1
            for (int j = warp >> 2; j * 32 < TN; j += 2) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + ((uint32_t)qrow << 16) + (uint32_t)(j * 32), v);
                tmem_wait_ld();
                if (row < rows) {
                    float4 *to = reinterpret_cast<float4 *>(part + row * kPitch + j * 32);
                    const int nc = TN - j * 32 >= 32 ? 8 : 4;  // TN is a multiple of 16
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c < nc) to[c] = make_float4(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]),
                                            __uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3]));
                }
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kSplitTmemCols);
    }
    if (q.parts > 1) cluster_sync();
    if (rows > 0) {
        // 8 columns a thread: the parts' sums in order, then the epilogue
        const bool f16 = p.f16 != 0;
        const int vecs = TN / 8, total = rows * vecs;
        const uint32_t part0 = smem_addr(part);
        for (int i = part_id * kSplitThreads + (int)threadIdx.x; i < total; i += q.parts * kSplitThreads) {
            const int r = i / vecs, c = (i % vecs) * 8, n = tl.n0 + c;
            if (n >= p.J) continue;
            F2 v[4];
#pragma unroll
            for (F2 &f : v) f = every<F2>(0.0f);
            const uint32_t at = part0 + (uint32_t)(r * kPitch + c) * 4u;
            for (int k = 0; k < q.parts; ++k) {
                const uint32_t from = q.parts > 1 ? mapa_shared(at, (uint32_t)k) : at;
                const float4 a = ld_cluster_f4(from), b = ld_cluster_f4(from + 16u);
                v[0] = add(v[0], f2(a.x, a.y));
                v[1] = add(v[1], f2(a.z, a.w));
                v[2] = add(v[2], f2(b.x, b.y));
                v[3] = add(v[3], f2(b.z, b.w));
            }
            const int64_t m = tl.m0 + r;
            auto packed = [&] {
                return make_uint4(pack16(v[0], f16), pack16(v[1], f16), pack16(v[2], f16), pack16(v[3], f16));
            };
            if (MODE == kFwd) {
                if (p.bias != nullptr)
                    add16(v, *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.bias) + (int64_t)tl.e * p.J + n),
                          f16);
                if (p.z != nullptr) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.z) + m * p.ldz + n) = packed();
                if (p.act != TGC_ACT_NONE)
                    with_act(p.act, [&](auto act) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = act_of<decltype(act)::value>(v[k]);
                    });
                if (p.residual != nullptr)
                    add16(v, *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.residual) + m * p.ldres + n),
                          f16);
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + m * p.ldy + n) = packed();
        }
    }
    __syncwarp();
    if (q.parts > 1) cluster_sync();  // no CTA leaves while another reads its partial tile
    if (p.early) stream_wait();
}

// ---------------------------------------------------------------- host side

int split_stages(int64_t a_rows, int64_t tn) {
    const int64_t n = kSplitRing / ((a_rows + tn) * kBK * 2);
    return n < kSplitMaxStages ? (int)n : kSplitMaxStages;
}

struct SplitRoom {
    bool done;
    int room[kMaxSplit + 1];
};

// Sets the kernel's shared-memory limit and asks what fits, once per device.
template <int MODE>
static int split_setup(int dev, SplitRoom **out) {
    static std::mutex mu;
    static SplitRoom cached[kLinMaxDevices] = {};
    if (dev < 0 || dev >= kLinMaxDevices) return TGC_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(mu);
    SplitRoom &r = cached[dev];
    if (!r.done) {
        cudaError_t e = cudaFuncSetAttribute(linear_split_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kSplitSmem);
        // the whole of it as shared memory, so that two CTAs fit (and the query counts them)
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(linear_split_kernel<MODE>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return cuda_fail(e);
        // The query counts one CTA an SM although two run there (a grid of 224 single CTAs starts
        // within 0.8 us on 152 SMs): its answers are doubled.
        for (int c = 1; c <= kMaxSplit; ++c) {
            cudaLaunchConfig_t cfg{};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)c;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3((unsigned)(c * 1024));
            cfg.blockDim = dim3(kSplitThreads);
            cfg.dynamicSmemBytes = kSplitSmem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&r.room[c], linear_split_kernel<MODE>, &cfg);
            if (e != cudaSuccess) return cuda_fail(e);
            r.room[c] *= 2;
        }
        r.done = true;
    }
    *out = &r;
    return TGC_OK;
}

int split_room(int mode, int device, int (&room)[kMaxSplit + 1]) {
    SplitRoom *r = nullptr;
    const int rc = mode == kFwd     ? split_setup<kFwd>(device, &r)
                   : mode == kDgrad ? split_setup<kDgrad>(device, &r)
                                    : split_setup<kWgrad>(device, &r);
    if (rc == TGC_OK) std::memcpy(room, r->room, sizeof r->room);
    return rc;
}

template <int MODE>
static int split_launch(const LinearProduct &q, int tn, int parts, cudaStream_t stream) {
    const int64_t rows = MODE == kWgrad ? q.I : q.M;
    SplitShape s{};
    s.parts = parts;
    s.tn = tn;
    s.row_box = split_row_box(q.M);
    // A's stage: the boxes that a tile can need (a group may fill it; kWgrad always does)
    s.a_bytes = MODE == kWgrad || rows > 96 ? 16384 : (int)((rows + s.row_box - 1) / s.row_box) * s.row_box * kBK * 2;
    s.stages = split_stages(s.a_bytes / (kBK * 2), tn);
    LinearMaps maps;
    if (!lin_maps(&maps, q, MODE, tn, s.row_box)) return TGC_ERR_CUDA;
    LinearParams p{};
    const int rc = lin_params(&p, q, tn);
    if (rc != TGC_OK) return rc;
    const int64_t tiles = split_tiles(q, MODE) * p.num_n;
    if (tiles * parts >= (int64_t(1) << 31)) return TGC_ERR_INVALID_ARG;
    const cudaError_t e = launch_overlapped(linear_split_kernel<MODE>, dim3((unsigned)(tiles * parts)), dim3(kSplitThreads),
                                            kSplitSmem, parts, stream, maps, p, s);
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
}

int launch_linear_split(const LinearProduct &q, int mode, int tn, int parts, cudaStream_t stream) {
    return mode == kFwd     ? split_launch<kFwd>(q, tn, parts, stream)
           : mode == kDgrad ? split_launch<kDgrad>(q, tn, parts, stream)
                            : split_launch<kWgrad>(q, tn, parts, stream);
}

}  // namespace tgc
