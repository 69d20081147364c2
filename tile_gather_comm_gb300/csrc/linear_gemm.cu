// linear_gemm.cu -- the tensor-core product of the linear operator (linear_gemm.cuh says which
// three products) on tcgen05 / TMEM / TMA.
//
// Bound by the tensor pipe once a call has a few hundred rows (2 flops x rows per weight byte
// against 280 flops a byte of the card).  Persistent: one CTA (CG = 1, tiles of 128 rows) or one
// pair (CG = 2, 256 rows, tcgen05 cta_group::2, which halves the bytes of B a CTA stages) walks
// tiles of 128 or 256 columns; two accumulators in TMEM alternate, so a tile's epilogue runs under
// the next tile's products.
//   warps 0, 3  TMA loads into a ring of 64-deep stages (128-byte swizzle); a tile with fewer rows
//               than it could hold loads boxes of 32 rows and no more.  MN-major operands take a
//               load for every 64 columns, so in kDgrad and kWgrad A's and B's are issued by a
//               warp each (8192 x 4096 x 14336: weight gradient 531 -> 505 us); kFwd's two a
//               stage by one (528 us against 535)
//   warp 1      TMEM owner; one lane issues the MMAs
//   warp 2      kWgrad with groups: a group's last stage also holds rows of the next group (or
//               beyond the last); it zeroes them in both operands before the MMA reads them, so
//               whatever they hold (NaN too) stays out of the sum.  Such a stage's loads count on a
//               barrier of their own (raw), the repair on another (fixed): both see only these
//               stages, so their phases cannot be taken for one another's
//   warps 4-11  epilogue: TMEM -> registers, bias, z, activation, residual in fp32, one rounding,
//               through shared memory and TMA stores; boxes that a group's end cuts are stored by
//               the lanes whose rows exist
// Measured, bf16, 8192 x 4096 x 14336: plain 492 us in a burst (1955 TFLOP/s) and 570 in a loop of a
// second (1689); with bias, gelu and z 597 to 627 a pass.  At 2048 rows the tensor pipe is active 79 % of
// the time forward, 76 % for the input gradient, 83 % for the weight gradient.  16 experts of 4096 x
// 4096 over 16384 uneven rows: 386 to 411 us with tanh-gelu and z, 71 tile rows where even groups fill 64.
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cudaTypedefs.h>

#include "linear_gemm.cuh"

namespace tgc {

constexpr int kLinThreads = 384;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kBoxBytes = 32 * 32 * 2;  // an epilogue warp's staging box: 32 rows x 32 columns
constexpr int kBiasBytes = 128 * 4;     // its columns' bias in fp32
constexpr uint32_t kLinTmemCols = 512;

template <int CG, int MODE, int TN>
struct LCfg {
    static constexpr int kTM = 128 * CG;
    static constexpr int kBRows = TN / CG;                // B's rows (along j) a CTA stages
    static constexpr int kABytes = 128 * kBK * 2;         // 16 KiB
    static constexpr int kBBytes = kBRows * kBK * 2;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kStages = 196608 / kStage;       // 4 of 48, 6 of 32, 8 of 24 KiB
    static constexpr bool kAMn = MODE == kWgrad, kBMn = MODE != kFwd;
    static constexpr uint32_t kBoxMn = 64 * kBK * 2;      // an MN-major box: 64 columns x 64 rows, 8 KiB
    static constexpr int kSmem = 1024 + kStages * kStage + kEpiWarps * (kBoxBytes + kBiasBytes) +
                                  (TGC_MAX_GROUPS + 8) * 4 + 512;
};

// kWgrad with groups: does step kb of the tile hold rows that are not the group's?
__device__ __forceinline__ bool needs_repair(const LinearParams &p, const Tile &tl, int kb) {
    return p.offsets != nullptr && kb == tl.num_kb - 1 && (kb + 1) * kBK != tl.red;
}

// ---------------------------------------------------------------- loads

// The loads of A (which also announce the stage's bytes), of B, or of both.
template <int CG, int MODE, int TN, bool A, bool B>
__device__ void lin_role_tma(const LinearMaps &maps, const LinearParams &p, const int *tile0, uint8_t *sA, uint8_t *sB,
                             uint64_t *full, uint64_t *empty, uint64_t *raw, uint32_t crank) {
    using C = LCfg<CG, MODE, TN>;
    uint32_t it = 0;
    bool ok = true;
    const uint32_t full0 = CG == 2 ? mapa_shared(smem_addr(full), 0) : smem_addr(full);
    const int tiles = num_tiles<MODE>(p, tile0);
    bool cut = false;  // this step's bytes count on this CTA's own raw barrier
    auto load = [&](void *dst, const CUtensorMap *map, uint32_t s, int c0, int c1, int c2) {
        if (MODE == kWgrad && cut) tma_load_3d(dst, map, &raw[s], c0, c1, c2);
        else if (CG == 1) tma_load_3d(dst, map, &full[s], c0, c1, c2);
        else tma_load_3d_pair(dst, map, full0 + s * 8u, c0, c1, c2);
    };
    // boxes of A that a CTA with `rows` existing rows loads: all 128 rows at once, or 32 at a time
    auto small_boxes = [](int rows) { return rows >= 128 ? 4 : rows <= 0 ? 0 : (rows + kRowBox - 1) / kRowBox; };
    for (int t = (int)blockIdx.x / CG; t < tiles && ok; t += (int)gridDim.x / CG) {
        const Tile tl = get_tile<MODE, C::kTM, TN>(p, tile0, t);
        const int m0 = tl.m0 + (int)crank * 128;
        const int j0 = tl.n0 + (int)crank * C::kBRows;
        int boxes = 4;
        uint32_t tx = CG * (C::kABytes + C::kBBytes);
        if (MODE != kWgrad) {
            boxes = small_boxes(tl.rows - (int)crank * 128);
            const int both = CG == 2 ? small_boxes(tl.rows) + small_boxes(tl.rows - 128) : boxes;
            tx = (uint32_t)(both * (C::kABytes / 4) + CG * C::kBBytes);
        }
        for (int kb = 0; kb < tl.num_kb; ++kb, ++it) {
            const uint32_t s = it % C::kStages, ph = (it / C::kStages) & 1u;
            if (!lin_wait(&empty[s], ph ^ 1u, p)) { ok = false; break; }
            if (MODE == kWgrad) cut = needs_repair(p, tl, kb);
            if (A) {
                if (cut) {
                    mbar_arrive_expect_tx(&raw[s], C::kABytes + C::kBBytes);
                    if (CG == 1 || crank == 0) mbar_arrive(&full[s]);
                } else if (CG == 1 || crank == 0) {
                    mbar_arrive_expect_tx(&full[s], tx);
                }
            }
            const int r0 = (MODE == kWgrad ? tl.red0 : 0) + kb * kBK;
            uint8_t *a = sA + s * C::kABytes, *b = sB + s * C::kBBytes;
            if (A) {
                if (C::kAMn) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) load(a + c * C::kBoxMn, &maps.a, s, m0 + c * 64, r0, 0);
                } else if (boxes == 4) {
                    load(a, &maps.a, s, r0, m0, 0);
                } else {
                    for (int c = 0; c < boxes; ++c)
                        load(a + c * (C::kABytes / 4), &maps.a_small, s, r0, m0 + c * kRowBox, 0);
                }
            }
            if (B) {
                if (C::kBMn) {
#pragma unroll
                    for (int c = 0; c < C::kBRows / 64; ++c)
                        load(b + c * C::kBoxMn, &maps.b, s, j0 + c * 64, r0, MODE == kWgrad ? 0 : tl.e);
                } else {
                    load(b, &maps.b, s, r0, j0, tl.e);
                }
            }
        }
    }
    if (!ok) {
        // let every stage this CTA expected land before shared memory is given up
        if (CG == 1 || crank == 0) {
            for (uint32_t s = 0; s < (uint32_t)C::kStages; ++s) {
                const uint32_t n = it / C::kStages + (s < it % C::kStages ? 1u : 0u);
                if (n > 0) mbar_drain_wait(&full[s], (n - 1) & 1u, kLinDrainNs);
            }
        } else {
            spin_for_ns(200000);
        }
        spin_for_ns(200000);  // and those counted on raw
    }
}

// ---------------------------------------------------------------- products

template <int CG, int MODE, int TN>
__device__ void lin_role_mma(const LinearParams &p, const int *tile0, uint8_t *sA, uint8_t *sB, uint64_t *full,
                             uint64_t *fixed, uint64_t *empty, uint64_t *tfull, uint64_t *tempty, uint64_t *drain,
                             uint32_t *progress, uint32_t tmem_base) {
    using C = LCfg<CG, MODE, TN>;
    const uint32_t idesc = make_idesc_16_f32(p.f16 != 0, C::kAMn, C::kBMn, C::kTM, TN);
    uint32_t it = 0, tc = 0, fixes = 0;  // fixes: per stage, the parity of its next repair
    bool ok = true;
    const int tiles = num_tiles<MODE>(p, tile0);
    const uint32_t a0 = smem_addr(sA), b0 = smem_addr(sB);
    for (int t = (int)blockIdx.x / CG; t < tiles && ok; t += (int)gridDim.x / CG, ++tc) {
        const Tile tl = get_tile<MODE, C::kTM, TN>(p, tile0, t);
        const uint32_t acc = tc & 1u, aph = (tc >> 1) & 1u;
        if (!lin_wait(&tempty[acc], aph ^ 1u, p)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * (uint32_t)TN;
        for (int kb = 0; kb < tl.num_kb; ++kb, ++it) {
            const uint32_t s = it % C::kStages, ph = (it / C::kStages) & 1u;
            if (MODE == kWgrad && needs_repair(p, tl, kb)) {
                if (!lin_wait<CG == 2>(&fixed[s], (fixes >> s) & 1u, p)) { ok = false; break; }
                fixes ^= 1u << s;
            }
            if (!lin_wait(&full[s], ph, p)) { ok = false; break; }
            tc_fence_after();
            const uint64_t ad = C::kAMn ? make_sw128_mnmajor_desc(a0 + s * C::kABytes, C::kBoxMn)
                                        : make_sw128_kmajor_desc(a0 + s * C::kABytes);
            const uint64_t bd = C::kBMn ? make_sw128_mnmajor_desc(b0 + s * C::kBBytes, C::kBoxMn)
                                        : make_sw128_kmajor_desc(b0 + s * C::kBBytes);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
                const uint64_t ak = ad + (uint64_t)(k * (C::kAMn ? 2048 >> 4 : 32 >> 4));
                const uint64_t bk = bd + (uint64_t)(k * (C::kBMn ? 2048 >> 4 : 32 >> 4));
                if (CG == 1) mma_bf16_ss(d, ak, bk, idesc, (kb | k) != 0 ? 1u : 0u);
                else mma_bf16_ss_pair(d, ak, bk, idesc, (kb | k) != 0 ? 1u : 0u);
            }
            if (CG == 1) mma_commit(&empty[s]);
            else mma_commit_pair_mc(&empty[s], (uint16_t)0x3);
            if ((it & 15) == 0) publish_progress(progress, it + 1);
        }
        if (ok) {
            if (CG == 1) mma_commit(&tfull[acc]);
            else mma_commit_pair_mc(&tfull[acc], (uint16_t)0x3);
        }
    }
    if (CG == 1) mma_commit(drain);  // arrives once every MMA issued above has completed
    else mma_commit_pair_mc(drain, (uint16_t)0x1);
    mbar_drain_wait(drain, 0, kLinDrainNs);
    if (!ok) {
        // The loads of the steps that now take none have time to land before shared memory is given up:
        // those counted here (a pair's on the even CTA), then those counted on raw.
        for (uint32_t n = 0; n < (uint32_t)C::kStages; ++n, ++it)
            mbar_drain_wait(&full[it % C::kStages], (it / C::kStages) & 1u, kLinDrainNs);
        spin_for_ns(200000);
    }
}

// kWgrad with groups: zero the rows of a group's last stage that are not the group's.
template <int CG, int MODE, int TN>
__device__ void lin_role_fix(const LinearParams &p, const int *tile0, uint8_t *sA, uint8_t *sB, uint64_t *raw,
                             uint64_t *fixed, uint32_t progress, int lane) {
    using C = LCfg<CG, MODE, TN>;
    uint32_t it = 0, phases = 0;  // phases: per stage, the parity of its next cut step
    const int tiles = num_tiles<MODE>(p, tile0);
    const uint32_t fixed0 = CG == 2 ? mapa_shared(smem_addr(fixed), 0) : smem_addr(fixed);
    for (int t = (int)blockIdx.x / CG; t < tiles; t += (int)gridDim.x / CG) {
        const Tile tl = get_tile<MODE, C::kTM, TN>(p, tile0, t);
        it += (uint32_t)tl.num_kb;
        if (!needs_repair(p, tl, tl.num_kb - 1)) continue;
        const int valid = tl.red - (tl.num_kb - 1) * kBK;
        const uint32_t s = (it - 1) % C::kStages, ph = (phases >> s) & 1u;
        phases ^= 1u << s;
        bool ok = true;
        if (lane == 0) ok = lin_wait(&raw[s], ph, p, progress);
        if (__shfl_sync(0xffffffffu, ok ? 1 : 0, 0) == 0) return;
        __syncwarp();
        // a row of a box is 128 bytes whatever the swizzle; 8 lanes zero one
        auto wipe = [&](uint8_t *box) {
            for (int r = valid + lane / 8; r < kBK; r += 4)
                *reinterpret_cast<uint4 *>(box + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        };
        for (int c = 0; c < 2; ++c) wipe(sA + s * C::kABytes + c * C::kBoxMn);
        for (int c = 0; c < C::kBRows / 64; ++c) wipe(sB + s * C::kBBytes + c * C::kBoxMn);
        fence_proxy_async_shared();  // the MMA reads through the async proxy
        __syncwarp();
        if (lane == 0) {
            if (CG == 1) mbar_arrive(&fixed[s]);
            else mbar_arrive_cluster(fixed0 + s * 8u);
        }
    }
}

// ---------------------------------------------------------------- epilogue

template <int CG, int MODE, int TN>
__device__ void lin_role_epilogue(const LinearMaps &maps, const LinearParams &p, const int *tile0, uint8_t *sC,
                                  float *sBias, uint64_t *tfull, uint64_t *tempty, uint32_t progress, uint32_t tmem_base,
                                  uint32_t crank, int warp, int lane) {
    using C = LCfg<CG, MODE, TN>;
    const int ew = warp - kEpiWarp0, q = warp & 3;  // q: the TMEM lane quarter a warp may read
    const int col0 = (ew >> 2) * (TN / 2);
    uint8_t *box = sC + ew * kBoxBytes;
    float *bias = sBias + ew * (kBiasBytes / 4);
    const uint32_t tempty0 = CG == 2 ? mapa_shared(smem_addr(tempty), 0) : smem_addr(tempty);
    const bool f16 = p.f16 != 0;
    const int tiles = num_tiles<MODE>(p, tile0);
    uint32_t tc = 0;
    for (int t = (int)blockIdx.x / CG; t < tiles; t += (int)gridDim.x / CG, ++tc) {
        const Tile tl = get_tile<MODE, C::kTM, TN>(p, tile0, t);
        const uint32_t acc = tc & 1u, aph = (tc >> 1) & 1u;
        const int wrow = (int)crank * 128 + q * 32;     // this warp's first row of the tile
        const int m_box = tl.m0 + wrow, m = m_box + lane;
        const int rows = tl.rows - wrow;                // rows of the box that exist (may be <= 0 or > 32)
        // dense outputs and dw are clipped by their tensor map; inside grouped rows a cut box is not
        const bool by_tma = rows > 0 && (rows >= 32 || MODE == kWgrad || p.offsets == nullptr);
        const bool row_ok = lane < rows;
        // What the epilogue reads is asked for before the products are done: the bias of this
        // warp's columns (to shared memory, in fp32) and a chunk of the residual at a time.
        uint4 res[4];
        auto fetch_residual = [&](int n) {
            const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.residual) +
                                                             (int64_t)m * p.ldres + n);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (row_ok && n + c * 8 < p.J) res[c] = r[c];
        };
        if (MODE == kFwd) {
            const int n = tl.n0 + col0;
            if (p.bias != nullptr) {
                __syncwarp();  // the last tile's readers are done
                if (lane * 8 < TN / 2 && n + lane * 8 < p.J) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.bias) +
                                                                     (int64_t)tl.e * p.J + n + lane * 8);
                    F2 *to = reinterpret_cast<F2 *>(bias + lane * 8);
                    to[0] = unpack16(w.x, f16);
                    to[1] = unpack16(w.y, f16);
                    to[2] = unpack16(w.z, f16);
                    to[3] = unpack16(w.w, f16);
                }
            }
            if (p.residual != nullptr) fetch_residual(n);
            __syncwarp();
        }
        bool ok = true;
        if (lane == 0) ok = lin_wait(&tfull[acc], aph, p, progress);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;  // warp-uniform: tcgen05.ld is .sync.aligned
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * (uint32_t)TN + (uint32_t)col0;
        auto put = [&](const CUtensorMap *map, void *base, int64_t ld, int n, const uint32_t (&w)[16]) {
            if (by_tma) {
                if (lane == 0) bulk_wait_read<0>();  // the box's last store has read it
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 4; ++c)  // 64-byte swizzle: 16-byte chunk c of row r at c ^ ((r >> 1) & 3)
                    *reinterpret_cast<uint4 *>(box + lane * 64 + (c ^ ((lane >> 1) & 3)) * 16) =
                        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(map, box, n, m_box, MODE == kWgrad ? tl.e : 0);
                    bulk_commit();
                }
            } else if (row_ok) {
                uint8_t *to = static_cast<uint8_t *>(base) + ((int64_t)m * ld + n) * 2;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (n + c * 8 < p.J)
                        *reinterpret_cast<uint4 *>(to + c * 16) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            }
        };
#pragma unroll 1
        for (int j = 0; j < TN / 64; ++j) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(taddr + (uint32_t)(j * 32), v);
            tmem_wait_ld();
            if (j == TN / 64 - 1) {  // the accumulator is in registers: hand it back
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 1) mbar_arrive(&tempty[acc]);
                    else mbar_arrive_cluster(tempty0 + acc * 8u);
                }
            }
            const int n = tl.n0 + col0 + j * 32;
            if (n >= p.J || rows <= 0) continue;  // warp-uniform
            F2 f[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = f2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            auto packed = [&](uint32_t (&w)[16]) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack16(f[i], f16);
            };
            uint32_t w[16];
            if (MODE == kFwd) {
                if (p.bias != nullptr) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {  // the same address in every lane
                        const ulonglong2 b = reinterpret_cast<const ulonglong2 *>(bias + j * 32)[c];
                        f[2 * c] = add(f[2 * c], F2{b.x});
                        f[2 * c + 1] = add(f[2 * c + 1], F2{b.y});
                    }
                }
                if (p.z != nullptr) {
                    packed(w);
                    put(&maps.z, p.z, p.ldz, n, w);
                }
                if (p.act != TGC_ACT_NONE)
                    with_act(p.act, [&](auto act) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) f[i] = act_of<decltype(act)::value>(f[i]);
                    });
                if (p.residual != nullptr) {
                    if (row_ok) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (n + c * 8 < p.J) add16(reinterpret_cast<F2(&)[4]>(f[4 * c]), res[c], f16);
                    }
                    if (j + 1 < TN / 64) fetch_residual(n + 32);
                }
            }
            packed(w);
            put(&maps.y, p.y, p.ldy, n, w);
        }
    }
    if (lane == 0) bulk_wait<0>();  // every store has landed and read its box
    __syncwarp();
}

// ---------------------------------------------------------------- kernel

template <int CG, int MODE, int TN>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_gemm_kernel(const __grid_constant__ LinearMaps maps, const LinearParams p) {
    using C = LCfg<CG, MODE, TN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *sA = smem;
    uint8_t *sB = sA + C::kStages * C::kABytes;
    uint8_t *sC = sB + C::kStages * C::kBBytes;
    float *sBias = reinterpret_cast<float *>(sC + kEpiWarps * kBoxBytes);
    int *tile0 = reinterpret_cast<int *>(sBias + kEpiWarps * (kBiasBytes / 4));
    uint64_t *full = reinterpret_cast<uint64_t *>(tile0 + TGC_MAX_GROUPS + 8);
    uint64_t *empty = full + C::kStages;
    uint64_t *fixed = empty + C::kStages;
    uint64_t *raw = fixed + C::kStages;
    uint64_t *tfull = raw + C::kStages;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1), *progress = tmem_holder + 1;
    static_assert((4 * C::kStages + 5) * 8 + 8 <= 512, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = CG == 2 ? cluster_ctarank() : 0u;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&fixed[s], CG);
            mbar_init(&raw[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], kEpiWarps * CG);
        }
        mbar_init(drain, 1);
        *progress = 0u;
        fence_mbarrier_init();
        fence_proxy_async_shared();
        prefetch_tensormap(&maps.a);
        prefetch_tensormap(&maps.b);
    }
    if (warp == 1) {
        if (CG == 1) { tmem_alloc(tmem_holder, kLinTmemCols); tmem_relinquish(); }
        else { tmem_alloc_pair(tmem_holder, kLinTmemCols); tmem_relinquish_pair(); }
    }
    if (!p.early) stream_wait();
    stream_release();
    if (warp == 2 && MODE != kWgrad) build_tile_table(p, C::kTM, tile0, lane);
    tc_fence_before();
    if (CG == 1) __syncthreads(); else cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    const uint32_t progress0 = CG == 2 ? mapa_shared(smem_addr(progress), 0) : smem_addr(progress);  // the MMAs' steps

    if (warp == 0) {
        if (lane == 0) lin_role_tma<CG, MODE, TN, true, MODE == kFwd>(maps, p, tile0, sA, sB, full, empty, raw, crank);
    } else if (warp == 3) {
        if (MODE != kFwd && lane == 0)
            lin_role_tma<CG, MODE, TN, false, true>(maps, p, tile0, sA, sB, full, empty, raw, crank);
    } else if (warp == 1) {
        if (lane == 0 && crank == 0)
            lin_role_mma<CG, MODE, TN>(p, tile0, sA, sB, full, fixed, empty, tfull, tempty, drain, progress, tmem_base);
    } else if (warp == 2) {
        if (MODE == kWgrad && p.offsets != nullptr)
            lin_role_fix<CG, MODE, TN>(p, tile0, sA, sB, raw, fixed, progress0, lane);
    } else if (warp >= kEpiWarp0) {
        lin_role_epilogue<CG, MODE, TN>(maps, p, tile0, sC, sBias, tfull, tempty, progress0, tmem_base,
                                          crank, warp, lane);
    }
    // in a pair the even CTA's MMAs read the odd one's shared memory: neither leaves before both are done
    __syncwarp();
    tc_fence_before();
    if (CG == 1) __syncthreads(); else cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        if (CG == 1) tmem_dealloc(tmem_base, kLinTmemCols);
        else tmem_dealloc_pair(tmem_base, kLinTmemCols);
    }
    if (p.early) stream_wait();
}

// ---------------------------------------------------------------- host side

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// A stack of `count` (rows, cols) row-major 16-bit matrices, rows `ld` and matrices `stride`
// elements apart.
static bool lin_map(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t count, int64_t ld,
                    int64_t stride, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle,
                    CUtensorMapL2promotion promote) {
    auto enc = encode_fn();
    if (enc == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
    cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(count > 1 ? stride : ld) * 2};
    cuuint32_t box[3] = {box_cols, box_rows, 1}, one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sets the kernel's shared-memory limit once per device and returns how many clusters fit at once.
template <int CG, int MODE, int TN>
static int lin_clusters(int dev, int sms, int *out) {
    using C = LCfg<CG, MODE, TN>;
    static std::mutex mu;
    static int cached[kLinMaxDevices] = {};
    if (dev < 0 || dev >= kLinMaxDevices) return TGC_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(mu);
    if (cached[dev] == 0) {
        const cudaError_t e = cudaFuncSetAttribute(linear_gemm_kernel<CG, MODE, TN>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return cuda_fail(e);
        int n = sms;
        if (CG > 1) {
            cudaLaunchConfig_t cfg{};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = CG;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3((unsigned)(sms / CG * CG));
            cfg.blockDim = dim3(kLinThreads);
            cfg.dynamicSmemBytes = C::kSmem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, linear_gemm_kernel<CG, MODE, TN>, &cfg) != cudaSuccess || n <= 0)
                n = sms / CG;
        }
        cached[dev] = n;
    }
    *out = cached[dev];
    return TGC_OK;
}

bool lin_maps(LinearMaps *maps, const LinearProduct &q, int mode, int b_rows, int row_box) {
    std::memset(maps, 0, sizeof *maps);
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B, sw_out = CU_TENSOR_MAP_SWIZZLE_64B;
    const auto l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B, none = CU_TENSOR_MAP_L2_PROMOTION_NONE;
    const int64_t E = q.ngroups;
    bool ok;
    if (mode == kWgrad) {
        ok = lin_map(&maps->a, q.a, q.I, q.M, 1, q.lda, 0, 64, kBK, sw, l2) &&
             lin_map(&maps->b, q.b, q.J, q.M, 1, q.ldb, 0, 64, kBK, sw, l2);
    } else {
        ok = lin_map(&maps->a, q.a, q.R, q.M, 1, q.lda, 0, kBK, 128, sw, l2) &&
             lin_map(&maps->a_small, q.a, q.R, q.M, 1, q.lda, 0, kBK, (uint32_t)row_box, sw, l2) &&
             (mode == kFwd ? lin_map(&maps->b, q.b, q.R, q.J, E, q.ldb, q.b_stride, kBK, (uint32_t)b_rows, sw, l2)
                           : lin_map(&maps->b, q.b, q.J, q.R, E, q.ldb, q.b_stride, 64, kBK, sw, l2));
    }
    const int64_t out_rows = mode == kWgrad ? q.I : q.M, out_count = mode == kWgrad ? E : 1;
    ok = ok && lin_map(&maps->y, q.y, q.J, out_rows, out_count, q.ldy, q.I * q.ldy, 32, 32, sw_out, none);
    if (q.z != nullptr) ok = ok && lin_map(&maps->z, q.z, q.J, q.M, 1, q.ldz, 0, 32, 32, sw_out, none);
    return ok;
}

int lin_params(LinearParams *p, const LinearProduct &q, int tile_n) {
    p->M = (int)q.M; p->I = (int)q.I; p->J = (int)q.J; p->R = (int)q.R;
    p->num_n = (int)((q.J + tile_n - 1) / tile_n);
    p->ngroups = q.ngroups;
    p->group_m = TGC_DEFAULT_GROUP_M;
    p->offsets = q.offsets;
    p->bias = q.bias; p->residual = q.residual; p->y = q.y; p->z = q.z;
    p->ldres = q.ldres; p->ldy = q.ldy; p->ldz = q.ldz;
    p->act = q.act;
    p->f16 = q.f16;
    p->early = q.early;
    p->timeout_ns = TGC_LINEAR_TIMEOUT_NS;
    return device_fault_word(&p->fault);
}

template <int CG, int MODE, int TN>
static int lin_launch(const LinearProduct &q, int dev, int sms, cudaStream_t stream) {
    using C = LCfg<CG, MODE, TN>;
    LinearMaps maps;
    if (!lin_maps(&maps, q, MODE, C::kBRows, kRowBox)) return TGC_ERR_CUDA;
    int clusters = 0;
    int rc = lin_clusters<CG, MODE, TN>(dev, sms, &clusters);
    if (rc != TGC_OK) return rc;
    LinearParams p{};
    rc = lin_params(&p, q, TN);
    if (rc != TGC_OK) return rc;
    int64_t tiles;
    if (MODE == kWgrad) {
        p.num_m = (int)((q.I + C::kTM - 1) / C::kTM);
        tiles = (int64_t)q.ngroups * p.num_m * p.num_n;
    } else {
        // with groups: no more than one partial tile row each
        const int64_t listed = q.M / C::kTM + (q.offsets != nullptr ? (q.ngroups < q.M ? q.ngroups : q.M) : 0) +
                               (q.M % C::kTM != 0 || q.offsets != nullptr ? 1 : 0);
        p.listed = (int)listed;
        tiles = listed * p.num_n;
    }
    if (tiles >= (int64_t(1) << 31)) return TGC_ERR_INVALID_ARG;
    if (clusters > tiles) clusters = (int)tiles;
    const cudaError_t e = launch_overlapped(linear_gemm_kernel<CG, MODE, TN>, dim3((unsigned)(clusters * CG)),
                                            dim3(kLinThreads), C::kSmem, CG, stream, maps, p);
    return e == cudaSuccess ? TGC_OK : cuda_fail(e);
}

// ---------------------------------------------------------------- which kernel, which tile

// A form's time in SM cycles is the largest of three bounds and what nothing overlaps:
//   l2     what L2 hands out: 2.83 / SMs cycles for every 128-byte row of an operand tile that any SM
//          takes in; rows that do not start on a 128-byte line (they take two) 1.09 times that
//   hbm    every operand once, 2120 bytes a cycle.  That is below what many CTAs stream (48 rows over 16
//          experts: 6.9 TB/s): where it is the largest bound, forms tie on it and the first of them is
//          taken, 112 CTAs for a token of 4096 x 14336 and 128 for 48 x 14336 x 4096, on 152 SMs
//   sm     the busiest SM's steps -- the products (2 cycles a column of the tile) or the rows it takes
//          in -- and, for the persistent kernel, no less than an epilogue a tile
//   extra  start, the last epilogue, and the split kernel's exchange
// The constants were fitted to 13,900 timings (190 shapes of 1..8192 x 64..14336 x 64..14336, three
// products, every form): the form taken is 2.5 % slower than the best on the geometric mean, where
// one persistent form for all rows above 128 and the split kernel below was 18 % slower.  No grouped shape
// was among them.
struct LinearForm {
    int cg, tn;  // the persistent kernel's; cg 0: the split kernel's tn and parts
    int parts;
    int64_t l2, hbm, sm, extra;
    int64_t bound() const { return l2 > hbm ? (l2 > sm ? l2 : sm) : (hbm > sm ? hbm : sm); }
    int64_t cycles() const { return bound() + extra; }
};

enum : int { kPairs = 1, kNarrowPairs = 2, kSingles = 4, kSplits = 8, kAllForms = 15 };

// The best of `forms` on `sms` of the device's `all` SMs; false if none fits.
template <int MODE>
static bool lin_choose(const LinearProduct &q, int all, int sms, const int (&room)[kMaxSplit + 1], int forms,
                       LinearForm *best) {
    const int64_t groups = q.offsets != nullptr ? q.ngroups : 1;
    const int64_t rows = MODE == kWgrad ? q.I : q.M;
    const int64_t steps = ((MODE == kWgrad ? (q.M + groups - 1) / groups : q.R) + kBK - 1) / kBK;
    // Tile rows of height h: exact without groups; with them (kFwd, kDgrad) half a tile more a
    // group that can have rows.
    auto tile_rows = [&](int64_t h) -> int64_t {
        if (MODE == kWgrad) return groups * ((rows + h - 1) / h);
        if (q.offsets == nullptr) return (rows + h - 1) / h;
        const int64_t used = groups < rows ? groups : rows;
        return rows / h + (used + 1) / 2;
    };
    // L2 cycles of `count` steps that take in so many rows of A and of B; what HBM needs
    const int64_t a_cost = q.lda % 64 != 0 ? 308 : 283, b_cost = q.ldb % 64 != 0 ? 308 : 283;
    const int64_t inner = MODE == kWgrad ? q.M : q.R;
    const int64_t hbm = 2 * (rows * inner + inner * q.J * (MODE == kWgrad ? 1 : groups) +
                             rows * q.J * (MODE == kWgrad ? groups : 1)) / 2120;
    auto l2_of = [&](int64_t count, int64_t a_rows, int64_t b_rows) {
        return count * (a_rows * a_cost + b_rows * b_cost) / (100 * all);
    };
    auto step_of = [](int64_t tn, int64_t load) { return 2 * tn > load ? 2 * tn : load; };
    bool any = false;
    auto consider = [&](const LinearForm &f) {
        if (!any || f.cycles() < best->cycles()) *best = f;
        any = true;
    };
    static constexpr int kForms[4][2] = {{2, 256}, {2, 128}, {1, 256}, {1, 128}};
    for (const auto &f : kForms) {
        const int cg = f[0], tn = f[1];
        if (!(forms & (cg == 1 ? kSingles : tn == 256 ? kPairs : kNarrowPairs)) || sms < cg) continue;
        const int64_t tiles = tile_rows(128 * cg) * ((q.J + tn - 1) / tn);
        const int64_t rounds = (tiles + sms / cg - 1) / (sms / cg);
        const int64_t epilogue = cg == 2 ? 5340 + tn * 25 / 2 : 1690 + tn * 21;
        const int64_t tile = steps * step_of(tn, (128 + tn / cg) * 231 / 100);
        consider({cg, tn, 0, l2_of(tiles * cg * steps, 128, tn / cg), hbm, rounds * (tile > epilogue ? tile : epilogue),
                  epilogue * 6 / 10 + (cg == 2 ? 14400 : 4700)});
    }
    if (!(forms & kSplits) || (MODE == kWgrad && q.offsets != nullptr)) return any;
    const int64_t tm = split_tiles(q, MODE);
    const int box = split_row_box(q.M);
    const int64_t a_rows = MODE == kWgrad || rows > 96 ? 128 : (rows + box - 1) / box * box;
    for (int tn = 128; tn >= 48; tn -= 16) {
        if (MODE != kFwd && tn % 64 != 0) continue;
        const int64_t tiles = tm * ((q.J + tn - 1) / tn);
        for (int parts = 1; parts <= kMaxSplit && parts <= steps; ++parts) {
            if (room[parts] <= 0) continue;
            // one CTA on an SM while there are no more than SMs, two beyond; then further rounds
            const int64_t rounds = (tiles + room[parts] - 1) / room[parts];
            const int64_t mine = (steps + parts - 1) / parts;
            const int64_t load = (a_rows * 250 + tn * (MODE == kFwd ? 432 : 604)) / 100;
            int64_t step = step_of(tn, load) * (tiles * parts <= sms ? 1 : 2);
            const int64_t late = 2660 / split_stages(a_rows, tn);  // a load's way through the ring
            if (step < late) step = late;
            const int64_t exchange = parts > 1 ? 740 + 221 * parts : 0;
            const int64_t epilogue = 4190 + (rows < 128 ? rows : 128) * tn * 264 / (1000 * parts);
            consider({0, tn, parts, l2_of(tiles * steps, a_rows, tn), hbm, rounds * (mine * step + exchange + epilogue), 5330});
        }
    }
    return any;
}

template <int MODE>
static int lin_launch_form(const LinearProduct &q, const LinearForm &f, int dev, int sms, cudaStream_t stream) {
    if (f.cg == 0) return launch_linear_split(q, MODE, f.tn, f.parts, stream);
    if (f.cg == 2)
        return f.tn == 256 ? lin_launch<2, MODE, 256>(q, dev, sms, stream) : lin_launch<2, MODE, 128>(q, dev, sms, stream);
    return f.tn == 256 ? lin_launch<1, MODE, 256>(q, dev, sms, stream) : lin_launch<1, MODE, 128>(q, dev, sms, stream);
}

template <int MODE>
static int lin_dispatch(const LinearProduct &q, cudaStream_t stream) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const int sms = sm_count(dev);
    int room[kMaxSplit + 1];
    const int rc = split_room(MODE, dev, room);
    if (rc != TGC_OK) return rc;
    LinearForm f;
    if (!lin_choose<MODE>(q, sms, sms, room, kAllForms, &f)) return TGC_ERR_INVALID_ARG;
    // A last tile row that is mostly empty can cost a whole round.  Where the full rows' tiles leave
    // SMs idle, the rest of the rows go to the split kernel on those, at the same time: 777 x 4104 x
    // 5000 44 -> 36 us (45.6 -> 39.2 with a residual; kFwd only, kDgrad's MN-major weight made the rest
    // the longer part).
    const int64_t full = q.M / 256 * 256;
    if (MODE == kFwd && q.offsets == nullptr && full > 0 && full < q.M) {
        LinearProduct main = q, rest = q;
        main.M = full;
        rest.M = q.M - full;
        rest.early = 1;  // needs what the main part needs
        auto rows_on = [&](auto *p, int64_t ld) { return p == nullptr ? p : (decltype(p))((char *)p + full * ld * 2); };
        rest.a = rows_on(q.a, q.lda);
        rest.y = rows_on(q.y, q.ldy);
        rest.z = rows_on(q.z, q.ldz);
        rest.residual = rows_on(q.residual, q.ldres);
        LinearForm fm, fr;
        lin_choose<MODE>(main, sms, sms, room, kPairs, &fm);
        const int64_t tiles = full / 256 * ((q.J + 255) / 256);
        const int idle = sms - 2 * (int)(tiles < sms / 2 ? tiles : sms / 2);
        int there[kMaxSplit + 1] = {};
        for (int c = 1; c <= kMaxSplit; ++c) there[c] = room[c] < 2 * idle / c ? room[c] : 2 * idle / c;
        if (idle > 0 && lin_choose<MODE>(rest, sms, idle, there, kSplits, &fr)) {
            int64_t both = fm.bound();
            if (both < fm.l2 + fr.l2) both = fm.l2 + fr.l2;
            if (both < fr.sm / 2) both = fr.sm / 2;  // the weight comes from L2: the main part has read it
            both += (fm.extra > fr.extra ? fm.extra : fr.extra) + 2000;
            if (both * 11 / 10 < f.cycles()) {
                const int r = lin_launch_form<MODE>(main, fm, dev, sms, stream);
                return r != TGC_OK ? r : lin_launch_form<MODE>(rest, fr, dev, sms, stream);
            }
        }
    }
    return lin_launch_form<MODE>(q, f, dev, sms, stream);
}

int launch_linear(const LinearProduct &q, int mode, cudaStream_t stream) {
    if (mode == kFwd) return lin_dispatch<kFwd>(q, stream);
    if (mode == kDgrad) return lin_dispatch<kDgrad>(q, stream);
    return lin_dispatch<kWgrad>(q, stream);
}

}  // namespace tgc
