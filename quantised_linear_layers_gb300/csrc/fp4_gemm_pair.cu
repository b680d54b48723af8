// 4-bit product on CTA pairs (fp4_gemm.cuh): 256 x 256 tiles of D, the tensor
// cores of two SMs driven by one instruction stream (cta_group::2).
//
// X's rows are split over the pair (128 per CTA) and so are W's (128 of the
// 256 columns of D per CTA); each CTA's tensor memory holds the scales of its
// own X rows and of all W rows of the tile, in a slot for every stage of shared
// memory (five of 48 columns beside the accumulator's 256).
//
// What bounds it is an SM's shared memory at 128 bytes a cycle: a stage of 256
// columns writes 38 KB (nv; mx 35) by TMA, and the instructions read 32 KB of
// codes, the copies to tensor memory 6 KB (3) of scales: 608 cycles (560) for 512
// of the tensor core. Hence the widest instruction and tile (256 x 256; halves of
// 128 columns read X twice: 620 -> 700 us at 16384 x 18432 x 7168), with one
// accumulator, whose registers are read out in one go so that the next tile
// starts at once. Measured nv / mx: 8192 x 8192 x 7168 139 / 134 us (6.9 / 7.2
// PFLOP/s), 16384 x 18432 x 7168 606 / 565 us in a short run, 662 / 603 under the
// power cap; tensor pipe 79 / 81 % active.
//
// Roles (384 threads per CTA): warp 0 TMA producer, warp 1 of the leader MMA
// issuer, warps 4-11 epilogue (32 rows x 128 columns of D each, staged in
// shared memory and written by TMA tile stores; rows that end inside a warp's
// 32, as an expert's last ones do, are stored by the warp).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "common.cuh"
#include "epilogue_tma.cuh"
#include "fp4.cuh"
#include "fp4_gemm.cuh"
#include "gemm.cuh"

namespace ql {
namespace {

constexpr int kThreads = 384;
constexpr int kMathThreads = 256;
constexpr int BM = 128;          // rows of X per CTA
constexpr int BN = 256;          // rows of W per pair

template <int FMT>
struct PairCfg {
    static constexpr int kWords = FMT == kFp4Nv ? 4 : 2;
    static constexpr int kStageX = BM * 128;
    static constexpr int kStageW = BN / 2 * 128;
    static constexpr int kSfBox = kWords * kFp4SfBlock;           // 128 rows x 256 columns
    static constexpr int kStageSf = 3 * kSfBox;                   // X's own rows, W's two blocks
    static constexpr int kBytes = kStageX + kStageW + kStageSf;
    static constexpr int kStages = 5;
    static constexpr int kSlot = 12 * kWords;
    static constexpr int kSfCol = BN;
    static constexpr int kTmem = 512;
    static constexpr int kOutWarp = 32 * 128;
    static constexpr int kOffW = kStages * kStageX;
    static constexpr int kOffOut = kOffW + kStages * kStageW;
    static constexpr int kOffSf = kOffOut + 8 * kOutWarp;
    static constexpr int kOffBar = kOffSf + kStages * kStageSf;
    static constexpr int kOffOff = kOffBar + 256;
    static constexpr int kSmem = kOffOff + (kFp4MaxExperts + 1) * 4 + 12 + 1024;
    static_assert(kOffSf % 1024 == 0 && kSmem <= 232448, "shared memory");
    static_assert((2 * kStages + 3) * 8 + 16 <= 256, "barriers");
    static_assert(kSfCol + kStages * kSlot <= kTmem, "tensor memory");
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl)) != 0;
}

// Eight rows of 64 bf16 columns out of a warp's staging buffer (from its row
// r0, a multiple of 8) to rows of D that start on 4-byte boundaries.
__device__ __forceinline__ void store_pairs8(const uint8_t* stg, int r0, __nv_bfloat16* d, int64_t ldd, const Bounds& bnd) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        w[j] = *reinterpret_cast<const uint32_t*>(stg + (r0 + j) * 128 + (((lane >> 2) ^ j) << 4) + (lane & 3) * 4);
    d += 2 * lane;
#pragma unroll
    for (int j = 0; j < 8; ++j, d += ldd)
        if (QL_IN(bnd, 0, d, 4)) *reinterpret_cast<uint32_t*>(d) = w[j];
}

// The same rows stored by the warp itself, for rows that end inside its 32 and
// for a D that TMA cannot address: through the warp's staging buffer, so that
// a store instruction writes neighbouring columns of one row (a lane storing
// its own row would touch 32 rows at a time: 40 us instead of 10 at
// 512 x 1001 x 2051).
template <int CPT, bool OUT_F32>
__device__ __forceinline__ void store_warp_rows(const float* acc, uint8_t* stg, const Fp4GemmParams& p, int row0, int rows,
                                                int c0) {
    constexpr int CW = OUT_F32 ? 32 : 64;
    const int lane = static_cast<int>(threadIdx.x & 31);
    if (lane == 0) bulk_wait_read_all();          // an earlier tile store has read the buffer
    __syncwarp();
#pragma unroll
    for (int c = 0; c < CPT; c += CW) {
        if (c0 + c >= p.n) break;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint4 v;
            if constexpr (OUT_F32) {
                v = make_uint4(__float_as_uint(acc[c + 4 * k]), __float_as_uint(acc[c + 4 * k + 1]),
                               __float_as_uint(acc[c + 4 * k + 2]), __float_as_uint(acc[c + 4 * k + 3]));
            } else {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[c + 8 * k + 2 * e], acc[c + 8 * k + 2 * e + 1]);
                    h[e] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                v = make_uint4(h[0], h[1], h[2], h[3]);
            }
            *reinterpret_cast<uint4*>(stg + lane * 128 + ((k ^ (lane & 7)) << 4)) = v;
        }
        __syncwarp();
        const int64_t at = static_cast<int64_t>(row0) * p.ldd + c0 + c + lane;
        const bool in0 = c0 + c + lane < p.n;
        if constexpr (OUT_F32) {
            float* d = static_cast<float*>(p.d) + at;
#pragma unroll 4
            for (int r = 0; r < rows; ++r, d += p.ldd) {
                const float v = *reinterpret_cast<const float*>(stg + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                if (in0 && QL_IN(p.bnd, 0, d, 4)) *d = p.accumulate ? *d + v : v;
            }
        } else {
            __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.d) + at;
            int r = 0;
            // pairs of columns, if all rows start on 4-byte boundaries (2592 x 14540 x 96
            // 35.2 -> 27.6 us; with rows that start between two, whose ends are stores of
            // their own, 35.5 -> 58)
            if (c0 + c + CW <= p.n && (p.ldd & 1) == 0 && (reinterpret_cast<uintptr_t>(p.d) & 2u) == 0)
                for (; r + 8 <= rows; r += 8, d += 8 * p.ldd) store_pairs8(stg, r, d - lane, p.ldd, p.bnd);
            const bool in1 = c0 + c + lane + 32 < p.n;
#pragma unroll 4
            for (; r < rows; ++r, d += p.ldd) {
                const uint8_t* row = stg + r * 128 + (lane & 7) * 2;
                const __nv_bfloat16 v0 = *reinterpret_cast<const __nv_bfloat16*>(row + (((lane >> 3) ^ (r & 7)) << 4));
                const __nv_bfloat16 v1 = *reinterpret_cast<const __nv_bfloat16*>(row + (((4 + (lane >> 3)) ^ (r & 7)) << 4));
                if (in0 && QL_IN(p.bnd, 0, d, 2)) d[0] = v0;
                if (in1 && QL_IN(p.bnd, 0, d + 32, 2)) d[32] = v1;
            }
        }
        __syncwarp();
    }
}

template <int FMT, bool OUT_F32>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_sfx, const __grid_constant__ CUtensorMap map_sfw,
                         const __grid_constant__ CUtensorMap map_d, const Fp4GemmParams p) {
    using C = PairCfg<FMT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);   // leader: both CTAs' copies landed
    uint64_t* empty = full + C::kStages;                               // stage free (both CTAs)
    uint64_t* tfull = empty + C::kStages;                              // accumulator ready (both CTAs)
    uint64_t* tempty = tfull + 1;                                      // leader: both epilogues have read it
    uint64_t* done_bar = tempty + 1;
    uint32_t* tmem_base_sm = reinterpret_cast<uint32_t*>(done_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_sm + 1);
    volatile uint32_t* peer_issued = reinterpret_cast<volatile uint32_t*>(tmem_base_sm + 2);
    int* s_off = reinterpret_cast<int*>(smem + C::kOffOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int first = static_cast<int>(cluster_id_x()), step = static_cast<int>(num_clusters_x());

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        mbar_init(tfull, 1);
        mbar_init(tempty, 2 * kMathThreads);
        mbar_init(done_bar, 1);
        *peer_issued = 0;
        *abort_flag = 0;
        fence_mbar_init();
    }
    pdl_launch_dependents();
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_sfx);
        tma_prefetch_desc(&map_sfw);
    }
    if (warp == 1) { tmem_alloc_pair(tmem_base_sm, C::kTmem); tmem_relinquish_pair(); }
    pdl_wait_prior();
    if (warp == 2 && p.form != kFp4Plain) fp4_load_offsets(s_off, p);
    tc_fence_before_sync();
    cluster_sync_all();          // both CTAs' barriers exist before any remote arrive
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_base_sm;
    const WaitCtl ctl{abort_flag, p.dev_status, p.wait_limit_ns};
    uint32_t issued = 0;
    Fp4Walk<2 * BM, BN> walk;
    Fp4Tile t = {};

    if (warp < 4) {
        regs_dealloc<136>();     // 128 x 136 + 256 x 184 = 384 x 168 registers
        if (warp == 0) {
            if (elect_one()) {
                uint32_t it = 0;
                bool ok = true;
                const uint32_t leader_full0 = mapa_shared(&full[0], 0);
                for (int i = first; ok && walk.get(i, p, s_off, t) && !p.stall_producer; i += step) {
                    const int x_row = t.x_row + static_cast<int>(rank) * BM;
                    const int w_row = t.w_row + static_cast<int>(rank) * (BN / 2);
                    const int kbs = (t.k64 + 3) >> 2;
                    for (int kb = 0; kb < kbs; ++kb, ++it) {
                        const uint32_t s = it % C::kStages, ph = (it / C::kStages) & 1u;
                        if (!mbar_wait(&empty[s], ph ^ 1u, ctl)) { ok = false; break; }
                        if (leader) mbar_arrive_expect_tx(&full[s], 2 * C::kBytes);
                        const uint32_t bar = leader_full0 + s * 8u;
                        const int x = (t.k0 + kb) * 128, kblk = (t.k0 + kb) * C::kWords;
                        uint8_t* sf = smem + C::kOffSf + s * C::kStageSf;
                        tma_load_2d_pair(smem + s * C::kStageX, &map_x, bar, x, x_row);
                        tma_load_2d_pair(smem + C::kOffW + s * C::kStageW, &map_w, bar, x, w_row);
                        tma_load_2d_pair(sf, &map_sfx, bar, 0, ((t.x_blk + static_cast<int>(rank)) * p.kblocks + kblk) * 4);
                        tma_load_2d_pair(sf + C::kSfBox, &map_sfw, bar, 0, (t.w_blk * p.kblocks + kblk) * 4);
                        tma_load_2d_pair(sf + 2 * C::kSfBox, &map_sfw, bar, 0, ((t.w_blk + 1) * p.kblocks + kblk) * 4);
                    }
                }
                issued = it;
                if (!leader) st_shared_cluster(mapa_shared(const_cast<uint32_t*>(peer_issued), 0), it);
            }
            issued = __reduce_max_sync(0xffffffffu, issued);
        } else if (warp == 1 && leader) {
            if (elect_one()) {
                uint32_t it = 0, tc = 0;
                bool ok = true;
                for (int i = first; ok && walk.get(i, p, s_off, t); i += step) {
                    const int kbs = (t.k64 + 3) >> 2;
                    if (kbs == 0) continue;
                    if (!mbar_wait_cluster(tempty, (tc & 1u) ^ 1u, ctl)) { ok = false; break; }
                    tc_fence_after_sync();
                    for (int kb = 0; kb < kbs; ++kb, ++it) {
                        const uint32_t s = it % C::kStages;
                        if (!mbar_wait_cluster(&full[s], (it / C::kStages) & 1u, ctl)) { ok = false; break; }
                        tc_fence_after_sync();
                        const uint32_t sfx = tmem_base + C::kSfCol + s * C::kSlot;
                        const uint32_t sfw = sfx + 4 * C::kWords;      // per word: 4 columns of each W block
                        const uint32_t ps = smem_addr(smem + C::kOffSf + s * C::kStageSf);
#pragma unroll
                        for (int j = 0; j < C::kWords; ++j) {
                            tmem_cp_pair_32x128b_warpx4(sfx + 4 * j, rows16_desc(ps + j * kFp4SfBlock));
                            tmem_cp_pair_32x128b_warpx4(sfw + 8 * j, rows16_desc(ps + C::kSfBox + j * kFp4SfBlock));
                            tmem_cp_pair_32x128b_warpx4(sfw + 8 * j + 4, rows16_desc(ps + 2 * C::kSfBox + j * kFp4SfBlock));
                        }
                        const uint64_t dx = sw128_kmajor_desc(smem_addr(smem + s * C::kStageX));
                        const uint64_t dw = sw128_kmajor_desc(smem_addr(smem + C::kOffW + s * C::kStageW));
                        const int steps = t.k64 - 4 * kb;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j >= steps) break;
                            const int word = FMT == kFp4Nv ? j : j >> 1;
                            const uint32_t byte = FMT == kFp4Nv ? 0u : 2u * (j & 1);
                            mma_fp4<FMT, true>(tmem_base, dx + 2 * j, dw + 2 * j, idesc_fp4<FMT>(2 * BM, BN, byte),
                                               sfx + 4 * word, sfw + 8 * word, (kb > 0 || j > 0) ? 1u : 0u);
                        }
                        mma_commit_pair_multicast(&empty[s], 0x3);
                    }
                    if (!ok) break;
                    mma_commit_pair_multicast(tfull, 0x3);
                    ++tc;
                }
                mma_commit_pair_multicast(done_bar, 0x1);
                mbar_wait_drain(done_bar, 0, p.wait_limit_ns);
            }
            __syncwarp();
        } else if (warp >= 2 && p.zero_rest) {
            fp4_zero_rest<OUT_F32>(p, s_off);
        }
    } else {
        regs_alloc<184>();
        constexpr int CPT = BN / 2;
        const int wg = (warp - 4) >> 2, q = warp & 3;
        const uint32_t leader_tempty = mapa_shared(tempty, 0);
        const float alpha = (p.tx != nullptr ? __ldg(p.tx) : 1.0f) * (p.tw != nullptr ? __ldg(p.tw) : 1.0f);
        uint32_t tc = 0;
        for (int i = first; walk.get(i, p, s_off, t); i += step) {
            float acc[CPT];
            uint32_t(&bits)[CPT] = reinterpret_cast<uint32_t(&)[CPT]>(acc);
            if (t.k64 > 0) {
                if (!warp_wait(tfull, tc & 1u, ctl)) break;
                ++tc;
                tc_fence_after_sync();
                const uint32_t col = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + wg * CPT;
#pragma unroll
                for (int c = 0; c < CPT; c += 32) tmem_ld_32x32b_x32(col + c, reinterpret_cast<uint32_t(&)[32]>(bits[c]));
                tmem_wait_ld(bits);
                tc_fence_before_sync();
                if (leader) mbar_arrive(tempty);
                else mbar_arrive_remote_relaxed(leader_tempty);
            } else {
#pragma unroll
                for (int c = 0; c < CPT; ++c) acc[c] = 0.0f;
            }
#pragma unroll
            for (int c = 0; c < CPT; ++c) acc[c] *= alpha;
            const int in = static_cast<int>(rank) * BM + q * 32;       // first of the warp's rows in the tile
            const int left = t.rows - in;                              // rows of D from there
            const int c0 = t.col + wg * CPT;
            if (p.tma_d && left >= 32) {
                tma_store_warp_rows<CPT, 128, OUT_F32>(acc, smem + C::kOffOut + (warp - 4) * C::kOutWarp, &map_d, c0,
                                                       t.d_row + in, p.accumulate != 0);
            } else if (left > 0) {
                store_warp_rows<CPT, OUT_F32>(acc, smem + C::kOffOut + (warp - 4) * C::kOutWarp, p, t.d_row + in,
                                              left < 32 ? left : 32, c0);
            }
            __syncwarp();
        }
        if (p.tma_d && lane == 0) bulk_wait_all();     // the staged rows are written before the buffers go away
        __syncwarp();
    }

    tc_fence_before_sync();
    cluster_sync_all();          // every role of both CTAs has stopped issuing
    // Drain the copies that either CTA issued and nobody waited for: after a
    // time-out the producers may have stopped at different stages. A stage that
    // only the peer issued is armed now for the peer's bytes, one that only the
    // leader issued gives up the peer's share.
    if (leader && warp == 0 && lane == 0) {
        const uint32_t it_l = issued, it_p = *peer_issued;
        const uint32_t hi = it_l > it_p ? it_l : it_p;
        const uint32_t lo = hi > static_cast<uint32_t>(C::kStages) ? hi - C::kStages : 0u;
        for (uint32_t j = lo; j < hi; ++j) {
            const uint32_t s = j % C::kStages, ph = (j / C::kStages) & 1u;
            if (j >= it_l) mbar_arrive_expect_tx(&full[s], C::kBytes);
            else if (j >= it_p) mbar_complete_tx(&full[s], C::kBytes);
            mbar_wait_drain(&full[s], ph, p.wait_limit_ns);
        }
    }
    __syncwarp();
    cluster_sync_all();          // nothing of either CTA is in flight
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, C::kTmem);
    }
}

template <int FMT, bool OUT_F32>
cudaError_t launch_t(const Fp4GemmArgs& a, cudaStream_t st, int num_sms) {
    using C = PairCfg<FMT>;
    Fp4GemmParams p{};
    fp4_fill_params(a, p);
    p.tiles_x = static_cast<int>((a.m + 2 * BM - 1) / (2 * BM));
    p.tiles_w = static_cast<int>((a.n + BN - 1) / BN);
    // 32 tiles of rows before the next columns: W passes through L2 half as often
    // as with 8 (16384 x 18432 x 7168 under the power cap: nv 680 -> 662 us, mx
    // 620 -> 603; 4096 rows have 16 tiles and do not care)
    p.group_x = 32;
    CUtensorMap mx, mw, msx, msw, md = {};
    const int64_t kbytes = (a.k + 1) / 2;
    const int64_t we = a.form == kFp4RagRows ? a.experts : 1;
    const int64_t de = a.form == kFp4RagK ? a.experts : 1;
    if (!fp4_codes_map(&mx, a.x, a.m, kbytes, a.ldx, BM) || !fp4_codes_map(&mw, a.w, a.n * we, kbytes, a.ldw, BN / 2) ||
        !fp4_scales_map(&msx, a.sfx, a.x_row_blocks * p.kblocks, a.fmt) ||
        !fp4_scales_map(&msw, a.sfw, we * p.w_row_blocks * p.kblocks, a.fmt))
        return cudaErrorInvalidValue;
    constexpr int es = OUT_F32 ? 4 : 2;
    if (fp4_tma_d(a) &&
        encode_2d_map(&md, a.d, OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.m * de,
                      a.n, a.ldd * es, 32, 128 / es, 128))
        p.tma_d = 1;
    int64_t tiles = static_cast<int64_t>(p.tiles_x) * p.tiles_w;
    if (a.form == kFp4RagRows) tiles = (a.m / (2 * BM) + (a.experts < a.m ? a.experts : a.m)) * p.tiles_w;
    if (a.form == kFp4RagK) tiles *= a.experts;
    int64_t pairs = num_sms / 2 < 1 ? 1 : num_sms / 2;
    if (tiles < pairs) pairs = tiles;
    auto kern = fp4_gemm_pair_kernel<FMT, OUT_F32>;
    if (cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmem); e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int most = max_active_clusters(reinterpret_cast<const void*>(kern), cfg);
    if (pairs > most) pairs = most;
    return launch_gemm_kernel(kern, static_cast<unsigned>(2 * pairs), 2, C::kSmem, st, mx, mw, msx, msw, md, p);
}

}  // namespace

bool fp4_tma_d(const Fp4GemmArgs& a) {
    const int64_t es = a.out_f32 ? 4 : 2;
    return (reinterpret_cast<uintptr_t>(a.d) & 15u) == 0 && (a.ldd * es) % 16 == 0 && (a.n * es) % 16 == 0;
}

cudaError_t launch_fp4_gemm_pair(const Fp4GemmArgs& a, cudaStream_t st, int num_sms) {
    if (a.fmt == kFp4Nv)
        return a.out_f32 ? launch_t<kFp4Nv, true>(a, st, num_sms) : launch_t<kFp4Nv, false>(a, st, num_sms);
    return a.out_f32 ? launch_t<kFp4Mx, true>(a, st, num_sms) : launch_t<kFp4Mx, false>(a, st, num_sms);
}

}  // namespace ql
