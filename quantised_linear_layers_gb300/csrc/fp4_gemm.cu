// 4-bit product on one SM per tile (fp4_gemm.cuh), for few rows of D, narrow
// tiles and experts with few rows each.
//
// The tile is 128 columns of D by NT rows: W's rows take the tensor core's 128
// lanes and X's rows its N side, so that a single token costs one 16-wide
// instruction and no lane idles, and a tile's rows can end anywhere: the
// accumulator's lanes are D's columns, so one store instruction of a warp
// writes 32 neighbouring columns of one row, and rows past a tile's end are
// simply not stored. With few rows the time is the stream of W from HBM, with
// many tiles the tensor core's; a K stage is 256 columns (128 bytes) of both
// operands and their scale blocks, all by TMA onto one barrier.
//
// With too few tiles for the SMs a cluster of 2, 4 or 8 CTAs takes one tile,
// each a part of K; the fp32 partial tiles meet in shared memory, and each CTA
// sums and stores its share of the rows in the CTAs' order.
//
// (Storing the partial rows straight into their owner's shared memory, with an
// mbarrier in place of the first cluster barrier, was slower: 64 x 4096 x 7168
// 8.6 us against 7.8.)
//
// Up to 8 rows of X, 16 with experts (fp4_cast_rows), can come as they are, bf16 or fp32: eight
// more warps then cast them into the stages, a warp taking every eighth stage,
// and the call is a single launch. Every CTA repeats the cast of its part of K
// while its weights are on their way. At 4096 x 7168 (us, weights from HBM)
// one row takes 7.6 cast inside and 8.8 with a launch for the cast, 8 rows 8.4
// and 9.2, 16 rows 9.5 and 9.2, 64 rows 15.2 and 10.5.
//
// Measured against 4096 x 7168, nv, weights from HBM: 1 row 6.4 us, 16 rows 6.7,
// 64 7.7, 128 8.9, 256 10.6; the weight alone is 2.4 us of HBM. 512 x 512 x 512
// takes 3.8 us, 16 rows over 8 experts of 4096 x 7168 24 us (5.5 TB/s).
//
// Roles (256 or 384 threads, 256 more with the cast): warp 0 TMA producer, warp 1 MMA issuer (tcgen05.cp of a
// stage's scales into tensor memory, then up to four instructions of K = 64),
// four or eight epilogue warps from warp 4 on. Tensor memory holds two accumulators and a scale slot for
// every stage of shared memory, so that a stage that has landed can be issued:
// the instructions that read its slot before are those that freed it.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "bounds.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "fp4_gemm.cuh"
#include "gemm.cuh"

namespace ql {
namespace {

constexpr int kCastWarps = 8;                // a warp casts every eighth stage
constexpr int TW = 128;

template <int NT, int FMT>
struct Cfg {
    static constexpr int kWords = FMT == kFp4Nv ? 4 : 2;          // scale blocks along a stage
    static constexpr int kStageW = TW * 128;
    static constexpr int kStageX = NT * 128;
    static constexpr int kStageSf = kWords * kFp4SfBlock;         // per operand
    static constexpr int kBytes = kStageW + kStageX + 2 * kStageSf;
    // epilogue warps: two per lane quarter, each with half the rows, or one when there are 16
    static constexpr int kEpiWarps = NT >= 64 ? 8 : 4;
    static constexpr int kThreads = 128 + 32 * kEpiWarps;
    static constexpr int kSlot = 8 * kWords;                      // tensor-memory columns of a stage's scales
    static constexpr int kSfCol = NT < 32 ? 64 : 2 * NT;          // accumulators at 0 and NT
    static constexpr int kTmem = 512;
    static constexpr int kMisc = 2304;                            // barriers, offsets
    static constexpr int kMaxStages = (232448 - 1024 - kMisc) / kBytes;
    static constexpr int kStages = kMaxStages > 8 ? 8 : kMaxStages;
    static constexpr int kOffX = kStages * kStageW;
    static constexpr int kOffSfw = kOffX + kStages * kStageX;
    static constexpr int kOffSfx = kOffSfw + kStages * kStageSf;
    static constexpr int kOffBar = kOffSfx + kStages * kStageSf;
    static constexpr int kOffOff = kOffBar + 192;
    static constexpr int kSmem = kOffBar + kMisc + 1024;
    static_assert((2 * kStages + 5) * 8 + 16 <= 192, "barriers");
    static_assert(kSfCol + kStages * kSlot <= kTmem, "tensor memory");
    static_assert(192 + (kFp4MaxExperts + 1) * 4 <= kMisc, "offsets");
    static_assert(kStageX % 1024 == 0 && kSmem <= 232448, "shared memory");
    static_assert(NT * TW * 4 <= kOffSfw, "partial tile fits in the operand ring");
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl)) != 0;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

template <bool OUT_F32>
__device__ __forceinline__ void store_one(const Fp4GemmParams& p, int64_t at, float v) {
    if constexpr (OUT_F32) {
        float* d = static_cast<float*>(p.d) + at;
        if (QL_IN(p.bnd, 0, d, 4)) *d = p.accumulate ? *d + v : v;
    } else {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.d) + at;
        if (QL_IN(p.bnd, 0, d, 2)) *d = __float2bfloat16_rn(v);
    }
}

// Sixteen rows of one column of D (the first `rows` of them). The whole case
// has no branch between its stores: a lone warp per scheduler would otherwise
// wait out every address and conversion (measured 100 cycles a row).
template <bool OUT_F32>
__device__ __forceinline__ void store_rows(const Fp4GemmParams& p, int64_t at, int rows, const uint32_t (&r)[16],
                                           float alpha) {
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]) * alpha;
    if (rows >= 16) {
        if constexpr (OUT_F32) {
            float* d = static_cast<float*>(p.d) + at;
            if (p.accumulate) {
                const float* s = d;
#pragma unroll
                for (int j = 0; j < 16; ++j, s += p.ldd)
                    if (QL_IN(p.bnd, 0, s, 4)) v[j] += *s;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j, d += p.ldd)
                if (QL_IN(p.bnd, 0, d, 4)) *d = v[j];
        } else {
            __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.d) + at;
#pragma unroll
            for (int j = 0; j < 16; ++j, d += p.ldd)
                if (QL_IN(p.bnd, 0, d, 2)) *d = __float2bfloat16_rn(v[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j, at += p.ldd)
            if (j < rows) store_one<OUT_F32>(p, at, v[j]);
    }
}

// This CTA's share of the rows of a tile split along K: the CTAs' partial
// tiles (fp32 [NT][128] at the same offset of each CTA's shared memory) added
// in the CTAs' order. A thread takes four columns of a row and has the loads of
// kAhead rows in flight.
template <int NT, bool OUT_F32>
__device__ __forceinline__ void sum_parts(uint32_t part, const Fp4GemmParams& p, const Fp4Tile& t, int rank, int split) {
    constexpr int kAhead = 4, kRowsPer = 4 + (NT >= 64 ? 8 : 4);
    const float alpha = (p.tx != nullptr ? __ldg(p.tx) : 1.0f) * (p.tw != nullptr ? __ldg(p.tw) : 1.0f);
    const int c4 = (threadIdx.x & 31) * 4, col = t.col + c4;
    const int rows = t.rows < NT ? t.rows : NT;
    const int lo = rows * rank / split, hi = rows * (rank + 1) / split;
    if (col >= p.n) return;
    for (int r0 = lo + static_cast<int>(threadIdx.x >> 5); r0 < hi; r0 += kRowsPer * kAhead) {
        float4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < split; ++s) {
            uint32_t base;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base) : "r"(part), "r"(s));
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int row = r0 + j * kRowsPer;
                if (row >= hi) continue;
                const float4 o = ld_cluster_f32x4(base + (row * TW + c4) * 4);
                v[j].x += o.x; v[j].y += o.y; v[j].z += o.z; v[j].w += o.w;
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = r0 + j * kRowsPer;
            if (row >= hi) continue;
            const int64_t at = static_cast<int64_t>(t.d_row + row) * p.ldd + col;
            const float f[4] = {v[j].x * alpha, v[j].y * alpha, v[j].z * alpha, v[j].w * alpha};
            if (!OUT_F32 && p.vec_store && col + 4 <= p.n) {
                const __nv_bfloat162 h0 = __floats2bfloat162_rn(f[0], f[1]), h1 = __floats2bfloat162_rn(f[2], f[3]);
                if (QL_IN(p.bnd, 0, static_cast<__nv_bfloat16*>(p.d) + at, 8))
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.d) + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < p.n) store_one<OUT_F32>(p, at + e, f[e]);
            }
        }
    }
}

// One stage of X cast in place of its copy: its rows' 256 columns from column
// c0 on, codes in the 128-byte swizzle the tensor core reads, scale bytes in a
// scale block's order. A lane has 16 columns of a row, a warp two rows.
template <typename T, int FMT>
__device__ __forceinline__ void cast_stage(const Fp4GemmParams& p, int x_row, int rows, int c0, uint8_t* codes,
                                           uint8_t* sf, const Fp4Tensor& tn) {
    constexpr int kAhead = 4;                    // pairs of rows in flight
    const int lane = static_cast<int>(threadIdx.x & 31), cg = lane & 15;
    const int c = c0 + cg * 16;
    const T* x = static_cast<const T*>(p.xr) + static_cast<int64_t>(x_row) * p.sxr;
    for (int rb = 0; rb < rows; rb += 2 * kAhead) {
        Raw16<T> raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = rb + 2 * i + (lane >> 4);
            if (r >= rows || c >= p.k) raw[i].zero();
            else if (p.xr_vec && c + 16 <= p.k) raw[i].load(x + r * p.sxr + c, p.bnd, 2);
            else raw[i].load_some(x + r * p.sxr + c, 1, p.k - c < 16 ? p.k - c : 16, p.bnd, 2);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = rb + 2 * i + (lane >> 4);
            if (rb + 2 * i >= rows) break;
            float amax = raw[i].amax();
            if constexpr (FMT == kFp4Mx) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            const Fp4Scale g = fp4_scale<FMT>(amax, tn);
            uint64_t v[8];
            raw[i].values(v);
            *reinterpret_cast<uint2*>(codes + r * 128 + (((cg >> 1) ^ (r & 7)) << 4) + (cg & 1) * 8) = fp4_codes16<FMT>(v, g);
            const int gi = FMT == kFp4Nv ? cg : cg >> 1;
            if (FMT == kFp4Nv || (cg & 1) == 0) {
                const bool live = c0 + gi * fp4_group(FMT) < p.k;
                sf[(gi >> 2) * kFp4SfBlock + r * 16 + (gi & 3)] = live ? static_cast<uint8_t>(g.byte) : 0;
            }
        }
    }
}

// T: void when X's codes are copied, else the type of X to cast. SPLIT: a
// cluster of CTAs per tile, one tile per cluster.
template <int NT, int FMT, bool OUT_F32, typename T, bool SPLIT>
__global__ void __launch_bounds__(Cfg<NT, FMT>::kThreads + (std::is_void<T>::value ? 0 : 32 * kCastWarps), 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_sfx, const __grid_constant__ CUtensorMap map_sfw,
                    const Fp4GemmParams p) {
    using C = Cfg<NT, FMT>;
    constexpr bool kCast = !std::is_void<T>::value;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* empty = full + C::kStages;
    uint64_t* tfull = empty + C::kStages;       // [2]
    uint64_t* tempty = tfull + 2;               // [2]
    uint64_t* done_bar = tempty + 2;
    uint32_t* tmem_base_sm = reinterpret_cast<uint32_t*>(done_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_sm + 1);
    int* s_off = reinterpret_cast<int*>(smem + C::kOffOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = SPLIT ? static_cast<int>(cluster_nctarank()) : 1;
    const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = SPLIT ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
    const int step = SPLIT ? static_cast<int>(num_clusters_x()) : static_cast<int>(gridDim.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) { mbar_init(&full[s], kCast ? 2 : 1); mbar_init(&empty[s], 1); }
        for (int s = 0; s < 2; ++s) { mbar_init(&tfull[s], 1); mbar_init(&tempty[s], 32 * C::kEpiWarps); }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    pdl_launch_dependents();
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_sfw);
        if constexpr (!kCast) {
            tma_prefetch_desc(&map_x);
            tma_prefetch_desc(&map_sfx);
        }
        if (p.form == kFp4Plain && first < p.tiles_x * p.tiles_w) {
            // the first tile's part of W into L2 while the previous kernel ends
            // (a prefetch, not a load: that kernel may still be writing W)
            Fp4Walk<NT, TW> ahead;
            Fp4Tile f = {};
            ahead.get(first, p, s_off, f);
            const int kb = (f.k64 + 3) >> 2;
            const int lo = rank * kb / split, hi = (rank + 1) * kb / split;
            for (int i = lo; i < hi && i < lo + p.ahead; ++i) tma_prefetch_l2_2d(&map_w, i * 128, f.w_row);
        }
    }
    if (warp == 1) { tmem_alloc(tmem_base_sm, C::kTmem); tmem_relinquish(); }
    pdl_wait_prior();
    if (warp == 2 && p.form != kFp4Plain) fp4_load_offsets(s_off, p);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_base_sm;
    const WaitCtl ctl{abort_flag, p.dev_status, p.wait_limit_ns};

    Fp4Walk<NT, TW> walk;
    Fp4Tile t = {};
    // this CTA's stages of a tile: [k_lo, k_hi) of its steps of 256
    auto stages = [&](int& lo, int& hi) {
        const int kb = (t.k64 + 3) >> 2;
        lo = static_cast<int>(static_cast<int64_t>(rank) * kb / split);
        hi = static_cast<int>(static_cast<int64_t>(rank + 1) * kb / split);
    };

    if (warp == 0) {
        if (elect_one()) {
            uint32_t it = 0;
            bool ok = true;
            for (int i = first; ok && walk.get(i, p, s_off, t) && !p.stall_producer; i += step) {
                int lo, hi;
                stages(lo, hi);
                for (int kb = lo; kb < hi; ++kb, ++it) {
                    const uint32_t s = it % C::kStages, ph = (it / C::kStages) & 1u;
                    if (!mbar_wait(&empty[s], ph ^ 1u, ctl)) { ok = false; break; }
                    mbar_arrive_expect_tx(&full[s], kCast ? C::kStageW + C::kStageSf : C::kBytes);
                    const int x = (t.k0 + kb) * 128, kblk = (t.k0 + kb) * C::kWords;
                    tma_load_2d(smem + s * C::kStageW, &map_w, &full[s], x, t.w_row);
                    tma_load_2d(smem + C::kOffSfw + s * C::kStageSf, &map_sfw, &full[s], 0, (t.w_blk * p.kblocks + kblk) * 4);
                    if constexpr (!kCast) {
                        tma_load_2d(smem + C::kOffX + s * C::kStageX, &map_x, &full[s], x, t.x_row);
                        tma_load_2d(smem + C::kOffSfx + s * C::kStageSf, &map_sfx, &full[s], 0,
                                    (t.x_blk * p.kblocks + kblk) * 4);
                    }
                }
            }
            if (!ok) {
                const uint32_t from = it > static_cast<uint32_t>(C::kStages) ? it - C::kStages : 0u;
                for (uint32_t j = from; j < it; ++j)
                    mbar_wait_drain(&full[j % C::kStages], (j / C::kStages) & 1u, p.wait_limit_ns);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            uint32_t it = 0, tc = 0;
            bool ok = true;
            for (int i = first; ok && walk.get(i, p, s_off, t); i += step) {
                int lo, hi;
                stages(lo, hi);
                if (hi <= lo) continue;
                const uint32_t as = tc & 1u;
                if (!mbar_wait(&tempty[as], ((tc >> 1) & 1u) ^ 1u, ctl)) { ok = false; break; }
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + as * NT;
                const uint32_t x_col = NT < 128 ? static_cast<uint32_t>(t.x_sub >> 5) : 0u;
                for (int kb = lo; kb < hi; ++kb, ++it) {
                    const uint32_t s = it % C::kStages;
                    if (!mbar_wait(&full[s], (it / C::kStages) & 1u, ctl)) { ok = false; break; }
                    tc_fence_after_sync();
                    const uint32_t sfw = tmem_base + C::kSfCol + s * C::kSlot;
                    const uint32_t sfx = sfw + 4 * C::kWords;
                    const uint32_t pw = smem_addr(smem + C::kOffSfw + s * C::kStageSf);
                    const uint32_t px = smem_addr(smem + C::kOffSfx + s * C::kStageSf);
#pragma unroll
                    for (int j = 0; j < C::kWords; ++j) {
                        tmem_cp_32x128b_warpx4(sfw + 4 * j, rows16_desc(pw + j * kFp4SfBlock));
                        tmem_cp_32x128b_warpx4(sfx + 4 * j, rows16_desc(px + j * kFp4SfBlock));
                    }
                    const uint64_t dw = sw128_kmajor_desc(smem_addr(smem + s * C::kStageW));
                    const uint64_t dx = sw128_kmajor_desc(smem_addr(smem + C::kOffX + s * C::kStageX));
                    const int steps = t.k64 - 4 * kb;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= steps) break;
                        const int word = FMT == kFp4Nv ? j : j >> 1;
                        const uint32_t byte = FMT == kFp4Nv ? 0u : 2u * (j & 1);
                        mma_fp4<FMT, false>(d_tmem, dw + 2 * j, dx + 2 * j, idesc_fp4<FMT>(TW, NT, byte), sfw + 4 * word,
                                            sfx + 4 * word + x_col, (kb > lo || j > 0) ? 1u : 0u);
                    }
                    mma_commit(&empty[s]);
                }
                if (!ok) break;
                mma_commit(&tfull[as]);
                ++tc;
            }
            mma_commit(done_bar);
            mbar_wait_drain(done_bar, 0, p.wait_limit_ns);
        }
        __syncwarp();
    } else if (warp >= 4 + C::kEpiWarps) {
        if constexpr (kCast) {
            const Fp4Tensor tn = fp4_tensor(p.tx);
            uint32_t it = 0;
            bool ok = true;
            for (int i = first; ok && walk.get(i, p, s_off, t); i += step) {
                int lo, hi;
                stages(lo, hi);
                const int rows = t.rows < NT ? t.rows : NT;
                for (int kb = lo; kb < hi; ++kb, ++it) {
                    if (static_cast<int>(it % kCastWarps) != warp - (4 + C::kEpiWarps)) continue;
                    const uint32_t s = it % C::kStages, ph = (it / C::kStages) & 1u;
                    if (!warp_wait(&empty[s], ph ^ 1u, ctl)) { ok = false; break; }
                    cast_stage<T, FMT>(p, t.x_row, rows, kb * 256, smem + C::kOffX + s * C::kStageX,
                                       smem + C::kOffSfx + s * C::kStageSf, tn);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[s]);
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int q = warp & 3;
        constexpr int kPart = NT / (C::kEpiWarps / 4);               // rows of the tile this warp stores
        const int part0 = (warp - 4) / 4 * kPart;
        const float alpha = (p.tx != nullptr ? __ldg(p.tx) : 1.0f) * (p.tw != nullptr ? __ldg(p.tw) : 1.0f);
        uint32_t tc = 0;
        for (int n = first; walk.get(n, p, s_off, t); n += step) {
            int lo, hi;
            stages(lo, hi);
            const bool any = hi > lo;
            const uint32_t as = tc & 1u;
            if (any) {
                if (!warp_wait(&tfull[as], (tc >> 1) & 1u, ctl)) break;
                tc_fence_after_sync();
                ++tc;
            }
            const int col = t.col + q * 32 + lane;
            const int rows = t.rows < NT ? t.rows : NT;
#pragma unroll
            for (int i = 0; i < kPart; i += 16) {
                const int c0 = part0 + i;
                if (c0 >= rows) break;
                uint32_t r[16];
                if (any) {
                    tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + as * NT + c0, r);
                    tmem_wait_ld(r);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] = 0u;
                }
                if constexpr (SPLIT) {
                    float* part = reinterpret_cast<float*>(smem);      // the operand ring, done with
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c0 + j) * TW + q * 32 + lane] = __uint_as_float(r[j]);
                } else if (col < p.n) {
                    store_rows<OUT_F32>(p, static_cast<int64_t>(t.d_row + c0) * p.ldd + col, rows - c0, r, alpha);
                }
            }
            tc_fence_before_sync();
            if (any) mbar_arrive(&tempty[as]);
        }
    } else {
        if constexpr (!SPLIT)                    // (a product of experts is never split)
            if (p.zero_rest) fp4_zero_rest<OUT_F32>(p, s_off);
    }
    if constexpr (SPLIT) {
        // one tile per cluster: the partial tiles are in every CTA's shared memory
        __syncwarp();
        cluster_sync_all();
        Fp4Walk<NT, TW> again;
        if (warp < 4 + C::kEpiWarps && again.get(first, p, s_off, t) && !*abort_flag)
            sum_parts<NT, OUT_F32>(smem_addr(smem), p, t, rank, split);
        __syncwarp();
        cluster_sync_all();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, C::kTmem);
    }
}

// CTAs per tile of a plain product. A cluster costs about as much as some
// stages of K (measured on 1 x 1024, 64 x 1024 and 128 x 1024 columns with K
// from 512 to 4096, where a stage takes 0.23 us); the cheapest of 1, 2, 4 and 8
// that fit on the SMs is taken. In tenths of a stage.
template <int NT>
int choose_split(int64_t tiles, int64_t kb, int num_sms) {
    constexpr int cost[4] = {0, NT <= 16 ? 43 : (NT <= 64 ? 64 : 94), NT <= 16 ? 51 : (NT <= 64 ? 72 : 115),
                             NT <= 16 ? 51 : (NT <= 64 ? 85 : 149)};
    int best = 1;
    int64_t least = 10 * kb;
    for (int i = 1, s = 2; i < 4 && tiles * s <= num_sms && s <= kb; ++i, s *= 2) {
        const int64_t c = 10 * ((kb + s - 1) / s) + cost[i];
        if (c < least) {
            least = c;
            best = s;
        }
    }
    return best;
}

template <int NT, int FMT, bool OUT_F32, typename T, bool SPLIT>
cudaError_t launch_s(const Fp4GemmArgs& a, Fp4GemmParams& p, int64_t tiles, int split, cudaStream_t st, int num_sms) {
    using C = Cfg<NT, FMT>;
    constexpr bool kCast = !std::is_void<T>::value;
    CUtensorMap mx, mw, msx, msw;
    const int64_t kbytes = (a.k + 1) / 2;
    const int64_t we = a.form == kFp4RagRows ? a.experts : 1;
    if constexpr (kCast) {
        mx = msx = CUtensorMap{};
    } else if (!fp4_codes_map(&mx, a.x, a.m, kbytes, a.ldx, NT) ||
               !fp4_scales_map(&msx, a.sfx, a.x_row_blocks * p.kblocks, a.fmt)) {
        return cudaErrorInvalidValue;
    }
    if (!fp4_codes_map(&mw, a.w, a.n * we, kbytes, a.ldw, TW) ||
        !fp4_scales_map(&msw, a.sfw, we * p.w_row_blocks * p.kblocks, a.fmt))
        return cudaErrorInvalidValue;
    auto kern = fp4_gemm_kernel<NT, FMT, OUT_F32, T, SPLIT>;
    if (cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmem); e != cudaSuccess) return e;
    const int64_t grid = SPLIT ? tiles * split : (tiles < num_sms ? tiles : num_sms);
    // at most 64 MB of W ahead over the grid, well inside L2
    p.ahead = static_cast<int>((int64_t(64) << 20) / (grid * C::kStageW));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(C::kThreads + (kCast ? 32 * kCastWarps : 0), 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, mx, mw, msx, msw, p);
}

template <int NT, int FMT, bool OUT_F32, typename T = void>
cudaError_t launch_t(const Fp4GemmArgs& a, cudaStream_t st, int num_sms) {
    Fp4GemmParams p{};
    fp4_fill_params(a, p);
    p.tiles_x = static_cast<int>((a.m + NT - 1) / NT);
    p.tiles_w = static_cast<int>((a.n + TW - 1) / TW);
    p.group_x = 16;
    p.vec_store = (reinterpret_cast<uintptr_t>(a.d) & 7u) == 0 && a.ldd % 4 == 0;
    if constexpr (!std::is_void<T>::value) {
        p.xr = a.xr;
        p.sxr = a.sxr;
        p.k = static_cast<int>(a.k);
        p.xr_vec = (reinterpret_cast<uintptr_t>(a.xr) & 15u) == 0 && (a.sxr * (a.xr_bf16 ? 2 : 4)) % 16 == 0;
    }
    int64_t tiles = static_cast<int64_t>(p.tiles_x) * p.tiles_w;
    if (a.form == kFp4Plain) {
        const int split = choose_split<NT>(tiles, (a.k + 255) / 256, num_sms);
        if (split > 1) return launch_s<NT, FMT, OUT_F32, T, true>(a, p, tiles, split, st, num_sms);
    }
    if (a.form == kFp4RagRows) tiles = (a.m / NT + (a.experts < a.m ? a.experts : a.m)) * p.tiles_w;
    if (a.form == kFp4RagK) tiles *= a.experts;
    return launch_s<NT, FMT, OUT_F32, T, false>(a, p, tiles, 1, st, num_sms);
}

template <int NT>
cudaError_t launch_n(const Fp4GemmArgs& a, cudaStream_t st, int num_sms) {
    if (a.fmt == kFp4Nv)
        return a.out_f32 ? launch_t<NT, kFp4Nv, true>(a, st, num_sms) : launch_t<NT, kFp4Nv, false>(a, st, num_sms);
    return a.out_f32 ? launch_t<NT, kFp4Mx, true>(a, st, num_sms) : launch_t<NT, kFp4Mx, false>(a, st, num_sms);
}

template <int NT>
cudaError_t launch_cast(const Fp4GemmArgs& a, cudaStream_t st, int num_sms) {
    if (a.xr_bf16)
        return a.fmt == kFp4Nv ? launch_t<NT, kFp4Nv, false, __nv_bfloat16>(a, st, num_sms)
                               : launch_t<NT, kFp4Mx, false, __nv_bfloat16>(a, st, num_sms);
    return a.fmt == kFp4Nv ? launch_t<NT, kFp4Nv, false, float>(a, st, num_sms)
                           : launch_t<NT, kFp4Mx, false, float>(a, st, num_sms);
}

}  // namespace

bool fp4_codes_map(CUtensorMap* map, const uint8_t* q, int64_t rows, int64_t kbytes, int64_t ld, int box_rows) {
    return encode_kmajor_map(map, q, rows, kbytes, ld, box_rows);
}

bool fp4_scales_map(CUtensorMap* map, const uint8_t* sf, int64_t blocks, int fmt) {
    return encode_2d_map(map, sf, CU_TENSOR_MAP_DATA_TYPE_UINT8, blocks * 4, 128, 128, fmt == kFp4Nv ? 16 : 8, 128, 0);
}

void fp4_fill_params(const Fp4GemmArgs& a, Fp4GemmParams& p) {
    p.form = a.form;
    p.experts = a.experts;
    p.m = static_cast<int>(a.m);
    p.n = static_cast<int>(a.n);
    p.k64 = static_cast<int>((a.k + 63) / 64);
    p.rows = static_cast<int>(a.rows);
    p.kblocks = static_cast<int>(fp4_kblocks(a.k, a.fmt));
    p.w_row_blocks = static_cast<int>((a.n + 127) / 128);
    p.offsets = a.offsets;
    p.tx = a.tx;
    p.tw = a.tw;
    p.d = a.d;
    p.ldd = a.ldd;
    p.accumulate = a.accumulate;
    p.zero_rest = a.form == kFp4RagRows && a.zero_rest;
    p.dev_status = a.dev_status;
    p.wait_limit_ns = a.wait_limit_ns;
    p.stall_producer = a.stall_producer;
    // what the kernels read and write with plain loads and stores
    const int64_t drows = a.m * (a.form == kFp4RagK ? a.experts : 1);
    p.bnd.s[0] = span_of(a.d, a.out_f32 ? 4 : 2, drows, a.ldd, a.n, 1);
    p.bnd.s[1] = span_of(a.offsets, 4, a.experts + 1, 1);
    p.bnd.s[2] = span_of(a.xr, a.xr_bf16 ? 2 : 4, a.m, a.sxr, a.k, 1);
    p.bnd.status = a.dev_status;
}

cudaError_t launch_fp4_gemm(const Fp4GemmArgs& a, cudaStream_t st, int num_sms) {
    if (a.xr != nullptr) return launch_cast<16>(a, st, num_sms);
    if (a.m <= 16) return launch_n<16>(a, st, num_sms);
    // narrow tiles as long as one covers an expert's rows on average (64 / 128 wide:
    // 2000 rows over 32 experts of 1024 x 1024 8.4 / 8.7 us, 512 over 8 of 4096 x
    // 7168 25.6 / 25.6; plain, 64 rows against 4096 x 7168 7.7 / 9.0)
    const int64_t per = a.form == kFp4RagRows ? a.m / a.experts : a.m;
    if (per <= 64) return launch_n<64>(a, st, num_sms);
    return launch_n<128>(a, st, num_sms);
}

}  // namespace ql
