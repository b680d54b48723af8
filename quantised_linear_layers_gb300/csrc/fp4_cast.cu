// Casts to and from the microscaled 4-bit formats of fp4.cuh.
//
//   fp4_cast_kernel     rows of x to codes and block-ordered scales
//   fp4_dual_kernel     rows and columns of x from one read (training)
//   fp4_dequant_kernel  codes and scales back to bf16 or fp32
//   fp4_tscale_kernel   the power of two t of a tensor (nv)
//
// All are bound by HBM: the least traffic per element is its input bytes plus
// 0.5 + 1/16 (nv) or 0.5 + 1/32 (mx) written, twice that for both
// orientations.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "gemm.cuh"

namespace ql {
namespace {

constexpr int kThreads = 256;

// Position of `row` among the experts' 128-row scale blocks: its row in the
// padded order, or -1 if no expert has it. The whole warp calls it.
__device__ __forceinline__ int64_t expert_sf_row(const int32_t* offsets, int experts, int64_t m, int64_t row) {
    const int lane = threadIdx.x & 31;
    int blocks = 0;             // blocks of the experts that end at or before the row
    int start = -1;
    for (int e0 = 0; e0 < experts; e0 += 32) {
        const int e = e0 + lane;
        int b = 0, s = -1;
        if (e < experts) {
            const int64_t lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
            if (hi <= row) b = static_cast<int>((hi - lo + 127) / 128);
            else if (lo <= row) s = static_cast<int>(lo);
        }
        blocks += __reduce_add_sync(0xffffffffu, b);
        start = max(start, __reduce_max_sync(0xffffffffu, s));
        if (start >= 0) break;
    }
    if (start < 0) return -1;
    return static_cast<int64_t>(blocks) * 128 + (row - start);
}

// One warp takes a row's 512-column pieces, U of them at a time (their loads
// are all issued before the first is used); each lane has 16 consecutive
// columns: an nv group, or half an mx group whose other half is the next
// lane's. VEC: 16-byte loads along contiguous rows; otherwise element loads
// with any strides. Rows are taken in the order of the scale blocks' sectors
// (rows r, r+32, r+64, r+96 of a block are neighbours there).
template <typename T, int FMT, bool VEC, int U>
__global__ void __launch_bounds__(kThreads) fp4_cast_kernel(const Fp4CastArgs p) {
    pdl_launch_dependents();
    pdl_wait_prior();
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    const int64_t kblocks = fp4_kblocks(p.k, FMT);
    const int pieces = static_cast<int>((p.k + 511) / 512);
    const int steps = (pieces + U - 1) / U;
    const int64_t seg_blocks = (p.seg_rows + 127) / 128;
    const int64_t segs = p.seg_rows > 0 ? (p.m / p.seg_rows) : 1;
    const int64_t rows = p.offsets != nullptr ? p.m : segs * seg_blocks * 128;   // rows in the order taken
    const Fp4Tensor tn = fp4_tensor(p.tscale);
    const int64_t tasks = rows * steps;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); t < tasks; t += nwarps) {
        // eight rows (one 32-byte sector of a scale block) side by side, then the next columns
        const int64_t r8 = t / (8 * steps);
        const int in8 = static_cast<int>(t % (8 * steps));
        int64_t ro, sf_row, row;
        int step;
        if (p.offsets != nullptr) {
            ro = t / steps;
            step = static_cast<int>(t % steps);
            row = ro;
            sf_row = expert_sf_row(p.offsets, p.num_experts, p.m, row);
            if (sf_row < 0 || (sf_row >> 7) >= p.sf_row_blocks) continue;
        } else {
            step = in8 / 8;
            ro = r8 * 8 + in8 % 8;
            const int i = static_cast<int>(ro & 127);
            sf_row = (ro & ~static_cast<int64_t>(127)) + (i & 3) * 32 + (i >> 2);
            const int64_t seg = (sf_row >> 7) / seg_blocks;
            const int64_t in_seg = sf_row - seg * seg_blocks * 128;
            if (in_seg >= p.seg_rows) continue;
            row = seg * p.seg_rows + in_seg;
        }
        const int64_t seg = row / p.seg_rows;
        const T* xr = static_cast<const T*>(p.x) + seg * p.sxseg + (row - seg * p.seg_rows) * p.sxm;
        Raw16<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = static_cast<int64_t>(step * U + u) * 512 + lane * 16;
            if (c >= p.k) raw[u].zero();
            else if (VEC && c + 16 <= p.k) raw[u].load(xr + c);
            else raw[u].load_some(xr + c * p.sxk, p.sxk, static_cast<int>(p.k - c < 16 ? p.k - c : 16));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = static_cast<int64_t>(step * U + u) * 512 + lane * 16;
            float amax = raw[u].amax();
            if constexpr (FMT == kFp4Mx) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            const Fp4Scale g = fp4_scale<FMT>(amax, tn);
            float v[16];
            raw[u].values(v);
            const uint2 codes = fp4_codes16<FMT>(v, g);
            if (c < p.k) *reinterpret_cast<uint2*>(p.q + row * p.ldq + (c >> 1)) = codes;
            // the four bytes of a block's row
            constexpr int lanes = FMT == kFp4Nv ? 1 : 2;           // lanes per group
            const bool live = (c & ~static_cast<int64_t>(fp4_group(FMT) - 1)) < p.k;
            uint32_t w = live ? g.byte << (8 * ((lane / lanes) & 3)) : 0u;
            if constexpr (lanes == 2) w = (lane & 1) ? 0u : w;
            if constexpr (lanes == 2) w |= __shfl_xor_sync(0xffffffffu, w, 1);
            w |= __shfl_xor_sync(0xffffffffu, w, lanes);
            w |= __shfl_xor_sync(0xffffffffu, w, 2 * lanes);
            const int64_t kb = c / (4 * fp4_group(FMT));
            if (lane % (4 * lanes) == 0 && kb < kblocks) {
                uint8_t* dst = p.sf + ((sf_row >> 7) * kblocks + kb) * kFp4SfBlock + (sf_row & 31) * 16 + ((sf_row >> 5) & 3) * 4;
                *reinterpret_cast<uint32_t*>(dst) = w;
            }
        }
    }
}

// Both casts of a 128 x 128 tile. The row cast is made from the loads'
// registers (a thread has 16 columns of a row); the raw elements also go to
// shared memory, from which the column cast reads 32 rows of two neighbouring
// columns per thread. Column codes and both tiles' scale blocks are gathered in
// shared memory and leave as whole 16-byte pieces.
template <typename T>
struct DualSmem {
    static constexpr int kPitch = 128 * sizeof(T) + 16;      // bytes per tile row
    static constexpr int kColPitch = 80;                     // bytes per column's 64 bytes of codes
    static constexpr int kOffCol = 128 * kPitch;
    static constexpr int kOffSfr = kOffCol + 128 * kColPitch;
    static constexpr int kOffSfc = kOffSfr + 2 * kFp4SfBlock;
    static constexpr int kBytes = kOffSfc + 2 * kFp4SfBlock;
};

template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) fp4_dual_kernel(const Fp4DualArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    using S = DualSmem<T>;
    __shared__ int64_t s_row0, s_rows, s_sfblk, s_kcol;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int tid = threadIdx.x;
    const int64_t bz = blockIdx.z;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 128;
    // this tile's rows: [row0, row0 + rows) of x, 128-row scale block sfblk of
    // the row cast, columns kcol .. kcol + 128 of the column cast
    if (p.offsets == nullptr) {
        if (tid == 0) {
            s_row0 = static_cast<int64_t>(blockIdx.y) * 128;
            s_rows = p.m - s_row0 < 128 ? p.m - s_row0 : 128;
            s_sfblk = blockIdx.y;
            s_kcol = s_row0;
        }
    } else if (tid == 0) {
        // walk the experts: each has ceil(rows / 256) pairs of tiles
        int64_t left = blockIdx.y, blk = 0, prev = 0;
        s_rows = -1;
        for (int e = 0; e < p.num_experts; ++e) {
            int64_t lo = __ldg(p.offsets + e), hi = __ldg(p.offsets + e + 1);
            lo = lo < prev ? prev : (lo > p.m ? p.m : lo);
            hi = hi < lo ? lo : (hi > p.m ? p.m : hi);
            prev = hi;
            const int64_t tiles = (hi - lo + 255) / 256 * 2;
            if (left < tiles) {
                s_row0 = lo + left * 128;
                const int64_t rest = hi - s_row0;
                s_rows = rest < 0 ? 0 : (rest < 128 ? rest : 128);
                s_sfblk = rest > 0 ? blk + left : -1;
                s_kcol = static_cast<int64_t>(blockIdx.y) * 128;
                break;
            }
            left -= tiles;
            blk += (hi - lo + 127) / 128;
        }
    }
    __syncthreads();
    const int64_t rows = s_rows, row0 = s_row0, sfblk = s_sfblk, kcol = s_kcol;
    if (rows < 0 || kcol >= p.kpad) return;
    const Fp4Tensor tn = fp4_tensor(p.tscale);
    const T* x = static_cast<const T*>(p.x) + bz * p.sxb;
    const int64_t kblocks_r = fp4_kblocks(p.k, FMT);
    constexpr int kWords = FMT == kFp4Nv ? 2 : 1;             // scale blocks across 128 columns
    {
        // rows: unit u = (row u / 8, 16 columns u % 8)
        Raw16<T> raw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = i * kThreads + tid, r = u >> 3;
            const int64_t c = c0 + (u & 7) * 16;
            if (r >= rows || c >= p.k) raw[i].zero();
            else if (VEC && c + 16 <= p.k) raw[i].load(x + (row0 + r) * p.sxm + c);
            else raw[i].load_some(x + (row0 + r) * p.sxm + c, 1, static_cast<int>(p.k - c < 16 ? p.k - c : 16));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = i * kThreads + tid, r = u >> 3, cg = u & 7;
            uint4* dst = reinterpret_cast<uint4*>(smem + r * S::kPitch + cg * 16 * sizeof(T));
            const uint4* src = reinterpret_cast<const uint4*>(&raw[i]);
#pragma unroll
            for (int j = 0; j < static_cast<int>(sizeof(T)); ++j) dst[j] = src[j];
            if (p.qr != nullptr) {
                float amax = raw[i].amax();
                if constexpr (FMT == kFp4Mx) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                const Fp4Scale g = fp4_scale<FMT>(amax, tn);
                float v[16];
                raw[i].values(v);
                const uint2 codes = fp4_codes16<FMT>(v, g);
                const int64_t c = c0 + cg * 16;
                if (r < rows && c < p.k)
                    *reinterpret_cast<uint2*>(p.qr + bz * p.sqrb + (row0 + r) * p.ldr + (c >> 1)) = codes;
                const int gi = FMT == kFp4Nv ? cg : cg >> 1;
                const bool live = c0 + gi * fp4_group(FMT) < p.k && r < rows;
                if (FMT == kFp4Nv || (cg & 1) == 0)
                    smem[S::kOffSfr + (gi >> 2) * kFp4SfBlock + (r & 31) * 16 + (r >> 5) * 4 + (gi & 3)] =
                        live ? static_cast<uint8_t>(g.byte) : 0;
            }
        }
    }
    __syncthreads();
    {
        // columns: columns 2 cp and 2 cp + 1, rows 32 tq .. 32 tq + 32
        const int cp = tid & 63, tq = tid >> 6;
        float v[2][32];
        float am[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint8_t* src = smem + (tq * 32 + h * 16 + j) * S::kPitch + cp * 2 * sizeof(T);
                if constexpr (sizeof(T) == 2) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(src);
                    v[0][h * 16 + j] = __uint_as_float(w << 16);
                    v[1][h * 16 + j] = __uint_as_float(w & 0xFFFF0000u);
                } else {
                    const float2 w = *reinterpret_cast<const float2*>(src);
                    v[0][h * 16 + j] = w.x;
                    v[1][h * 16 + j] = w.y;
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j) m = max_nan(m, fabsf(v[s][h * 16 + j]));
                am[s][h] = m;
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int col = 2 * cp + s;
            if constexpr (FMT == kFp4Mx) am[s][0] = am[s][1] = max_nan(am[s][0], am[s][1]);
            uint32_t out[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Fp4Scale g = fp4_scale<FMT>(am[s][h], tn);
                float y[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = v[s][h * 16 + j];
                const uint2 codes = fp4_codes16<FMT>(y, g);
                out[2 * h] = codes.x;
                out[2 * h + 1] = codes.y;
                const int gi = FMT == kFp4Nv ? tq * 2 + h : tq;
                if (FMT == kFp4Nv || h == 0)
                    smem[S::kOffSfc + (gi >> 2) * kFp4SfBlock + (col & 31) * 16 + (col >> 5) * 4 + (gi & 3)] =
                        static_cast<uint8_t>(g.byte);
            }
            *reinterpret_cast<uint4*>(smem + S::kOffCol + col * S::kColPitch + tq * 16) =
                make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
    __syncthreads();
    // column codes: 64 bytes per column
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int u = i * kThreads + tid, col = u >> 2, part = u & 3;
        if (c0 + col < p.k)
            *reinterpret_cast<uint4*>(p.qc + bz * p.sqcb + (c0 + col) * p.ldc + (kcol >> 1) + part * 16) =
                *reinterpret_cast<const uint4*>(smem + S::kOffCol + col * S::kColPitch + part * 16);
    }
    // scale blocks
    const int64_t kblocks_c = fp4_kblocks(p.offsets != nullptr ? p.kpad : p.m, FMT);
    if (tid < kWords * 32) {
        const int w = tid >> 5, l = tid & 31;
        const int64_t kb = kcol / (4 * fp4_group(FMT)) + w;
        if (kb < kblocks_c)
            *reinterpret_cast<uint4*>(p.sfc + bz * p.sscb + (static_cast<int64_t>(blockIdx.x) * kblocks_c + kb) * kFp4SfBlock + l * 16) =
                *reinterpret_cast<const uint4*>(smem + S::kOffSfc + w * kFp4SfBlock + l * 16);
    } else if (tid >= 128 && tid < 128 + kWords * 32 && p.qr != nullptr && sfblk >= 0 && sfblk < p.sfr_row_blocks) {
        const int w = (tid - 128) >> 5, l = tid & 31;
        const int64_t kb = c0 / (4 * fp4_group(FMT)) + w;
        if (kb < kblocks_r)
            *reinterpret_cast<uint4*>(p.sfr + bz * p.ssrb + (sfblk * kblocks_r + kb) * kFp4SfBlock + l * 16) =
                *reinterpret_cast<const uint4*>(smem + S::kOffSfr + w * kFp4SfBlock + l * 16);
    }
}

// Codes back to values: fl32(E2M1 * S), S the group's scale as the cast uses
// it, rounded once more for a bf16 output. A lane has 16 columns.
template <int FMT, bool OUT_BF16>
__global__ void __launch_bounds__(kThreads) fp4_dequant_kernel(const Fp4DequantArgs p) {
    pdl_launch_dependents();
    pdl_wait_prior();
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    const int64_t kblocks = fp4_kblocks(p.k, FMT);
    const int64_t pieces = (p.k + 511) / 512;
    const float t = p.tscale != nullptr && FMT == kFp4Nv ? __ldg(p.tscale) : 1.0f;
    constexpr int es = OUT_BF16 ? 2 : 4;
    const bool vec = (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0 && (p.ldo * es) % 16 == 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); i < p.m * pieces; i += nwarps) {
        const int64_t row = i / pieces;
        const int64_t c = (i % pieces) * 512 + lane * 16;
        if (c >= p.k) continue;
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.q + row * p.ldq + (c >> 1)));
        const int64_t g = c / fp4_group(FMT);
        const uint32_t b = __ldg(p.sf + ((row >> 7) * kblocks + (g >> 2)) * kFp4SfBlock + (row & 31) * 16 +
                                 ((row >> 5) & 3) * 4 + (g & 3));
        float s;
        if constexpr (FMT == kFp4Nv) s = __fmul_rn(e4m3_value(b), t);
        else s = b == 0xFFu ? __uint_as_float(0x7FC00000u) : (b == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23));
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t code = ((j < 8 ? w.x : w.y) >> (4 * (j & 7))) & 0xFu;
            const uint32_t e = (code >> 1) & 3u, m = code & 1u;
            // 0, 0.5, then (1 + m / 2) 2^(e - 1)
            const float mag = e == 0 ? 0.5f * static_cast<float>(m) : __uint_as_float((e + 126u) << 23 | m << 22);
            v[j] = __fmul_rn((code & 8u) ? -mag : mag, s);
        }
        if constexpr (OUT_BF16) {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + row * p.ldo + c;
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                h[j] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            if (vec && c + 16 <= p.k) {
                reinterpret_cast<uint4*>(o)[0] = make_uint4(h[0], h[1], h[2], h[3]);
                reinterpret_cast<uint4*>(o)[1] = make_uint4(h[4], h[5], h[6], h[7]);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < p.k) o[j] = __float2bfloat16_rn(v[j]);
            }
        } else {
            float* o = static_cast<float*>(p.out) + row * p.ldo + c;
            if (vec && c + 16 <= p.k) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    reinterpret_cast<float4*>(o)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < p.k) o[j] = v[j];
            }
        }
    }
}

// t = the least power of two with max|x| <= 2688 t (2688 = 6 * 448 = 1.3125 *
// 2^11), at least 2^-80; NaN if x has an infinity or a NaN. A power of two
// leaves every s * t and every halfway case of x / (s * t) exact. Each block
// makes the t of its own part and the largest, as bits, stays in a word that
// starts at zero: the order of the atomics does not matter.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) fp4_tscale_kernel(const T* x, int64_t m, int64_t k, int64_t sxm, int64_t sxk,
                                                            uint32_t* tscale) {
    pdl_wait_prior();
    float best = 0.0f;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t per_row = (k + 15) / 16;
    for (int64_t i = first; i < m * per_row; i += stride) {
        const int64_t row = i / per_row, c = (i - row * per_row) * 16;
        Raw16<T> raw;
        if (VEC && c + 16 <= k) raw.load(x + row * sxm + c);
        else raw.load_some(x + row * sxm + c * sxk, sxk, static_cast<int>(k - c < 16 ? k - c : 16));
        best = max_nan(best, raw.amax());
    }
    uint32_t b = __reduce_max_sync(0xffffffffu, __float_as_uint(best) & 0x7FFFFFFFu);
    __shared__ uint32_t s[kThreads / 32];
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = b;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) b = max(b, s[i]);
        const int e = static_cast<int>(b >> 23) - 11 + ((b & 0x7FFFFFu) > 0x280000u ? 1 : 0);
        const uint32_t least = 127 - 80;
        const uint32_t field = e < static_cast<int>(least) ? least : static_cast<uint32_t>(e);
        atomicMax(tscale, (b >> 23) == 255u ? 0x7FC00000u : field << 23);
    }
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, size_t smem, cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

bool vec_ok(const void* x, int64_t es, int64_t sxm, int64_t sxk, int64_t sxseg) {
    return (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && sxk == 1 && (sxm * es) % 16 == 0 && (sxseg * es) % 16 == 0;
}

template <typename T, int FMT, bool VEC>
cudaError_t cast_u(const Fp4CastArgs& a, cudaStream_t st, int num_sms) {
    const int64_t pieces = (a.k + 511) / 512;
    const int64_t seg_blocks = (a.seg_rows + 127) / 128;
    const int64_t rows = a.offsets != nullptr ? a.m : (a.m / a.seg_rows) * seg_blocks * 128;
    const bool two = a.m * pieces > static_cast<int64_t>(num_sms) * 64;
    const int64_t tasks = rows * (two ? (pieces + 1) / 2 : pieces);
    int64_t grid = (tasks + 7) / 8;
    if (grid > static_cast<int64_t>(num_sms) * 8) grid = static_cast<int64_t>(num_sms) * 8;
    return two ? launch(fp4_cast_kernel<T, FMT, VEC, 2>, dim3(static_cast<unsigned>(grid)), 0, st, a)
               : launch(fp4_cast_kernel<T, FMT, VEC, 1>, dim3(static_cast<unsigned>(grid)), 0, st, a);
}

template <typename T, int FMT>
cudaError_t cast_v(const Fp4CastArgs& a, cudaStream_t st, int num_sms) {
    return vec_ok(a.x, sizeof(T), a.sxm, a.sxk, a.sxseg) ? cast_u<T, FMT, true>(a, st, num_sms)
                                                         : cast_u<T, FMT, false>(a, st, num_sms);
}

template <typename T, int FMT, bool VEC>
cudaError_t dual_v(const Fp4DualArgs& a, cudaStream_t st, dim3 grid) {
    auto kern = fp4_dual_kernel<T, FMT, VEC>;
    constexpr int bytes = DualSmem<T>::kBytes;
    if (bytes > 48 * 1024)
        if (cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), bytes); e != cudaSuccess) return e;
    return launch(kern, grid, bytes, st, a);
}

template <typename T, int FMT>
cudaError_t dual_t(const Fp4DualArgs& a, cudaStream_t st, dim3 grid) {
    return vec_ok(a.x, sizeof(T), a.sxm, 1, a.sxb) ? dual_v<T, FMT, true>(a, st, grid)
                                                   : dual_v<T, FMT, false>(a, st, grid);
}

}  // namespace

cudaError_t launch_fp4_cast(const Fp4CastArgs& a, cudaStream_t st, int num_sms) {
    if (a.is_bf16)
        return a.fmt == kFp4Nv ? cast_v<__nv_bfloat16, kFp4Nv>(a, st, num_sms)
                               : cast_v<__nv_bfloat16, kFp4Mx>(a, st, num_sms);
    return a.fmt == kFp4Nv ? cast_v<float, kFp4Nv>(a, st, num_sms) : cast_v<float, kFp4Mx>(a, st, num_sms);
}

cudaError_t launch_fp4_cast_dual(const Fp4DualArgs& a, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((a.k + 127) / 128), static_cast<unsigned>(a.kpad / 128),
                    static_cast<unsigned>(a.batch));
    if (a.is_bf16)
        return a.fmt == kFp4Nv ? dual_t<__nv_bfloat16, kFp4Nv>(a, st, grid) : dual_t<__nv_bfloat16, kFp4Mx>(a, st, grid);
    return a.fmt == kFp4Nv ? dual_t<float, kFp4Nv>(a, st, grid) : dual_t<float, kFp4Mx>(a, st, grid);
}

cudaError_t launch_fp4_dequant(const Fp4DequantArgs& a, cudaStream_t st, int num_sms) {
    int64_t grid = (a.m * ((a.k + 511) / 512) + 7) / 8;
    if (grid > static_cast<int64_t>(num_sms) * 16) grid = static_cast<int64_t>(num_sms) * 16;
    const dim3 g(static_cast<unsigned>(grid));
    if (a.fmt == kFp4Nv)
        return a.out_bf16 ? launch(fp4_dequant_kernel<kFp4Nv, true>, g, 0, st, a)
                          : launch(fp4_dequant_kernel<kFp4Nv, false>, g, 0, st, a);
    return a.out_bf16 ? launch(fp4_dequant_kernel<kFp4Mx, true>, g, 0, st, a)
                      : launch(fp4_dequant_kernel<kFp4Mx, false>, g, 0, st, a);
}

cudaError_t launch_fp4_tensor_scale(const void* x, bool is_bf16, int64_t m, int64_t k, int64_t sxm, int64_t sxk, float* t,
                            cudaStream_t st, int num_sms) {
    if (cudaError_t e = cudaMemsetAsync(t, 0, 4, st); e != cudaSuccess) return e;
    int64_t grid = (m * ((k + 15) / 16) + kThreads - 1) / kThreads;
    if (grid > static_cast<int64_t>(num_sms) * 8) grid = static_cast<int64_t>(num_sms) * 8;
    if (grid < 1) grid = 1;
    const dim3 g(static_cast<unsigned>(grid));
    uint32_t* out = reinterpret_cast<uint32_t*>(t);
    if (is_bf16) {
        const auto* p = static_cast<const __nv_bfloat16*>(x);
        return vec_ok(x, 2, sxm, sxk, 0) ? launch(fp4_tscale_kernel<__nv_bfloat16, true>, g, 0, st, p, m, k, sxm, sxk, out)
                                         : launch(fp4_tscale_kernel<__nv_bfloat16, false>, g, 0, st, p, m, k, sxm, sxk, out);
    }
    const auto* p = static_cast<const float*>(x);
    return vec_ok(x, 4, sxm, sxk, 0) ? launch(fp4_tscale_kernel<float, true>, g, 0, st, p, m, k, sxm, sxk, out)
                                     : launch(fp4_tscale_kernel<float, false>, g, 0, st, p, m, k, sxm, sxk, out);
}

}  // namespace ql
