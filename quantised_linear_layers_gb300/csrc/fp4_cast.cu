// Casts to and from the microscaled 4-bit formats of fp4.cuh.
//
//   fp4_cast_kernel     rows of x to codes and block-ordered scales
//   fp4_dual_kernel     rows and columns of x from one read (training)
//   fp4_dequant_kernel  codes and scales back to bf16 or fp32
//   fp4_tscale_kernel   the power of two t of a tensor (nv)
//
// The least traffic per element is its input bytes plus 0.5 + 1/16 (nv) or 0.5 +
// 1/32 (mx) written, twice that for both orientations. Measured at 16384 x 7168
// bf16 (nv / mx), with the share of the card's copy rate (6.77 TB/s): cast 46.9 /
// 45.0 us, 0.95 / 0.97; both ways 71.6 / 65.9 us, 0.76 / 0.80, bound by
// instruction issue (14 to 16 instructions an element) between its barriers;
// read-back 66.8 / 66.3 us, 121.7 / 122.0 to fp32, where a fill of the same outputs
// takes 61.8 and 119.1 (writes alone: 3.8 to 4.1 TB/s); scale 39.0 us, 0.89.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "bounds.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "gemm.cuh"

namespace ql {
namespace {

constexpr int kThreads = 256;

// Position of `row` among the experts' 128-row scale blocks: its row in the
// padded order, or -1 if no expert has it. The whole warp calls it.
__device__ __forceinline__ int64_t expert_sf_row(const int32_t* offsets, int experts, int64_t row, const Bounds& bnd) {
    const int lane = threadIdx.x & 31;
    int blocks = 0;             // blocks of the experts that end at or before the row
    int start = -1;
    for (int e0 = 0; e0 < experts; e0 += 32) {
        const int e = e0 + lane;
        int b = 0, s = -1;
        if (e < experts && QL_IN(bnd, 3, offsets + e, 8)) {
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

// How the rows of x lie: on 16-byte boundaries, contiguous but starting
// anywhere, or with any strides.
constexpr int kRowsVec = 0, kRowsContiguous = 1, kRowsStrided = 2;

// 512 columns of a contiguous row that starts anywhere, one column per lane and
// load, through the warp's shared memory: 16 columns per lane from there. (A
// lane loading its own 16 columns one by one touches 32 lines per load:
// 1003 x 4099 fp32 took 21 us instead of 7.)
template <typename T>
__device__ __forceinline__ void load_piece(Raw16<T>& raw, const T* row, int64_t c0, int64_t k, T* buf, const Bounds& bnd) {
    const int lane = threadIdx.x & 31;
    T v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t c = c0 + i * 32 + lane;
        v[i] = c < k && QL_IN(bnd, 0, row + c, sizeof(T)) ? row[c] : T(0.0f);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) buf[i * 32 + lane] = v[i];
    __syncwarp();
    const uint4* s = reinterpret_cast<const uint4*>(buf + lane * 16);
    uint4* d = reinterpret_cast<uint4*>(&raw);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) d[i] = s[i];
}

// A warp takes a row, in pieces of 512 columns, U of them at a time with their
// loads issued first; a lane has 16 consecutive columns: an nv group, or half
// an mx group whose other half is the next lane's. A block's eight rows are
// those of one 32-byte sector of their scale block (rows r, r+32, r+64, r+96
// and the next four), whose words its warps write at about the same time; the
// columns are shared out over blockIdx.y when there are few rows.
template <typename T, int FMT, int ROWS, int U>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 4) fp4_cast_kernel(const Fp4CastArgs p) {
    __shared__ __align__(16) T s_buf[ROWS == kRowsContiguous ? kThreads / 32 * 512 : 1];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t kblocks = static_cast<uint32_t>(fp4_kblocks(p.k, FMT));
    const int pieces = static_cast<int>((p.k + 511) / 512);
    const int steps = (pieces + U - 1) / U;
    int64_t row, sf_row;
    const T* xr = static_cast<const T*>(p.x);
    if (p.offsets != nullptr) {
        row = static_cast<int64_t>(blockIdx.x) * 8 + warp;
        sf_row = row < p.m ? expert_sf_row(p.offsets, p.num_experts, row, p.bnd) : -1;
        if (sf_row < 0 || (sf_row >> 7) >= p.sf_row_blocks) return;
        xr += row * p.sxm;
    } else {
        const unsigned block = blockIdx.x >> 4, i = (blockIdx.x & 15u) * 8 + warp;
        const unsigned seg_blocks = static_cast<unsigned>((p.seg_rows + 127) >> 7);
        const unsigned seg = block / seg_blocks;
        sf_row = static_cast<int64_t>(block) * 128 + (i & 3) * 32 + (i >> 2);
        const int64_t in_seg = sf_row - static_cast<int64_t>(seg) * seg_blocks * 128;
        if (in_seg >= p.seg_rows) return;
        row = static_cast<int64_t>(seg) * p.seg_rows + in_seg;
        xr += seg * p.sxseg + in_seg * p.sxm;
    }
    const Fp4Tensor tn = fp4_tensor(p.tscale);
    uint8_t* q = p.q + row * p.ldq;
    uint8_t* sf = p.sf + (sf_row >> 7) * kblocks * kFp4SfBlock + (sf_row & 31) * 16 + ((sf_row >> 5) & 3) * 4;
    const uint32_t k = static_cast<uint32_t>(p.k);
    for (int step = blockIdx.y; step < steps; step += gridDim.y) {
        const uint32_t c0 = static_cast<uint32_t>(step) * (U * 512u) + lane * 16u;
        Raw16<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = c0 + u * 512u;
            if constexpr (ROWS == kRowsContiguous) load_piece(raw[u], xr, c - lane * 16, k, s_buf + warp * 512, p.bnd);
            else if (c >= k) raw[u].zero();
            else if (ROWS == kRowsVec && c + 16 <= k) raw[u].load(xr + c, p.bnd, 0);
            else raw[u].load_some(xr + c * p.sxk, p.sxk, static_cast<int>(k - c < 16 ? k - c : 16), p.bnd, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = c0 + u * 512u;
            float amax = raw[u].amax();
            if constexpr (FMT == kFp4Mx) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            const Fp4Scale g = fp4_scale<FMT>(amax, tn);
            uint64_t v[8];
            raw[u].values(v);
            const uint2 codes = fp4_codes16<FMT>(v, g);
            if (c < k && QL_IN(p.bnd, 1, q + (c >> 1), 8)) *reinterpret_cast<uint2*>(q + (c >> 1)) = codes;
            // the group's byte; the bytes of a block's row past the last group are zero
            const uint32_t gi = c / fp4_group(FMT);
            uint8_t* dst = sf + static_cast<int64_t>(gi >> 2) * kFp4SfBlock + (gi & 3);
            if ((FMT == kFp4Nv || (lane & 1) == 0) && (gi >> 2) < kblocks && QL_IN(p.bnd, 2, dst, 1))
                *dst = c < k ? static_cast<uint8_t>(g.byte) : 0;
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

template <typename T, int FMT, int ROWS>
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
            if (!QL_IN(p.bnd, 3, p.offsets + e, 8)) break;
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
    const int64_t row0 = s_row0, sfblk = s_sfblk, kcol = s_kcol;
    const int rows = static_cast<int>(s_rows);
    if (rows < 0 || kcol >= p.kpad) return;
    const int cols = static_cast<int>(p.k - c0 < 128 ? p.k - c0 : 128);
    const Fp4Tensor tn = fp4_tensor(p.tscale);
    const T* x = static_cast<const T*>(p.x) + bz * p.sxb + row0 * p.sxm + c0;
    const int64_t kblocks_r = fp4_kblocks(p.k, FMT);
    constexpr int kWords = FMT == kFp4Nv ? 2 : 1;             // scale blocks across 128 columns
    if constexpr (ROWS != kRowsVec) {
        // rows that start anywhere: one element per lane and load, kAhead loads in flight
        using E = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
        E* tile = reinterpret_cast<E*>(smem);
        constexpr int pitch = S::kPitch / sizeof(T), kAhead = 16, kRowStep = kThreads / 128;
        const int c = tid & 127;
        const E* src = reinterpret_cast<const E*>(x) + (tid >> 7) * p.sxm + c;
#pragma unroll 1
        for (int r0 = tid >> 7; r0 < 128; r0 += kAhead * kRowStep) {
            E v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i, src += kRowStep * p.sxm) {
                v[i] = 0;
                if (r0 + i * kRowStep < rows && c < cols && QL_IN(p.bnd, 0, src, sizeof(T))) v[i] = *src;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) tile[(r0 + i * kRowStep) * pitch + c] = v[i];
        }
        __syncthreads();
    }
    {
        // rows: unit u = (row u / 8, 16 columns u % 8)
        Raw16<T> raw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = i * kThreads + tid, r = u >> 3, c = (u & 7) * 16;
            if constexpr (ROWS != kRowsVec) {
                const uint4* src = reinterpret_cast<const uint4*>(smem + r * S::kPitch + c * sizeof(T));
#pragma unroll
                for (int j = 0; j < static_cast<int>(sizeof(T)); ++j) reinterpret_cast<uint4*>(&raw[i])[j] = src[j];
            } else {
                if (r >= rows || c >= cols) raw[i].zero();
                else if (c + 16 <= cols) raw[i].load(x + r * p.sxm + c, p.bnd, 0);
                else raw[i].load_some(x + r * p.sxm + c, 1, cols - c, p.bnd, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = i * kThreads + tid, r = u >> 3, cg = u & 7;
            if constexpr (ROWS == kRowsVec) {
                uint4* dst = reinterpret_cast<uint4*>(smem + r * S::kPitch + cg * 16 * sizeof(T));
#pragma unroll
                for (int j = 0; j < static_cast<int>(sizeof(T)); ++j) dst[j] = reinterpret_cast<const uint4*>(&raw[i])[j];
            }
            if (p.qr != nullptr) {
                float amax = raw[i].amax();
                if constexpr (FMT == kFp4Mx) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                const Fp4Scale g = fp4_scale<FMT>(amax, tn);
                uint64_t v[8];
                raw[i].values(v);
                const uint2 codes = fp4_codes16<FMT>(v, g);
                uint8_t* dst = p.qr + bz * p.sqrb + (row0 + r) * p.ldr + ((c0 + cg * 16) >> 1);
                if (r < rows && cg * 16 < cols && QL_IN(p.bnd, 1, dst, 8)) *reinterpret_cast<uint2*>(dst) = codes;
                const int gi = FMT == kFp4Nv ? cg : cg >> 1;
                const bool live = gi * fp4_group(FMT) < cols && r < rows;
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
        const uint8_t* src = smem + tq * 32 * S::kPitch + cp * 2 * sizeof(T);
        float am[2][2];                          // column, half
        uint32_t w[sizeof(T) == 2 ? 32 : 1];     // bf16: the pairs of both columns, kept
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = *reinterpret_cast<const uint32_t*>(src + j * S::kPitch);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t m = bf16x2_maxabs_nan(w[16 * h], w[16 * h + 1]);
#pragma unroll
                for (int j = 2; j < 16; ++j) m = bf16x2_maxabs_nan(m, w[16 * h + j]);
                am[0][h] = __uint_as_float((m << 16) & 0x7FFFFFFFu);
                am[1][h] = __uint_as_float(m & 0x7FFF0000u);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 e = *reinterpret_cast<const float2*>(src + (16 * h + j) * S::kPitch);
                    m0 = max_nan(m0, fabsf(e.x));
                    m1 = max_nan(m1, fabsf(e.y));
                }
                am[0][h] = m0;
                am[1][h] = m1;
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int col = 2 * cp + s;
            if constexpr (FMT == kFp4Mx) am[s][0] = am[s][1] = max_nan(am[s][0], am[s][1]);
            uint2 out[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Fp4Scale g = fp4_scale<FMT>(am[s][h], tn);
                uint64_t y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if constexpr (sizeof(T) == 2) {
                        const uint32_t a = w[16 * h + 2 * j], b = w[16 * h + 2 * j + 1];
                        y[j] = s == 0 ? f32x2(__uint_as_float(a << 16), __uint_as_float(b << 16))
                                      : f32x2(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u));
                    } else {
                        const uint8_t* e = src + (16 * h + 2 * j) * S::kPitch + 4 * s;
                        y[j] = f32x2(*reinterpret_cast<const float*>(e), *reinterpret_cast<const float*>(e + S::kPitch));
                    }
                }
                out[h] = fp4_codes16<FMT>(y, g);
                const int gi = FMT == kFp4Nv ? tq * 2 + h : tq;
                if (FMT == kFp4Nv || h == 0)
                    smem[S::kOffSfc + (gi >> 2) * kFp4SfBlock + (col & 31) * 16 + (col >> 5) * 4 + (gi & 3)] =
                        gi * fp4_group(FMT) < rows ? static_cast<uint8_t>(g.byte) : 0;
            }
            *reinterpret_cast<uint4*>(smem + S::kOffCol + col * S::kColPitch + tq * 16) =
                make_uint4(out[0].x, out[0].y, out[1].x, out[1].y);
        }
    }
    __syncthreads();
    // column codes: 64 bytes per column
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int u = i * kThreads + tid, col = u >> 2, part = u & 3;
        uint8_t* dst = p.qc + bz * p.sqcb + (c0 + col) * p.ldc + (kcol >> 1) + part * 16;
        if (col < cols && QL_IN(p.bnd, 4, dst, 16))
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(smem + S::kOffCol + col * S::kColPitch + part * 16);
    }
    // scale blocks
    const int64_t kblocks_c = fp4_kblocks(p.offsets != nullptr ? p.kpad : p.m, FMT);
    if (tid < kWords * 32) {
        const int wd = tid >> 5, l = tid & 31;
        const int64_t kb = kcol / (4 * fp4_group(FMT)) + wd;
        uint8_t* dst = p.sfc + bz * p.sscb + (static_cast<int64_t>(blockIdx.x) * kblocks_c + kb) * kFp4SfBlock + l * 16;
        if (kb < kblocks_c && QL_IN(p.bnd, 5, dst, 16))
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(smem + S::kOffSfc + wd * kFp4SfBlock + l * 16);
    } else if (tid >= 128 && tid < 128 + kWords * 32 && p.qr != nullptr && sfblk >= 0 && sfblk < p.sfr_row_blocks) {
        const int wd = (tid - 128) >> 5, l = tid & 31;
        const int64_t kb = c0 / (4 * fp4_group(FMT)) + wd;
        uint8_t* dst = p.sfr + bz * p.ssrb + (sfblk * kblocks_r + kb) * kFp4SfBlock + l * 16;
        if (kb < kblocks_r && QL_IN(p.bnd, 2, dst, 16))
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(smem + S::kOffSfr + wd * kFp4SfBlock + l * 16);
    }
}

// The two E2M1 codes of a byte as fp32.
__device__ __forceinline__ uint64_t e2m1x2_f32x2(uint32_t byte) {
    uint64_t d;
    asm("{\n"
        ".reg .b8 b, z1, z2, z3;\n"
        ".reg .b32 h;\n"
        ".reg .b16 l, u;\n"
        ".reg .f32 fl, fu;\n"
        "mov.b32 {b, z1, z2, z3}, %1;\n"
        "cvt.rn.f16x2.e2m1x2 h, b;\n"
        "mov.b32 {l, u}, h;\n"
        "cvt.f32.f16 fl, l;\n"
        "cvt.f32.f16 fu, u;\n"
        "mov.b64 %0, {fl, fu};\n"
        "}\n"
        : "=l"(d)
        : "r"(byte));
    return d;
}

// Codes back to values: fl32(E2M1 * S), S the group's scale as the cast uses
// it, rounded once more for a bf16 output. A warp takes a row (those of a
// block as in the cast), a lane 16 columns of each piece of 512. Rows of the
// output that start anywhere are written one column per lane and store.
template <int FMT, typename T, bool VEC, int U>
__global__ void __launch_bounds__(kThreads) fp4_dequant_kernel(const Fp4DequantArgs p) {
    __shared__ __align__(16) T s_buf[VEC ? 1 : kThreads / 32 * 512];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t kblocks = fp4_kblocks(p.k, FMT);
    const int steps = (static_cast<int>((p.k + 511) / 512) + U - 1) / U;
    const float t = p.tscale != nullptr && FMT == kFp4Nv ? __ldg(p.tscale) : 1.0f;
    const unsigned i8 = (blockIdx.x & 15u) * 8 + warp;
    const int64_t row = static_cast<int64_t>(blockIdx.x >> 4) * 128 + (i8 & 3) * 32 + (i8 >> 2);
    if (row >= p.m) return;
    const uint8_t* q = p.q + row * p.ldq;
    const uint8_t* sf = p.sf + (row >> 7) * kblocks * kFp4SfBlock + (row & 31) * 16 + ((row >> 5) & 3) * 4;
    T* out = static_cast<T*>(p.out) + row * p.ldo;
    for (int step = blockIdx.y; step < steps; step += gridDim.y) {
        uint2 codes[U];
        uint32_t b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = static_cast<int64_t>(step * U + u) * 512 + lane * 16;
            const int64_t g = c / fp4_group(FMT);
            const uint8_t* sb = sf + (g >> 2) * kFp4SfBlock + (g & 3);
            codes[u] = c < p.k && QL_IN(p.bnd, 1, q + (c >> 1), 8) ? __ldg(reinterpret_cast<const uint2*>(q + (c >> 1))) : make_uint2(0, 0);
            b[u] = c < p.k && QL_IN(p.bnd, 2, sb, 1) ? __ldg(sb) : 0u;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = static_cast<int64_t>(step * U + u) * 512 + lane * 16;
            float s;
            if constexpr (FMT == kFp4Nv) s = __fmul_rn(e4m3_value(b[u]), t);
            else s = b[u] == 0xFFu ? __uint_as_float(0x7FC00000u) : (b[u] == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(b[u] << 23));
            const uint64_t ss = f32x2(s, s);
            float v[16];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f32x2_get(mul2(e2m1x2_f32x2((j < 4 ? codes[u].x : codes[u].y) >> (8 * (j & 3))), ss), v[2 * j], v[2 * j + 1]);
            uint4 o[sizeof(T)];
            if constexpr (sizeof(T) == 2) {
                uint32_t h[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    h[j] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                o[0] = make_uint4(h[0], h[1], h[2], h[3]);
                o[1] = make_uint4(h[4], h[5], h[6], h[7]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                                      __float_as_uint(v[4 * j + 3]));
            }
            if (VEC && c + 16 <= p.k) {
#pragma unroll
                for (int j = 0; j < static_cast<int>(sizeof(T)); ++j)
                    if (QL_IN(p.bnd, 0, reinterpret_cast<uint4*>(out + c) + j, 16)) reinterpret_cast<uint4*>(out + c)[j] = o[j];
            } else if (VEC) {
                const T* e = reinterpret_cast<const T*>(o);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < p.k && QL_IN(p.bnd, 0, out + c + j, sizeof(T))) out[c + j] = e[j];
            } else {
                T* buf = s_buf + warp * 512;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < static_cast<int>(sizeof(T)); ++j) reinterpret_cast<uint4*>(buf + lane * 16)[j] = o[j];
                __syncwarp();
                const int64_t c0 = c - lane * 16 + lane;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c0 + j * 32 < p.k && QL_IN(p.bnd, 0, out + c0 + j * 32, sizeof(T))) out[c0 + j * 32] = buf[j * 32 + lane];
            }
        }
    }
}

// t = the least power of two with max|x| <= 2688 t (2688 = 6 * 448 = 1.3125 *
// 2^11), at least 2^-80; NaN if x has an infinity or a NaN. A power of two
// leaves every s * t and every halfway case of x / (s * t) exact. Each block
// makes the t of its own part and the largest, as bits, stays in a word that
// starts at zero: the order of the atomics does not matter. Up to 2 MB one
// cluster of eight blocks does it all (CLUSTER): its blocks' maxima meet in shared
// memory, and no word has to be set to zero by a launch of its own.
constexpr int kClusterThreads = 1024;

// FLAT: the rows lie one after the other and are taken as one.
template <typename T, int ROWS, bool FLAT, bool CLUSTER>
__global__ void __launch_bounds__(CLUSTER ? kClusterThreads : kThreads) fp4_tscale_kernel(const Fp4ScaleArgs p) {
    pdl_launch_dependents();
    pdl_wait_prior();
    constexpr int kBlock = CLUSTER ? kClusterThreads : kThreads;
    const T* x = static_cast<const T*>(p.x);
    uint32_t* tscale = reinterpret_cast<uint32_t*>(p.t);
    float best = 0.0f;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kBlock;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
    // rows [r0, r1), columns [lo, hi)
    int64_t r0 = 0, r1 = p.m, lo = 0, hi = p.k;
    if (p.offsets != nullptr && QL_IN(p.bnd, 1, p.offsets, 4) && QL_IN(p.bnd, 1, p.offsets + p.num_experts, 4)) {
        const int64_t a = __ldg(p.offsets), b = __ldg(p.offsets + p.num_experts);
        r0 = a < 0 ? 0 : (a > p.m ? p.m : a);
        r1 = b < r0 ? r0 : (b > p.m ? p.m : b);
    }
    if constexpr (FLAT) {
        lo = r0 * p.k;
        hi = r1 * p.k;
        r0 = 0;
        r1 = 1;
    }
    if constexpr (ROWS == kRowsVec) {
        const int64_t per_row = (hi + 15) / 16;
#pragma unroll 2
        for (int64_t i = r0 * per_row + lo / 16 + first; i < r1 * per_row; i += stride) {
            const int64_t row = FLAT ? 0 : i / per_row, c = (i - row * per_row) * 16;
            Raw16<T> raw;
            if ((!FLAT || c >= lo) && c + 16 <= hi) {
                raw.load(x + row * p.sxm + c, p.bnd, 0);
            } else {
                const int64_t c0 = c < lo ? lo : c, n = hi - c0;
                raw.load_some(x + row * p.sxm + c0, 1, static_cast<int>(n < c + 16 - c0 ? n : c + 16 - c0), p.bnd, 0);
            }
            best = max_nan(best, raw.amax());
        }
    } else {
        // one element per lane and load, eight loads in flight
        constexpr int kPiece = 8 * 32;
        const int lane = threadIdx.x & 31;
        const int64_t per_row = (hi + kPiece - 1) / kPiece;
        for (int64_t i = r0 * per_row + lo / kPiece + (first >> 5); i < r1 * per_row; i += stride >> 5) {
            const int64_t row = FLAT ? 0 : i / per_row, c0 = (i - row * per_row) * kPiece + lane;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t c = c0 + j * 32;
                const T* e = x + row * p.sxm + c * p.sxk;
                v[j] = c < hi && (!FLAT || c >= lo) && QL_IN(p.bnd, 0, e, sizeof(T)) ? static_cast<float>(*e) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) best = max_nan(best, fabsf(v[j]));
        }
    }
    uint32_t b = __reduce_max_sync(0xffffffffu, __float_as_uint(best) & 0x7FFFFFFFu);
    __shared__ uint32_t s[kBlock / 32], all;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = b;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < kBlock / 32; ++i) b = max(b, s[i]);
        all = b;
    }
    if constexpr (CLUSTER) {
        __syncwarp();
        cluster_sync_all();
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            for (unsigned r = 1; r < gridDim.x; ++r) {
                uint32_t v;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(&all, r)) : "memory");
                b = max(b, v);
            }
        }
        __syncwarp();
        cluster_sync_all();
        if (blockIdx.x != 0) return;
    }
    if (threadIdx.x == 0) {
        const int e = static_cast<int>(b >> 23) - 11 + ((b & 0x7FFFFFu) > 0x280000u ? 1 : 0);
        const int least = 127 - 80;
        const uint32_t t = (b >> 23) == 255u ? 0x7FC00000u : static_cast<uint32_t>(e < least ? least : e) << 23;
        if constexpr (CLUSTER) *tscale = t;
        else atomicMax(tscale, t);
    }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, int threads, unsigned cluster, size_t smem, cudaStream_t st,
                           const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, size_t smem, cudaStream_t st, const Args&... args) {
    return launch_cluster(kern, grid, kThreads, 1, smem, st, args...);
}

bool vec_ok(const void* x, int64_t es, int64_t sxm, int64_t sxk, int64_t sxseg) {
    return (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && sxk == 1 && (sxm * es) % 16 == 0 && (sxseg * es) % 16 == 0;
}

int rows_form(const void* x, int64_t es, int64_t sxm, int64_t sxk, int64_t sxseg) {
    if (vec_ok(x, es, sxm, sxk, sxseg)) return kRowsVec;
    return sxk == 1 ? kRowsContiguous : kRowsStrided;
}

// Blocks along the columns: all steps in one when the rows fill the SMs (eight
// blocks of 256 threads each), as many as there are steps when they do not.
unsigned column_blocks(int64_t rows, int64_t steps, int num_sms) {
    const int64_t sets = (rows + 7) / 8;
    int64_t y = (static_cast<int64_t>(num_sms) * 8 + sets - 1) / sets;
    if (y > steps) y = steps;
    return static_cast<unsigned>(y < 1 ? 1 : y);
}

template <typename T, int FMT, int ROWS>
cudaError_t cast_u(const Fp4CastArgs& a, cudaStream_t st, int num_sms) {
    const int64_t pieces = (a.k + 511) / 512;
    const int64_t sets = a.offsets != nullptr ? (a.m + 7) / 8 : (a.m / a.seg_rows) * ((a.seg_rows + 127) / 128) * 16;
    const unsigned x = static_cast<unsigned>(sets);
    // two pieces at a time once there is work for several rounds of blocks (one /
    // two, us: 512 x 7168 2.95 / 3.22, 2048 x 7168 7.18 / 6.66, 16384 x 7168 51.1 / 46.0)
    if (ROWS != kRowsContiguous && a.m * pieces > static_cast<int64_t>(num_sms) * 64)
        return launch(fp4_cast_kernel<T, FMT, ROWS, 2>, dim3(x, column_blocks(a.m, (pieces + 1) / 2, num_sms)), 0, st, a);
    return launch(fp4_cast_kernel<T, FMT, ROWS, 1>, dim3(x, column_blocks(a.m, pieces, num_sms)), 0, st, a);
}

template <typename T, int FMT>
cudaError_t cast_v(const Fp4CastArgs& a, cudaStream_t st, int num_sms) {
    switch (rows_form(a.x, sizeof(T), a.sxm, a.sxk, a.sxseg)) {
        case kRowsVec: return cast_u<T, FMT, kRowsVec>(a, st, num_sms);
        case kRowsContiguous: return cast_u<T, FMT, kRowsContiguous>(a, st, num_sms);
        default: return cast_u<T, FMT, kRowsStrided>(a, st, num_sms);
    }
}

template <typename T, int FMT, int ROWS>
cudaError_t dual_v(const Fp4DualArgs& a, cudaStream_t st, dim3 grid) {
    auto kern = fp4_dual_kernel<T, FMT, ROWS>;
    constexpr int bytes = DualSmem<T>::kBytes;
    if (bytes > 48 * 1024)
        if (cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), bytes); e != cudaSuccess) return e;
    return launch(kern, grid, bytes, st, a);
}

template <typename T, int FMT>
cudaError_t dual_t(const Fp4DualArgs& a, cudaStream_t st, dim3 grid) {
    return vec_ok(a.x, sizeof(T), a.sxm, 1, a.sxb) ? dual_v<T, FMT, kRowsVec>(a, st, grid)
                                                   : dual_v<T, FMT, kRowsContiguous>(a, st, grid);
}

template <int FMT, typename T>
cudaError_t dequant_t(const Fp4DequantArgs& a, cudaStream_t st, int num_sms) {
    const int64_t pieces = (a.k + 511) / 512;
    const unsigned x = static_cast<unsigned>((a.m + 127) / 128 * 16);
    if (!vec_ok(a.out, sizeof(T), a.ldo, 1, 0))
        return launch(fp4_dequant_kernel<FMT, T, false, 1>, dim3(x, column_blocks(a.m, pieces, num_sms)), 0, st, a);
    if (a.m * pieces > static_cast<int64_t>(num_sms) * 64)
        return launch(fp4_dequant_kernel<FMT, T, true, 2>, dim3(x, column_blocks(a.m, (pieces + 1) / 2, num_sms)), 0, st, a);
    return launch(fp4_dequant_kernel<FMT, T, true, 1>, dim3(x, column_blocks(a.m, pieces, num_sms)), 0, st, a);
}

template <typename T, int ROWS, bool FLAT>
cudaError_t tscale_v(const Fp4ScaleArgs& a, cudaStream_t st, int num_sms) {
    // one cluster / zeroing and atomics: 0.5 MB 3.1 / 5.0 us, 1 MB 3.8 / 4.7, 2 MB 5.3 / 6.0, 4 MB 7.9 / 6.2
    if (a.m * a.k * static_cast<int64_t>(sizeof(T)) <= (2 << 20))
        return launch_cluster(fp4_tscale_kernel<T, ROWS, FLAT, true>, dim3(8), kClusterThreads, 8, 0, st, a);
    if (cudaError_t e = cudaMemsetAsync(a.t, 0, 4, st); e != cudaSuccess) return e;
    const int64_t rows = FLAT ? 1 : a.m, cols = FLAT ? a.m * a.k : a.k;
    int64_t grid = ROWS == kRowsVec ? (rows * ((cols + 15) / 16) + kThreads - 1) / kThreads : (rows * ((cols + 255) / 256) + 7) / 8;
    if (grid > static_cast<int64_t>(num_sms) * 8) grid = static_cast<int64_t>(num_sms) * 8;
    return launch(fp4_tscale_kernel<T, ROWS, FLAT, false>, dim3(static_cast<unsigned>(grid < 1 ? 1 : grid)), 0, st, a);
}

template <typename T>
cudaError_t tscale_t(const Fp4ScaleArgs& a, cudaStream_t st, int num_sms) {
    // one long row if they follow one another: only its ends are ragged
    const bool flat = a.sxk == 1 && (a.sxm == a.k || a.m == 1);
    if (vec_ok(a.x, sizeof(T), flat ? 0 : a.sxm, a.sxk, 0))
        return flat ? tscale_v<T, kRowsVec, true>(a, st, num_sms) : tscale_v<T, kRowsVec, false>(a, st, num_sms);
    return flat ? tscale_v<T, kRowsStrided, true>(a, st, num_sms) : tscale_v<T, kRowsStrided, false>(a, st, num_sms);
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
    if (a.fmt == kFp4Nv)
        return a.out_bf16 ? dequant_t<kFp4Nv, __nv_bfloat16>(a, st, num_sms) : dequant_t<kFp4Nv, float>(a, st, num_sms);
    return a.out_bf16 ? dequant_t<kFp4Mx, __nv_bfloat16>(a, st, num_sms) : dequant_t<kFp4Mx, float>(a, st, num_sms);
}

cudaError_t launch_fp4_tensor_scale(const Fp4ScaleArgs& a, cudaStream_t st, int num_sms) {
    return a.is_bf16 ? tscale_t<__nv_bfloat16>(a, st, num_sms) : tscale_t<float>(a, st, num_sms);
}

}  // namespace ql
