// Arguments and shared device code of the 4-bit products (fp4_gemm.cu,
// fp4_gemm_pair.cu).
//
//   D[i, j] (+)= tx tw sum_g sx[i, g] sw[j, g] sum_{k in g} X[i, k] W[j, k]
//
// X [m, k] and W [n, k] are 4-bit tensors in the layouts of fp4.cuh. Forms:
//   kFp4Plain    one product
//   kFp4RagRows  experts: rows [offsets[e], offsets[e+1]) of X and D belong to
//                W[e]; X's scale blocks start anew with every expert
//   kFp4RagK     experts along K: D[e] = X_e W_e^T over expert e's columns,
//                which start on a multiple of 256 in both operands
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "gemm.cuh"

namespace ql {

constexpr int kFp4Plain = 0, kFp4RagRows = 1, kFp4RagK = 2;

struct Fp4GemmArgs {
    const uint8_t* x;
    int64_t ldx;
    const uint8_t* sfx;
    int64_t x_row_blocks;        // 128-row scale blocks of X
    const float* tx;             // tensor scales (device) or null for 1
    const uint8_t* w;
    int64_t ldw;
    const uint8_t* sfw;
    const float* tw;
    int fmt, form;
    int64_t m, n, k;             // ragged K: k is the padded extent
    const int32_t* offsets;
    int experts;
    int64_t rows;                // ragged: the offsets' upper bound (rows of X, or tokens)
    void* d;
    int64_t ldd;
    bool out_f32;
    int accumulate;
    bool zero_rest;              // ragged rows: rows of no expert become zero
    // X not cast yet (m <= fp4_cast_rows): the product casts it itself
    const void* xr;
    bool xr_bf16;
    int64_t sxr;                 // elements between its rows
    uint32_t* dev_status;
    uint64_t wait_limit_ns;
    int stall_producer;
};

// Kernel parameters.
struct Fp4GemmParams {
    int form, experts;
    int m, n;                    // D's rows and columns (ragged rows: all rows)
    int k64;                     // steps of 64 along K (plain and ragged rows)
    int rows;                    // upper bound of the offsets
    int tiles_x, tiles_w;        // tiles along D's rows (plain, ragged K) and columns
    int group_x;                 // tiles of D's rows taken together (pair kernel)
    int kblocks;                 // scale blocks along K of one 128-row block
    int w_row_blocks;            // 128-row scale blocks of one W
    const int32_t* offsets;
    const float* tx;
    const float* tw;
    void* d;
    int64_t ldd;
    int accumulate;
    int tma_d;                   // whole 32-row pieces leave through TMA tile stores
    int vec_store;               // bf16 D: 8-byte stores of four columns
    uint32_t* dev_status;
    uint64_t wait_limit_ns;
    int stall_producer;
    const void* xr;              // X before the cast (the kernel's casting form)
    int64_t sxr;
    int k, xr_vec;               // columns; rows start on 16 bytes
    Bounds bnd;                  // D, offsets, X before the cast
    int zero_rest;
    int ahead;                   // stages of W brought into L2 before the previous kernel ends
};

// Largest m whose X the product casts itself: with experts each tile casts its
// own expert's rows only, so that more rows in all are worth it.
constexpr int64_t fp4_cast_rows(int experts) { return experts > 0 ? 16 : 8; }

cudaError_t launch_fp4_gemm(const Fp4GemmArgs& a, cudaStream_t st, int num_sms);
cudaError_t launch_fp4_gemm_pair(const Fp4GemmArgs& a, cudaStream_t st, int num_sms);

// Whether TMA can write D: rows that start and end on 16-byte boundaries (a copy
// may write a row's last 16-byte piece whole).
bool fp4_tma_d(const Fp4GemmArgs& a);

// Tensor maps of an operand's codes (box_rows x 128 bytes = 256 columns) and of
// its scale blocks (the blocks of 128 rows x 256 columns).
bool fp4_codes_map(CUtensorMap* map, const uint8_t* q, int64_t rows, int64_t kbytes, int64_t ld, int box_rows);
bool fp4_scales_map(CUtensorMap* map, const uint8_t* sf, int64_t blocks, int fmt);
void fp4_fill_params(const Fp4GemmArgs& a, Fp4GemmParams& p);

#ifdef __CUDACC__
// D(tmem) (+)= A B^T over 64 columns of K, both operands E2M1, fp32
// accumulation, scales in tensor memory.
template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (FMT == kFp4Nv && PAIR)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else if constexpr (FMT == kFp4Nv)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else if constexpr (PAIR)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// Instruction descriptor: A and B E2M1 (1 at bits 7-9 and 10-12), both K-major,
// N >> 3 at [17,23), scale type at bit 23 (0 E4M3, 1 UE8M0), M >> 4 at [24,29),
// K = 64 (bit 31 = 0). The byte of a 32-bit scale word where the instruction's
// scales start, at [29,31) for A and [4,6) for B: 0 for four scales per step,
// 0 or 2 for two.
template <int FMT>
__device__ __forceinline__ constexpr uint32_t idesc_fp4(uint32_t M, uint32_t N, uint32_t sf_byte) {
    return (sf_byte << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((FMT == kFp4Mx ? 1u : 0u) << 23) |
           ((M >> 4) << 24) | (sf_byte << 29);
}

// The experts' row ranges into shared memory, in order and inside [0, rows]
// whatever the caller gave (a range that was not is reported). One warp.
__device__ __forceinline__ void fp4_load_offsets(int* s_off, const Fp4GemmParams& p) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    bool bad = false;
    for (int i0 = 0; i0 <= p.experts; i0 += 32) {
        const int i = i0 + lane;
        int v = i <= p.experts && QL_IN(p.bnd, 1, p.offsets + i, 4) ? __ldg(p.offsets + i) : 0;
        const int raw = v;
        v = v < 0 ? 0 : (v > p.rows ? p.rows : v);
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, v, s);
            if (lane >= s) v = max(v, o);
        }
        v = max(v, carry);
        if (i <= p.experts) {
            s_off[i] = v;
            bad |= v != raw;
        }
        carry = __shfl_sync(0xffffffffu, v, 31);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) atomicOr(p.dev_status, kDevErrBadIndex);
}

// Zeros in the rows of D before the first and after the last expert's: warps 2
// and 3 of every CTA, which have nothing else to do by then, a row at a time.
template <bool OUT_F32>
__device__ __forceinline__ void fp4_zero_rest(const Fp4GemmParams& p, const int* s_off) {
    constexpr int es = OUT_F32 ? 4 : 2, kVec = 16 / es;
    const int lane = threadIdx.x & 31;
    const int before = s_off[0], after = s_off[p.experts];
    const int rest = before + p.m - after;
    uint8_t* d = static_cast<uint8_t*>(p.d);
    const bool vec = ((reinterpret_cast<uintptr_t>(d) | static_cast<uintptr_t>(p.ldd * es)) & 15u) == 0;
    for (int64_t i = blockIdx.x * 2 + (threadIdx.x >> 5) - 2; i < rest; i += gridDim.x * 2) {
        uint8_t* row = d + (i < before ? i : after + (i - before)) * p.ldd * es;
        int c = 0;
        if (vec) {
            for (int j = lane; j < p.n / kVec; j += 32)
                if (QL_IN(p.bnd, 0, row + 16 * static_cast<int64_t>(j), 16)) *reinterpret_cast<uint4*>(row + 16 * static_cast<int64_t>(j)) = make_uint4(0, 0, 0, 0);
            c = p.n / kVec * kVec;
        }
        for (int64_t j = c + lane; j < p.n; j += 32) {
            if (!QL_IN(p.bnd, 0, row + j * es, es)) continue;
            if constexpr (OUT_F32) *reinterpret_cast<float*>(row + j * es) = 0.0f;
            else *reinterpret_cast<uint16_t*>(row + j * es) = 0;
        }
    }
}

// One tile of D.
struct Fp4Tile {
    int x_row, w_row;      // first rows of the operands' codes
    int x_blk, w_blk;      // first 128-row scale blocks
    int x_sub;             // first row inside that block
    int k0;                // first step of 256 along K
    int k64;               // steps of 64
    int d_row, rows;       // D's rows [d_row, d_row + rows); rows may exceed the tile's
    int col;               // first column of D
};

// Tiles in order; TX: tile rows along D's rows, TW: along its columns. Calls
// come with growing t.
template <int TX, int TW>
struct Fp4Walk {
    int e = 0, base = 0, blk = 0, kpos = 0;      // expert, its first tile, scale block, step of 256

    __device__ __forceinline__ bool get(int t, const Fp4GemmParams& p, const int* s_off, Fp4Tile& o) {
        int local = t, tiles_x = p.tiles_x, r0 = 0, cnt = p.m;
        o.k0 = 0;
        o.k64 = p.k64;
        if (p.form != kFp4Plain) {
            for (;; ++e) {
                if (e >= p.experts) return false;
                r0 = s_off[e];
                cnt = s_off[e + 1] - r0;
                if (p.form == kFp4RagRows) tiles_x = (cnt + TX - 1) / TX;
                const int tiles = tiles_x * p.tiles_w;
                if (t - base < tiles) break;
                base += tiles;
                blk += (cnt + 127) >> 7;
                kpos += (cnt + 255) >> 8;
            }
            local = t - base;
        } else if (t >= p.tiles_x * p.tiles_w) {
            return false;
        }
        // group_x tiles of D's rows, then the next columns
        const int group = local / (p.group_x * p.tiles_w);
        const int first = group * p.group_x;
        const int gx = tiles_x - first < p.group_x ? tiles_x - first : p.group_x;
        const int in = local - group * p.group_x * p.tiles_w;
        const int ix = first + in % gx, iw = in / gx;
        const int x0 = ix * TX, w0 = iw * TW;
        o.col = w0;
        o.x_sub = x0 & 127;
        o.w_row = w0;
        o.w_blk = w0 >> 7;
        if (p.form == kFp4RagRows) {
            o.x_row = r0 + x0;
            o.x_blk = blk + (x0 >> 7);
            o.w_row += e * p.n;
            o.w_blk += e * p.w_row_blocks;
            o.d_row = r0 + x0;
            o.rows = cnt - x0;
        } else {
            o.x_row = x0;
            o.x_blk = x0 >> 7;
            o.d_row = x0;
            o.rows = p.m - x0;
            if (p.form == kFp4RagK) {
                o.d_row += e * p.m;
                o.k0 = kpos;
                o.k64 = (cnt + 63) >> 6;
            }
        }
        return true;
    }
};
#endif

}  // namespace ql
