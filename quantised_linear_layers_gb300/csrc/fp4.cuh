// Microscaled 4-bit floating point (E2M1): formats, layouts, group arithmetic
// and the launch arguments of the 4-bit operators.
//
// E2M1 holds 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign. A row is cut into groups
// along the reduction axis, each with one scale:
//   kFp4Nv  16 elements, E4M3 scale s = E4M3(amax / (6 t)) held in
//           [2^-9, 448], under one fp32 scale t per tensor: the element stands
//           for E2M1 * (s * t)
//   kFp4Mx  32 elements, scale 2^p, p = ceil(log2(amax / 6)) held in
//           [-127, 127] and stored as p + 127 (UE8M0)
// A group with an infinity or a NaN gets the scale NaN (0x7F / 0xFF) and codes
// of zero, so it is NaN in every product and when it is read back.
//
// Layouts. Codes: row-major bytes, element 2j in the low and 2j + 1 in the
// high half of byte j; rows start on 16-byte boundaries; the unused half byte of an
// odd number of columns is zero. Scales: blocks of 128
// rows x 4 groups (512 bytes), all groups of one 128-row block one after the
// other; inside a block the byte of (row r, group g) is at
// (r % 32) * 16 + (r / 32) * 4 + g, which is how the tensor core wants the
// scales of 128 rows in tensor memory, so the products copy whole blocks
// without touching a byte. Scale bytes of groups past the last are zero.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"

namespace ql {

constexpr int kFp4Nv = 0, kFp4Mx = 1;
constexpr int kFp4SfBlock = 512;         // bytes of one 128 x 4 scale block
constexpr int kFp4KAlign = 256;          // an expert's reduction axis starts on a multiple of it
constexpr int kFp4MaxExperts = 512;

__host__ __device__ constexpr int fp4_group(int fmt) { return fmt == kFp4Nv ? 16 : 32; }
// scale blocks along k columns
__host__ __device__ constexpr int64_t fp4_kblocks(int64_t k, int fmt) {
    return (k + 4 * fp4_group(fmt) - 1) / (4 * fp4_group(fmt));
}

// Cast of the rows of x; see include/qlinear.h for the row-segment forms.
struct Fp4CastArgs {
    const void* x;
    bool is_bf16;
    int64_t m, k;              // all rows, columns
    int64_t sxm, sxk;          // element strides
    int64_t seg_rows, sxseg;   // rows per segment (m if there is one), stride between segments
    int fmt;
    const float* tscale;       // t (device), or null for 1
    uint8_t* q;
    int64_t ldq;
    uint8_t* sf;
    const int32_t* offsets;    // row ranges of the experts (num_experts + 1), or null
    int num_experts;
    int64_t sf_row_blocks;     // blocks of 128 rows in sf
    uint32_t* dev_status;
};

// Casts of x along its rows and along its columns from one read.
struct Fp4DualArgs {
    const void* x;
    bool is_bf16;
    int64_t batch, m, k;       // x [batch][m][k]
    int64_t sxb, sxm;
    int fmt;
    const float* tscale;
    uint8_t* qr;               // rows: [batch][m][ldr] (null: not wanted)
    int64_t ldr, sqrb;
    uint8_t* sfr;
    int64_t ssrb;
    uint8_t* qc;               // columns: [batch][k][ldc]
    int64_t ldc, sqcb;
    uint8_t* sfc;
    int64_t sscb;
    const int32_t* offsets;    // experts' row ranges (batch == 1), or null
    int num_experts;
    int64_t sfr_row_blocks;    // 128-row blocks in sfr (experts: one more per expert)
    int64_t kpad;              // columns the column cast's codes have room for
    uint32_t* dev_status;
};

struct Fp4DequantArgs {
    const uint8_t* q;
    int64_t ldq;
    const uint8_t* sf;
    int fmt;
    const float* tscale;
    int64_t m, k;
    void* out;
    bool out_bf16;
    int64_t ldo;
    uint32_t* dev_status;
};

cudaError_t launch_fp4_cast(const Fp4CastArgs& a, cudaStream_t st, int num_sms);
cudaError_t launch_fp4_cast_dual(const Fp4DualArgs& a, cudaStream_t st);
cudaError_t launch_fp4_dequant(const Fp4DequantArgs& a, cudaStream_t st, int num_sms);
cudaError_t launch_fp4_tensor_scale(const void* x, bool is_bf16, int64_t m, int64_t k, int64_t sxm, int64_t sxk, float* t,
                            cudaStream_t st, int num_sms);

#ifdef __CUDACC__
// Larger of two magnitudes; a NaN operand gives NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight values to eight E2M1 codes (v[0] lowest), round to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t d;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n"
        "}\n"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
    return __half2float(__half(h));
}

// The tensor's scale as the groups' scales use it.
struct Fp4Tensor {
    float t, t6;     // t, 6 t
};
__device__ __forceinline__ Fp4Tensor fp4_tensor(const float* tscale) {
    const float t = tscale != nullptr ? __ldg(tscale) : 1.0f;
    return Fp4Tensor{t, __fmul_rn(6.0f, t)};
}

// Scale of one group: its stored byte, its value S and 1 / S (mx: exactly).
struct Fp4Scale {
    uint32_t byte;
    float s, r;
    bool finite;
};
template <int FMT>
__device__ __forceinline__ Fp4Scale fp4_scale(float amax, const Fp4Tensor& tn) {
    Fp4Scale o;
    o.finite = amax <= 3.402823466e38f;              // false for infinity and NaN
    if constexpr (FMT == kFp4Nv) {
        float d = __fdiv_rn(amax, tn.t6);
        d = fminf(fmaxf(d, 0.001953125f), 448.0f);
        o.byte = static_cast<uint32_t>(__nv_cvt_float_to_fp8(d, __NV_SATFINITE, __NV_E4M3));
        o.s = __fmul_rn(e4m3_value(o.byte), tn.t);
        o.r = __frcp_rn(o.s);
        if (!o.finite) o.byte = 0x7F;
    } else {
        const uint32_t b = __float_as_uint(amax);
        int e = static_cast<int>((b >> 23) & 0xFFu) - 2 + ((b & 0x7FFFFFu) > 0x400000u ? 1 : 0);
        e = e < 0 ? 0 : e;
        o.byte = static_cast<uint32_t>(e);
        if (!o.finite) { o.byte = 0xFF; e = 127; }
        o.r = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        o.s = 0.0f;                                  // not used
    }
    return o;
}

// x / S, correctly rounded. mx: a power of two. nv: one step of Markstein's
// correction (P. Markstein, IBM J. Res. Dev. 34, 1990): from the correctly
// rounded reciprocal r, q = x r is within an ulp of x / S, and q + r (x - q S)
// with the residual exact in an FMA rounds to the quotient. Halfway cases of
// E2M1 (x = S times a midpoint, common for bf16 x) are therefore kept.
template <int FMT>
__device__ __forceinline__ float fp4_quot(float x, const Fp4Scale& g) {
    const float q = __fmul_rn(x, g.r);
    if constexpr (FMT == kFp4Mx) return q;
    return __fmaf_rn(__fmaf_rn(-q, g.s, x), g.r, q);
}

// Sixteen values of one group (or half an mx group) to two words of codes.
template <int FMT>
__device__ __forceinline__ uint2 fp4_codes16(const float (&x)[16], const Fp4Scale& g) {
    float v[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = fp4_quot<FMT>(x[i], g);
        w[i] = fp4_quot<FMT>(x[8 + i], g);
    }
    uint2 o = make_uint2(e2m1x8(v), e2m1x8(w));
    if (!g.finite) o = make_uint2(0u, 0u);
    return o;
}

__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Sixteen consecutive elements of a row as they lie in memory.
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
    uint4 u[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        u[0] = __ldg(reinterpret_cast<const uint4*>(p));
        u[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { u[0] = u[1] = make_uint4(0, 0, 0, 0); }
    // element by element, `n` of them (0 .. 16), `s` elements apart
    __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int64_t s, int n) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo = 0, hi = 0;
            if (2 * i < n) lo = __bfloat16_as_ushort(p[(2 * i) * s]);
            if (2 * i + 1 < n) hi = __bfloat16_as_ushort(p[(2 * i + 1) * s]);
            w[i] = lo | (hi << 16);
        }
        u[0] = make_uint4(w[0], w[1], w[2], w[3]);
        u[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    __device__ __forceinline__ float amax() const {
        const uint32_t k = 0x7FFF7FFFu;
        uint32_t m = bf16x2_max_nan(bf16x2_max_nan(u[0].x & k, u[0].y & k), bf16x2_max_nan(u[0].z & k, u[0].w & k));
        m = bf16x2_max_nan(m, bf16x2_max_nan(bf16x2_max_nan(u[1].x & k, u[1].y & k),
                                             bf16x2_max_nan(u[1].z & k, u[1].w & k)));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
    __device__ __forceinline__ void values(float (&v)[16]) const {
        unpack8(u[0], v);
        unpack8(u[1], v + 8);
    }
};
template <>
struct Raw16<float> {
    float f[16];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(f + 4 * i) = __ldg(reinterpret_cast<const float4*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 0.0f;
    }
    __device__ __forceinline__ void load_some(const float* p, int64_t s, int n) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = i < n ? p[i * s] : 0.0f;
    }
    __device__ __forceinline__ float amax() const {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max_nan(m, fabsf(f[i]));
        return m;
    }
    __device__ __forceinline__ void values(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = f[i];
    }
};
#endif

}  // namespace ql
