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
// A group with an infinity or a NaN (or, nv, whose amax / (6 t) overflows) gets
// the scale NaN (0x7F / 0xFF), so it is NaN in every product and when it is read
// back, whatever its codes.
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
    Bounds bnd;                // x, row codes, row scales, offsets, column codes, column scales
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
    Bounds bnd;                // x, row codes, row scales, offsets, column codes, column scales
};

// The scale t of x [m][k], or of the rows that experts have: [offsets[0],
// offsets[num_experts]), inside [0, m].
struct Fp4ScaleArgs {
    const void* x;
    bool is_bf16;
    int64_t m, k;
    int64_t sxm, sxk;
    const int32_t* offsets;    // or null
    int num_experts;
    float* t;
    Bounds bnd;                // x, offsets
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
    Bounds bnd;                // out, codes, scales
};

cudaError_t launch_fp4_cast(const Fp4CastArgs& a, cudaStream_t st, int num_sms);
cudaError_t launch_fp4_cast_dual(const Fp4DualArgs& a, cudaStream_t st);
cudaError_t launch_fp4_dequant(const Fp4DequantArgs& a, cudaStream_t st, int num_sms);
cudaError_t launch_fp4_tensor_scale(const Fp4ScaleArgs& a, cudaStream_t st, int num_sms);

#ifdef __CUDACC__
// Larger of two magnitudes; a NaN operand gives NaN. The bf16 form takes two
// pairs of values of any sign and leaves signs that the caller drops.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_maxabs_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Two fp32 values in one 64-bit register: one instruction, each half rounded
// as the scalar operation.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void f32x2_get(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float rcp_approx(float v) {        // within 1 ulp
    float d;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
    return d;
}

// Eight values to eight E2M1 codes (v[0] lowest), round to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8(const uint64_t (&v)[4]) {
    uint32_t d;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        ".reg .f32 l0, h0, l1, h1, l2, h2, l3, h3;\n"
        "mov.b64 {l0, h0}, %1;\n"
        "mov.b64 {l1, h1}, %2;\n"
        "mov.b64 {l2, h2}, %3;\n"
        "mov.b64 {l3, h3}, %4;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, h0, l0;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, h1, l1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, h2, l2;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, h3, l3;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n"
        "}\n"
        : "=r"(d)
        : "l"(v[0]), "l"(v[1]), "l"(v[2]), "l"(v[3]));
    return d;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
    return __half2float(__half(h));
}

// The tensor's scale as the groups' scales use it.
struct Fp4Tensor {
    float t, t6, r6;     // t, 6 t, 1 / (6 t)
};
__device__ __forceinline__ Fp4Tensor fp4_tensor(const float* tscale) {
    Fp4Tensor o;
    o.t = tscale != nullptr ? __ldg(tscale) : 1.0f;
    o.t6 = __fmul_rn(6.0f, o.t);
    o.r6 = __frcp_rn(o.t6);
    return o;
}

// a / b from r, 1 / b within an ulp: q = a r is within a few ulps, the residual
// a - q b is exact in an FMA, and q + r (a - q b) is a / b to within 2^-44
// before it is rounded (the last step of P. Markstein, IBM J. Res. Dev. 34,
// 1990). A quotient that fp32 holds, such as a halfway case of E2M1, is found
// exactly; with t a power of two S has four significant bits, no other quotient
// is that near to a rounding boundary, and the result is the correctly rounded
// one.
__device__ __forceinline__ float quot(float a, float b, float r) {
    const float q = __fmul_rn(a, r);
    return __fmaf_rn(__fmaf_rn(-q, b, a), r, q);
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Scale of one group: its stored byte and what its elements are divided by.
// nv: S and 1 / S; mx: the power of two 1 / S alone. nv: an amax of infinity or
// NaN makes the quotient, and with it the byte, NaN.
struct Fp4Scale {
    uint32_t byte;
    float s, r;
};
template <int FMT>
__device__ __forceinline__ Fp4Scale fp4_scale(float amax, const Fp4Tensor& tn) {
    Fp4Scale o;
    if constexpr (FMT == kFp4Nv) {
        const float d = min_nan(max_nan(quot(amax, tn.t6, tn.r6), 0.001953125f), 448.0f);
        o.byte = static_cast<uint32_t>(__nv_cvt_float_to_fp8(d, __NV_SATFINITE, __NV_E4M3));
        o.s = __fmul_rn(e4m3_value(o.byte), tn.t);
        o.r = rcp_approx(o.s);
    } else {
        const uint32_t b = __float_as_uint(amax);
        // exponent of amax / 6 rounded up: amax > 1.5 * 2^(e + 2) takes the next
        int e = static_cast<int>((b + 0x3FFFFFu) >> 23) - 2;
        e = e < 0 ? 0 : e;
        o.byte = b >= 0x7F800000u ? 0xFFu : static_cast<uint32_t>(e);
        o.r = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        o.s = 0.0f;                                  // not used
    }
    return o;
}

// Sixteen values of one group (or half an mx group), as pairs, to two words of codes.
template <int FMT>
__device__ __forceinline__ uint2 fp4_codes16(const uint64_t (&x)[8], const Fp4Scale& g) {
    const uint64_t r = f32x2(g.r, g.r);
    uint64_t v[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint64_t q = mul2(x[i], r);
        if constexpr (FMT == kFp4Nv) {
            const uint64_t ns = f32x2(-g.s, -g.s);
            q = fma2(fma2(q, ns, x[i]), r, q);
        }
        v[i >> 2][i & 3] = q;
    }
    return make_uint2(e2m1x8(v[0]), e2m1x8(v[1]));
}

__device__ __forceinline__ uint64_t bf16x2_f32x2(uint32_t w) {
    return f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// The larger magnitude of a pair that bf16x2_maxabs_nan left.
__device__ __forceinline__ float bf16x2_amax(uint32_t m) {
    return max_nan(__uint_as_float((m << 16) & 0x7FFFFFFFu), __uint_as_float(m & 0x7FFF0000u));
}

// Sixteen consecutive elements of a row as they lie in memory.
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
    uint4 u[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p, const Bounds& b, int i) {
        if (!QL_IN(b, i, p, 32)) return zero();
        u[0] = __ldg(reinterpret_cast<const uint4*>(p));
        u[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { u[0] = u[1] = make_uint4(0, 0, 0, 0); }
    // element by element, `n` of them (0 .. 16), `s` elements apart
    __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int64_t s, int n, const Bounds& b, int bi) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo = 0, hi = 0;
            if (2 * i < n && QL_IN(b, bi, p + (2 * i) * s, 2)) lo = __bfloat16_as_ushort(p[(2 * i) * s]);
            if (2 * i + 1 < n && QL_IN(b, bi, p + (2 * i + 1) * s, 2)) hi = __bfloat16_as_ushort(p[(2 * i + 1) * s]);
            w[i] = lo | (hi << 16);
        }
        u[0] = make_uint4(w[0], w[1], w[2], w[3]);
        u[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    __device__ __forceinline__ float amax() const {
        const uint32_t a = bf16x2_maxabs_nan(bf16x2_maxabs_nan(u[0].x, u[0].y), bf16x2_maxabs_nan(u[0].z, u[0].w));
        const uint32_t b = bf16x2_maxabs_nan(bf16x2_maxabs_nan(u[1].x, u[1].y), bf16x2_maxabs_nan(u[1].z, u[1].w));
        return bf16x2_amax(bf16x2_maxabs_nan(a, b));
    }
    __device__ __forceinline__ void values(uint64_t (&v)[8]) const {
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bf16x2_f32x2(w[i]);
    }
};
template <>
struct Raw16<float> {
    float f[16];
    __device__ __forceinline__ void load(const float* p, const Bounds& b, int bi) {
        if (!QL_IN(b, bi, p, 64)) return zero();
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(f + 4 * i) = __ldg(reinterpret_cast<const float4*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 0.0f;
    }
    __device__ __forceinline__ void load_some(const float* p, int64_t s, int n, const Bounds& b, int bi) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = i < n && QL_IN(b, bi, p + i * s, 4) ? p[i * s] : 0.0f;
    }
    __device__ __forceinline__ float amax() const {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max_nan(m, fabsf(f[i]));
        return m;
    }
    __device__ __forceinline__ void values(uint64_t (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f32x2(f[2 * i], f[2 * i + 1]);
    }
};
#endif

}  // namespace ql
