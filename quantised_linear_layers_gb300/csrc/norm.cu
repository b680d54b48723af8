// Layer norm: y = (x - mean) rstd w + b over the rows of x, and its gradients.
//
// mean and variance are those of the row's own elements in fp32: a first sum for
// the mean, then sums of d = x - mean and of d^2, whose first corrects the mean's
// rounding (so rows far from zero lose nothing to it).
//
// Backward, with h = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum(g) / n - h sum(g h) / n),  dw = sum_rows dy h,  db = sum_rows dy
#include "norm.cuh"

#include "rows.cuh"

namespace ql {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kSms = 152;             // for sizes that a caller asks for without a device

template <typename B>
__device__ __forceinline__ float weight_at(const void* w, bool bf16, int64_t i, const B& b, int span) {
    return bf16 ? to_f32(load_one(static_cast<const __nv_bfloat16*>(w) + i, b, span, from_f32<__nv_bfloat16>(0.0f)))
                : load_one(static_cast<const float*>(w) + i, b, span, 0.0f);
}

// ---------------------------------------------------------------- any length
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) norm_any_kernel(const NormArgs p) {
    __shared__ float s_sum[4 * 32];
    pdl_launch_dependents();
    pdl_wait_prior();
    const float n = static_cast<float>(p.n);
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + row * p.sx;
        O* y = static_cast<O*>(p.y) + row * p.sy;
        const T zero = from_f32<T>(0.0f);
        float one[1] = {0.0f};
        for (int64_t i = threadIdx.x; i < p.n; i += kThreads) one[0] += to_f32(load_one(x + i, p.bnd, 0, zero));
        __syncthreads();                     // the last row's sums have been read
        sum_over_row<1, false>(one, s_sum);
        const float about = one[0] / n;
        float two[2] = {0.0f, 0.0f};
        for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
            const float d = to_f32(load_one(x + i, p.bnd, 0, zero)) - about;
            two[0] += d;
            two[1] = fmaf(d, d, two[1]);
        }
        sum_over_row<2, false>(two, s_sum + 32);
        const float off = two[0] / n;
        const float rstd = 1.0f / sqrtf(fmaxf(two[1] / n - off * off, 0.0f) + p.eps);
        if (p.mean != nullptr && threadIdx.x == 0) {
            store_one(p.mean + row, about + off, p.bnd, 4);
            store_one(p.rstd + row, rstd, p.bnd, 5);
        }
        for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
            float h = (to_f32(load_one(x + i, p.bnd, 0, zero)) - about - off) * rstd;
            if (p.w != nullptr) h *= weight_at(p.w, p.w_bf16, i, p.bnd, 1);
            if (p.b != nullptr) h += weight_at(p.b, p.w_bf16, i, p.bnd, 2);
            store_one(y + i, from_f32<O>(h), p.bnd, 3);
        }
    }
}

template <typename T, typename D>
__global__ void __launch_bounds__(kThreads) norm_dx_any_kernel(const NormBackArgs p) {
    __shared__ float s_sum[2 * 32];
    pdl_launch_dependents();
    pdl_wait_prior();
    const float n = static_cast<float>(p.n);
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + row * p.sx;
        const D* dy = static_cast<const D*>(p.dy) + row * p.sdy;
        T* dx = static_cast<T*>(p.dx) + row * p.sdx;
        const float mean = load_one(p.mean + row, p.bnd, 2, 0.0f), rstd = load_one(p.rstd + row, p.bnd, 3, 0.0f);
        float c[2] = {0.0f, 0.0f};
        for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
            float g = to_f32(load_one(dy + i, p.bnd, 0, from_f32<D>(0.0f)));
            if (p.w != nullptr) g *= weight_at(p.w, p.w_bf16, i, p.bnd, 4);
            c[0] += g;
            c[1] = fmaf(g, (to_f32(load_one(x + i, p.bnd, 1, from_f32<T>(0.0f))) - mean) * rstd, c[1]);
        }
        __syncthreads();
        sum_over_row<2, false>(c, s_sum);
        const float c1 = c[0] / n, c2 = c[1] / n;
        for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
            float g = to_f32(load_one(dy + i, p.bnd, 0, from_f32<D>(0.0f)));
            if (p.w != nullptr) g *= weight_at(p.w, p.w_bf16, i, p.bnd, 4);
            const float h = (to_f32(load_one(x + i, p.bnd, 1, from_f32<T>(0.0f))) - mean) * rstd;
            store_one(dx + i, from_f32<T>(rstd * (g - c1 - h * c2)), p.bnd, 5);
        }
    }
}

// Sums of dy h and dy over the rows of a part, a column per thread of a row of
// threads; part blockIdx.y has rows [y * rows, (y + 1) * rows).
template <typename T, typename D>
__global__ void __launch_bounds__(kThreads) norm_dw_any_kernel(const NormBackArgs p, int64_t rows) {
    pdl_launch_dependents();
    pdl_wait_prior();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (col >= p.n) return;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows, r1 = r0 + rows < p.m ? r0 + rows : p.m;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = to_f32(load_one(static_cast<const D*>(p.dy) + r * p.sdy + col, p.bnd, 0, from_f32<D>(0.0f)));
        const float x = to_f32(load_one(static_cast<const T*>(p.x) + r * p.sx + col, p.bnd, 1, from_f32<T>(0.0f)));
        dw = fmaf(dy, (x - load_one(p.mean + r, p.bnd, 2, 0.0f)) * load_one(p.rstd + r, p.bnd, 3, 0.0f), dw);
        db += dy;
    }
    float* part = p.part + static_cast<int64_t>(blockIdx.y) * 2 * p.n;
    store_one(part + col, dw, p.bnd, 6);
    store_one(part + p.n + col, db, p.bnd, 6);
}

// dw and db: the parts' sums, 32 columns by 8 shares of the parts per block, in a
// fixed order.
__global__ void __launch_bounds__(kThreads) norm_dw_join_kernel(const NormBackArgs p, int parts) {
    __shared__ float s[8][33];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + tx;      // of 2 n
    float v = 0.0f;
    if (col < 2 * p.n)
#pragma unroll 4
        for (int i = ty; i < parts; i += 8) v += load_one(p.part + i * 2 * p.n + col, p.bnd, 6, 0.0f);
    s[ty][tx] = v;
    __syncthreads();
    if (ty == 0 && col < 2 * p.n) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][tx];
        if (col < p.n) store_one(p.dw + col, v, p.bnd, 7);
        else store_one(p.db + col - p.n, v, p.bnd, 8);
    }
}

unsigned grid_of(int64_t n, int64_t most) { return static_cast<unsigned>(n < 1 ? 1 : (n < most ? n : most)); }

// Parts of the rows for the column sums: enough blocks for every SM to have four.
int64_t any_parts(int64_t m, int64_t n) {
    const int64_t cols = (n + kThreads - 1) / kThreads;
    int64_t parts = (kSms * 4 + cols - 1) / cols;
    if (parts > (m + 15) / 16) parts = (m + 15) / 16;
    return parts < 1 ? 1 : parts;
}

template <typename T, typename O>
cudaError_t norm_t(const NormArgs& a, cudaStream_t st, int num_sms) {
    return launch_after(norm_any_kernel<T, O>, dim3(grid_of(a.m, static_cast<int64_t>(num_sms) * 8)), kThreads, 0, st, a);
}

template <typename T, typename D>
cudaError_t back_t(const NormBackArgs& a, cudaStream_t st, int num_sms) {
    if (cudaError_t e = launch_after(norm_dx_any_kernel<T, D>, dim3(grid_of(a.m, static_cast<int64_t>(num_sms) * 8)), kThreads, 0, st, a);
        e != cudaSuccess || a.dw == nullptr)
        return e;
    const int64_t parts = any_parts(a.m, a.n), rows = (a.m + parts - 1) / parts;
    if (cudaError_t e = launch_after(norm_dw_any_kernel<T, D>, dim3(static_cast<unsigned>((a.n + kThreads - 1) / kThreads), static_cast<unsigned>(parts)),
                                     kThreads, 0, st, a, rows);
        e != cudaSuccess)
        return e;
    return launch_after(norm_dw_join_kernel, dim3(static_cast<unsigned>((2 * a.n + 31) / 32)), kThreads, 0, st, a, static_cast<int>(parts));
}

}  // namespace

size_t norm_back_workspace(int64_t m, int64_t n) {
    return static_cast<size_t>(any_parts(m, n)) * 2 * static_cast<size_t>(n) * sizeof(float);
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st, int num_sms) {
    if (a.x_bf16) return a.y_bf16 ? norm_t<__nv_bfloat16, __nv_bfloat16>(a, st, num_sms) : norm_t<__nv_bfloat16, float>(a, st, num_sms);
    return a.y_bf16 ? norm_t<float, __nv_bfloat16>(a, st, num_sms) : norm_t<float, float>(a, st, num_sms);
}

cudaError_t launch_norm_back(const NormBackArgs& a, cudaStream_t st, int num_sms) {
    if (a.x_bf16) return a.dy_bf16 ? back_t<__nv_bfloat16, __nv_bfloat16>(a, st, num_sms) : back_t<__nv_bfloat16, float>(a, st, num_sms);
    return a.dy_bf16 ? back_t<float, __nv_bfloat16>(a, st, num_sms) : back_t<float, float>(a, st, num_sms);
}

}  // namespace ql
