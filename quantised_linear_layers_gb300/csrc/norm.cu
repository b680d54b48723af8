// Layer norm: y = (x - mean) rstd w + b over the rows of x. Backward: norm_back.cu.
//
// mean and variance are those of the row's own elements in fp32: a first sum for
// the mean, then sums of d = x - mean and of d^2, whose first corrects the mean's
// rounding (so rows far from zero lose nothing to it). A row is read once and stays
// in its threads' registers, as pairs of fp32; bound by memory, and by instructions
// next to it. 16384 x 7168 bf16: 75.4 us, 0.92 of a copy's rate; one row 2.8 us, a launch.
#include "gemm.cuh"
#include "norm.cuh"
#include "norm_rows.cuh"

namespace ql {
namespace {

constexpr int kThreads = 256;

// A run's deviations from `about`, in its place, and the sums of them and of their squares;
// runs from column n on stay zero.
template <int W>
__device__ __forceinline__ void deviations(F2* v, float about, int c, int n, F2& s1, F2& s2) {
    const F2 off = f2(-about, -about);
    if (c < n) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) v[i] = add2(v[i], off);
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        s1 = add2(s1, v[i]);
        s2 = fma2(v[i], v[i], s2);
    }
}

// From the mean of the deviations and that of their squares; NaN stays NaN.
__device__ __forceinline__ float rstd_of(float m1, float m2, float eps) {
    const float var = fmaf(-m1, m1, m2);
    return rsqrtf((var < 0.0f ? 0.0f : var) + eps);
}

// Two sums over a warp's or a block's row.
template <bool WARP>
__device__ __forceinline__ void team_sum(float& a, float& b, float* s) {
    if constexpr (WARP) {
        const float v = sums_over_warp(a, b);
        a = __shfl_sync(0xffffffffu, v, 0);
        b = __shfl_sync(0xffffffffu, v, 16);
    } else {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        float v = sums_over_warp(a, b);
        if ((lane & 15) == 0) s[(lane >> 4) * 32 + (threadIdx.x >> 5)] = v;
        __syncthreads();
        a = lane < warps ? s[lane] : 0.0f;
        b = lane < warps ? s[32 + lane] : 0.0f;
        v = sums_over_warp(a, b);
        a = __shfl_sync(0xffffffffu, v, 0);
        b = __shfl_sync(0xffffffffu, v, 16);
    }
}

// ---------------------------------------------------------------- rows in registers
// Element i of run u of thread t: whole vectors, or (SPREAD) elements a team apart, which
// take any boundary and any length and are whole lines to a warp all the same.
template <int W, bool SPREAD>
__device__ __forceinline__ int column(int u, int i, int t, int team) {
    return SPREAD ? (u * W + i) * team + t : (u * team + t) * W + i;
}
template <int W, bool SPREAD, typename T, typename B>
__device__ __forceinline__ void load_columns(F2* v, const T* row, int u, int t, int team, int n, const B& bnd, int span) {
    Pack<T, W> p = zero_pack<T, W>();
    if constexpr (SPREAD) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (column<W, true>(u, i, t, team) < n) p.v[i] = load_one(row + column<W, true>(u, i, t, team), bnd, span, p.v[i]);
    } else if (column<W, false>(u, 0, t, team) < n) {
        p = load_pack<T, W>(row + column<W, false>(u, 0, t, team), bnd, span);
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) v[i] = pair_of<W>(p, i);
}
template <int W, bool SPREAD, typename B>
__device__ __forceinline__ void load_weight_columns(F2* v, const void* p, bool bf16, float other, int u, int t, int team, int n, const B& bnd, int span) {
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) v[i] = f2(other, other);
    } else if (bf16) {
        load_columns<W, SPREAD>(v, static_cast<const __nv_bfloat16*>(p), u, t, team, n, bnd, span);
    } else {
        load_columns<W, SPREAD>(v, static_cast<const float*>(p), u, t, team, n, bnd, span);
    }
}

// A row to a warp (eight rows to a block) or to a block.
template <typename T, typename O, int W, int E, bool WARP, bool SPREAD>
__global__ void __launch_bounds__(WARP ? 256 : (E <= 8 ? 1024 : 512)) norm_kernel(const NormArgs p) {
    constexpr int U = E / W, H = W / 2;
    __shared__ float s_sum[WARP ? 1 : 2 * 64];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int t = WARP ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int team = WARP ? 32 : static_cast<int>(blockDim.x);
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5) : static_cast<int64_t>(blockIdx.x);
    if (row >= p.m) return;
    const int n = static_cast<int>(p.n);
    const T* x = static_cast<const T*>(p.x) + row * p.sx;
    F2 v[E / 2], sum = 0ull;
#pragma unroll
    for (int u = 0; u < U; ++u) load_columns<W, SPREAD>(v + u * H, x, u, t, team, n, p.bnd, 0);
    // where registers hold them, the weights are on their way beside the row: 1003 x 4099 fp32 13.0 -> 11.7 us
    constexpr bool EARLY = E <= 8;
    F2 w0[EARLY ? E / 2 : 1], b0[EARLY ? E / 2 : 1];
    if constexpr (EARLY) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            load_weight_columns<W, SPREAD>(w0 + u * H, p.w, p.w_bf16, 1.0f, u, t, team, n, p.bnd, 1);
            load_weight_columns<W, SPREAD>(b0 + u * H, p.b, p.w_bf16, 0.0f, u, t, team, n, p.bnd, 2);
        }
    }
#pragma unroll
    for (int e = 0; e < E / 2; ++e) sum = add2(sum, v[e]);
    const float inv_n = 1.0f / static_cast<float>(n);
    float about = sum2(sum), none = 0.0f;
    team_sum<WARP>(about, none, s_sum);
    about *= inv_n;
    F2 s1 = 0ull, s2 = 0ull;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < H; ++i) {                      // elements past the row's end stay zero
            F2& d = v[u * H + i];
            if constexpr (SPREAD) {
                float a, b;
                unpack(d, a, b);
                d = f2(column<W, true>(u, 2 * i, t, team) < n ? a - about : 0.0f, column<W, true>(u, 2 * i + 1, t, team) < n ? b - about : 0.0f);
            } else if (column<W, false>(u, 0, t, team) < n) {
                d = add2(d, f2(-about, -about));
            }
            s1 = add2(s1, d);
            s2 = fma2(d, d, s2);
        }
    float m1 = sum2(s1), m2 = sum2(s2);
    team_sum<WARP>(m1, m2, s_sum + (WARP ? 0 : 64));
    m1 *= inv_n;
    const float rstd = rstd_of(m1, m2 * inv_n, p.eps);
    if (p.mean != nullptr && t == 0) {
        store_one(p.mean + row, about + m1, p.bnd, 4);
        store_one(p.rstd + row, rstd, p.bnd, 5);
    }
    const F2 r2 = f2(rstd, rstd), back = f2(-m1 * rstd, -m1 * rstd);
    O* y = static_cast<O*>(p.y) + row * p.sy;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (column<W, SPREAD>(u, 0, t, team) >= n) continue;
        F2 w[H], b[H];
        if constexpr (EARLY) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
                w[i] = w0[u * H + i];
                b[i] = b0[u * H + i];
            }
        } else {
            load_weight_columns<W, SPREAD>(w, p.w, p.w_bf16, 1.0f, u, t, team, n, p.bnd, 1);
            load_weight_columns<W, SPREAD>(b, p.b, p.w_bf16, 0.0f, u, t, team, n, p.bnd, 2);
        }
        Pack<O, W> o;
#pragma unroll
        for (int i = 0; i < H; ++i) set_pair<W>(o, i, fma2(fma2(v[u * H + i], r2, back), w[i], b[i]));
        if constexpr (SPREAD) {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (column<W, true>(u, i, t, team) < n) store_one(y + column<W, true>(u, i, t, team), o.v[i], p.bnd, 3);
        } else {
            store_pack<O, W>(y + column<W, false>(u, 0, t, team), o, p.bnd, 3);
        }
    }
}

// ---------------------------------------------------------------- many rows
// The same by teams with their rows on the way through shared memory, R rows at a time
// so that their sums share exchanges and barriers: a row's arithmetic is 6 instructions
// an element, and a thread's part of the sums 100 a row were it alone. Rows are found by
// index: of the 72 registers that 896 threads have none is left for addresses, and what
// spills goes to L2, with so little L1 beside the ring (16384 x 7168 75 us, 83 with
// addresses kept; 4096 x 7167 32 and 37).
template <typename T, typename O, int E, bool EDGE>
__global__ void __launch_bounds__(E <= 16 ? 896 : 512) norm_rows_kernel(const NormArgs p, const Teams f, bool y_vec, bool w_vec) {
    constexpr int W = 16 / sizeof(T), U = E / W, H = W / 2, XB = 16;
    constexpr int R = E <= 16 ? 2 : 1;                     // (32 elements twice: no registers left)
    extern __shared__ __align__(16) uint8_t s_mem[];
    __shared__ float s_sum[2][128];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int id = static_cast<int>(threadIdx.x) / f.team, t = static_cast<int>(threadIdx.x) - id * f.team;
    const uint32_t rows = static_cast<uint32_t>(p.m), first = blockIdx.x + gridDim.x * id, step = gridDim.x * f.teams;
    const int all = static_cast<int>(blockDim.x);
    Ends end{0, static_cast<int>(p.n), -1};
    if constexpr (EDGE) end = ends_of<W>(static_cast<int>((f.at.base + static_cast<int64_t>(blockIdx.x) * f.at.stride) % W), static_cast<int>(p.n), t >= f.team - 32);
    const int n = end.tail;                                // of the runs
    const int c0 = end.head + t * W, cu = f.team * W;      // run u starts at column c0 + u * cu

    // [stage][R][U] runs, a thread's side by side; then a team's weights and biases, [2][E];
    // then (EDGE) [stage][R][teams] words of the lanes that have a row's ends
    const int line = all * E * static_cast<int>(sizeof(T)), stage = R * line;
    uint8_t* my_x = s_mem + threadIdx.x * XB;
    ulonglong2* my_w = reinterpret_cast<ulonglong2*>(s_mem + f.stages * stage) + t;               // + i * team
    uint32_t* my_end = reinterpret_cast<uint32_t*>(s_mem + f.stages * stage + f.team * E * 8) + id * 32 + (t & 31);
    const int end_row = f.teams * 32;                      // words
    if (n < U * cu)
        for (int s = 0; s < f.stages * R * U; ++s) *reinterpret_cast<uint4*>(my_x + s * all * XB) = make_uint4(0u, 0u, 0u, 0u);
    const T* x = static_cast<const T*>(p.x);
    const OneOf<T> one_of(x + first * p.sx, end.col, static_cast<int>(p.n), p.sx);
    auto fetch = [&](int at, int turn, uint32_t row) {     // R rows from that on into the turn-th stage, which begins at byte `at`
#pragma unroll
        for (int r = 0; r < R; ++r, row += step)
            if (row < rows) {
                const T* from = x + row * p.sx;
#pragma unroll
                for (int u = 0; u < U; ++u) fetch_run<W>(my_x + at + r * line + u * all * XB, from, c0 + u * cu, n, true, p.bnd, 0);
                if (EDGE && end.col >= 0) one_of.fetch(my_end + (turn * R + r) * end_row, from + end.col, row, rows, p.bnd, 0);
            }
        copy_commit();                                     // a group for every stage, also past the last row
    };
    // the weights between the first stage and the rest: behind all of them they wait for the ring to fill
    fetch(0, 0, first);
    if (id == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            F2 w[H], b[H];
            weight_run<W>(w, p.w, p.w_bf16, 1.0f, c0 + u * cu, n, !EDGE || (w_vec && end.head == 0), p.bnd, 1);
            weight_run<W>(b, p.b, p.w_bf16, 0.0f, c0 + u * cu, n, !EDGE || (w_vec && end.head == 0), p.bnd, 2);
#pragma unroll
            for (int i = 0; i < H / 2; ++i) {
                my_w[(u * (H / 2) + i) * f.team] = make_ulonglong2(w[2 * i], w[2 * i + 1]);
                my_w[(E / 4 + u * (H / 2) + i) * f.team] = make_ulonglong2(b[2 * i], b[2 * i + 1]);
            }
        }
    }
    float end_w = 0.0f, end_b = 0.0f;
    if (EDGE && end.col >= 0) {
        end_w = weight_one(p.w, p.w_bf16, 1.0f, end.col, p.bnd, 1);
        end_b = weight_one(p.b, p.w_bf16, 0.0f, end.col, p.bnd, 2);
    }
    for (int s = 1; s < f.stages; ++s) fetch(s * stage, s, first + s * R * step);
    __syncthreads();
    const float inv_n = 1.0f / static_cast<float>(p.n);
    int at = 0, turn = 0;
    for (uint32_t row = first; row < rows; row += R * step) {
        copy_wait(f.stages);
        F2 v[R][E / 2];
        float one[R];                                      // of the row's ends
        float about[2] = {0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            F2 sum = 0ull;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Pack<T, W> x = *reinterpret_cast<const Pack<T, W>*>(my_x + at + r * line + u * all * XB);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    v[r][u * H + i] = pair_of<W>(x, i);
                    sum = add2(sum, v[r][u * H + i]);
                }
            }
            about[r] = sum2(sum);
            if (EDGE && end.col >= 0) {
                one[r] = one_of.value(my_end + (turn * R + r) * end_row);
                about[r] += one[r];
            }
        }
        fetch(at, turn, row + f.stages * R * step);                                   // the rows are in registers
        at += stage;
        if (++turn == f.stages) at = turn = 0;
        sum_over_team(about[0], about[1], s_sum[0], f.team, id);
        float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};             // sums of d, then of d^2
#pragma unroll
        for (int r = 0; r < R; ++r) {
            about[r] *= inv_n;
            F2 s1 = 0ull, s2 = 0ull;
#pragma unroll
            for (int u = 0; u < U; ++u) deviations<W>(v[r] + u * H, about[r], c0 + u * cu, n, s1, s2);
            m[r] = sum2(s1);
            m[2 + r] = sum2(s2);
            if (EDGE && end.col >= 0) {
                one[r] -= about[r];
                m[r] += one[r];
                m[2 + r] = fmaf(one[r], one[r], m[2 + r]);
            }
        }
        if constexpr (R == 2) sum4_over_team(m, s_sum[1], f.team, id);
        else sum_over_team(m[0], m[2], s_sum[1], f.team, id);
        F2 r2[R], back[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float m1 = m[r] * inv_n, rstd = rstd_of(m1, m[2 + r] * inv_n, p.eps);
            if (p.mean != nullptr && t == 0 && row + r * step < rows) {
                store_one(p.mean + row + r * step, about[r] + m1, p.bnd, 4);
                store_one(p.rstd + row + r * step, rstd, p.bnd, 5);
            }
            r2[r] = f2(rstd, rstd);
            back[r] = f2(-m1 * rstd, -m1 * rstd);
            if (EDGE && end.col >= 0 && row + r * step < rows)
                store_one(static_cast<O*>(p.y) + (row + r * step) * p.sy + end.col, from_f32<O>(fmaf(fmaf(one[r], rstd, -m1 * rstd), end_w, end_b)), p.bnd, 3);
        }
        O* y = static_cast<O*>(p.y) + row * p.sy;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * cu;
            if (c >= n) continue;
            F2 o[R][H];
#pragma unroll
            for (int i = 0; i < H / 2; ++i) {
                const ulonglong2 w = my_w[(u * (H / 2) + i) * f.team], b = my_w[(E / 4 + u * (H / 2) + i) * f.team];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    o[r][2 * i] = fma2(fma2(v[r][u * H + 2 * i], r2[r], back[r]), w.x, b.x);
                    o[r][2 * i + 1] = fma2(fma2(v[r][u * H + 2 * i + 1], r2[r], back[r]), w.y, b.y);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r == 0 || row + r * step < rows) store_run<W>(y + r * step * p.sy, o[r], c, n, !EDGE || y_vec, p.bnd, 3);
        }
    }
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
        LongSum sum;
        for (int64_t i0 = threadIdx.x; i0 < p.n; i0 += kLongRun * kThreads) {
            const int64_t i1 = i0 + long_run(i0, p.n, kThreads) * kThreads;
            float run = 0.0f;
#pragma unroll 16
            for (int64_t i = i0; i < i1; i += kThreads) run += to_f32(load_one(x + i, p.bnd, 0, zero));
            sum.add(run);
        }
        float one[1] = {sum.value()};
        __syncthreads();                     // the last row's sums have been read
        sum_over_row<1, false>(one, s_sum);
        const float about = one[0] / n;
        LongSum s1, s2;
        for (int64_t i0 = threadIdx.x; i0 < p.n; i0 += kLongRun * kThreads) {
            const int64_t i1 = i0 + long_run(i0, p.n, kThreads) * kThreads;
            float r1 = 0.0f, r2 = 0.0f;
#pragma unroll 16
            for (int64_t i = i0; i < i1; i += kThreads) {
                const float d = to_f32(load_one(x + i, p.bnd, 0, zero)) - about;
                r1 += d;
                r2 = fmaf(d, d, r2);
            }
            s1.add(r1);
            s2.add(r2);
        }
        float two[2] = {s1.value(), s2.value()};
        sum_over_row<2, false>(two, s_sum + 32);
        const float off = two[0] / n;
        const float rstd = rstd_of(off, two[1] / n, p.eps);
        if (p.mean != nullptr && threadIdx.x == 0) {
            store_one(p.mean + row, about + off, p.bnd, 4);
            store_one(p.rstd + row, rstd, p.bnd, 5);
        }
        for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
            const float h = (to_f32(load_one(x + i, p.bnd, 0, zero)) - about - off) * rstd;
            float w[1], b[1];
            load_weights<1>(w, p.w, p.w_bf16, i, 1.0f, p.bnd, 1);
            load_weights<1>(b, p.b, p.w_bf16, i, 0.0f, p.bnd, 2);
            store_one(y + i, from_f32<O>(fmaf(h, w[0], b[0])), p.bnd, 3);
        }
    }
}

// Whether a call's rows are whole aligned vectors.
template <typename T, typename O>
bool whole_vectors(const NormArgs& a) {
    constexpr int W = 16 / sizeof(T);
    const Boundary x = boundary_of(a.x, sizeof(T), a.sx, a.m, W);
    return x.base == 0 && x.stride == 0 && a.n % W == 0 && same_boundary(x, boundary_of(a.y, sizeof(O), a.sy, a.m, W)) &&
           aligned_to(a.w, 16) && aligned_to(a.b, 16);
}

template <typename T, typename O, int E, bool WARP>
cudaError_t norm_e(const NormArgs& a, bool whole, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    const dim3 grid(static_cast<unsigned>(WARP ? (a.m + 7) / 8 : a.m));
    const int threads = WARP ? 256 : team_of(a.n, E);
    if (whole) return launch_after(norm_kernel<T, O, W, E, WARP, false>, grid, threads, 0, st, a);
    return launch_after(norm_kernel<T, O, W, E, WARP, true>, grid, threads, 0, st, a);
}

// Rows to a team from which the ring pays for its start (for fp32 it is half as many rows
// deep). Measured, teams / a row to a block or warp, us:
//   bf16  300 x 7167 (1 row) 6.9 / 6.9, 600 x 4099 (1.3) 6.8 / 7.2, 512 x 7168 (1.7) 5.8 / 5.7, 512 x 7167 8.0 / 12.3, 2048 x 2048 (1.9)
//         5.4 / 6.1, 800 x 7168 (2.6) 8.3 / 9.4, 2000 x 7168 (7) 15.8 / 18.5, 16384 x 1024 (8) 15.9 / 20.9, 4096 x 4096 (9) 17.3 / 19.0,
//         4096 x 4095 (9) 21.0 / 42.4, 4096 x 7168 (13) 24.0 / 31.6, 16384 x 7168 (54) 75 / 108
//   fp32  1003 x 4096 (2.2) 10.3 / 8.9, 1003 x 4099 (2.2) 11.6 / 11.9, 2000 x 2049 (2.2) 12.0 / 10.8, 2000 x 4096 (4.4) 15.5 / 16.8,
//         1024 x 8000 (7) 16.1 / 19.4
// and never for the shortest rows: 16384 x 96 5.3 / 5.0, 16384 x 97 8.4 / 5.8.
constexpr double kLeastRows = 1.25, kLeastRows32 = 3;

// Rows by teams: false where that many rows are too few for it.
template <typename T, typename O, int E>
bool rows_e(const NormArgs& a, bool whole, cudaStream_t st, int num_sms, cudaError_t& e) {
    constexpr int W = 16 / sizeof(T);
    Teams f{};
    f.at = boundary_of(a.x, sizeof(T), a.sx, a.m, W);
    const bool y_vec = same_boundary(f.at, boundary_of(a.y, sizeof(O), a.sy, a.m, W)), w_vec = aligned_to(a.w, 16) && aligned_to(a.b, 16);
    auto kern = whole ? norm_rows_kernel<T, O, E, false> : norm_rows_kernel<T, O, E, true>;
    f.team = runs_team_of(a.n, E, W);
    const int64_t blocks = blocks_of(a.m, num_sms, f.at.stride == 0);
    f.teams = teams_of(a.m, blocks, f.team, E <= 16 ? 896 : 512);
    if (static_cast<double>(a.m) < static_cast<double>(blocks * f.teams) * (sizeof(T) == 4 ? kLeastRows32 : kLeastRows)) return false;
    const int threads = f.team * f.teams, stage = threads * E * static_cast<int>(sizeof(T)) * (E <= 16 ? 2 : 1), weights = f.team * E * 8;
    const int ends = whole ? 0 : f.teams * 128 * (E <= 16 ? 2 : 1);     // of a stage
    f.stages = (kNormRoom - weights) / (stage + ends);
    if (f.stages > 4) f.stages = 4;
    const int smem = f.stages * (stage + ends) + weights;
    e = cudaSuccess;
    if (smem > 46 * 1024)                                  // 48 KB without being asked for
        e = ensure_smem_attr(reinterpret_cast<const void*>(kern), kNormRoom);
    if (e == cudaSuccess) e = launch_after(kern, dim3(static_cast<unsigned>(blocks)), threads, static_cast<size_t>(smem), st, a, f, y_vec, w_vec);
    return true;
}
template <typename T, typename O>
cudaError_t norm_t(const NormArgs& a, cudaStream_t st, int num_sms) {
    constexpr int W = 16 / sizeof(T);
    if (a.n > kNormLongest) {
        const int64_t most = static_cast<int64_t>(num_sms) * 8;
        return launch_after(norm_any_kernel<T, O>, dim3(static_cast<unsigned>(a.m < most ? a.m : most)), kThreads, 0, st, a);
    }
    const bool whole = whole_vectors<T, O>(a);
    cudaError_t e;
    if (a.n <= 256 - W) return norm_e<T, O, 8, true>(a, whole, st);
    if (a.n <= 8192 - W ? rows_e<T, O, 16>(a, whole, st, num_sms, e) : rows_e<T, O, 32>(a, whole, st, num_sms, e)) return e;
    // a row to a warp / to a block, us: 200 x 1000 3.3 / 2.2, 2048 x 1000 5.1 / 4.5, 4000 x 504 3.9 / 4.9, fp32 4000 x 1000 8.0 / 9.3,
    // 8000 x 504 8.4 / 10.2
    if (a.n <= 1024 - W && a.m > 10 * num_sms) return norm_e<T, O, 32, true>(a, whole, st);
    // few elements to a thread where few rows leave a block alone on its SM (1 x 7168 2.8 us, 12.6 by a
    // loop of 256 threads) and where elements go one by one; 4096 x 7168 takes 31.7 with 32 and 67 with 8,
    // 1003 x 4099 fp32 12.8 with 32, 14.9 with 16 and 11.7 with 8
    if (a.n <= 8192 - W && (a.m <= num_sms || a.n <= 1024 - W || !whole)) return norm_e<T, O, 8, false>(a, whole, st);
    return norm_e<T, O, 32, false>(a, whole, st);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st, int num_sms) {
    if (a.x_bf16) return a.y_bf16 ? norm_t<__nv_bfloat16, __nv_bfloat16>(a, st, num_sms) : norm_t<__nv_bfloat16, float>(a, st, num_sms);
    return a.y_bf16 ? norm_t<float, __nv_bfloat16>(a, st, num_sms) : norm_t<float, float>(a, st, num_sms);
}

}  // namespace ql
