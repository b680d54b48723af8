// Layer norm's gradients. With h = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum(g) / n - h sum(g h) / n),  dw = sum_rows dy h,  db = sum_rows dy
//
// Bound by memory: x and dy are read once for all three. Every block goes over rows
// with a fixed set of columns to each thread, which adds up their dw and db in
// registers; a second kernel joins the blocks' sums in a fixed order. 16384 x 7168 bf16:
// 114.7 us, 5 of them the joining; without it 0.95 of a copy's rate.
#include "gemm.cuh"
#include "norm.cuh"
#include "norm_rows.cuh"

namespace ql {
namespace {

constexpr int kThreads = 256;
constexpr int kRowThreads = 512;          // of a block with whole rows
constexpr int kCluster = 8;               // blocks that join their sums themselves
constexpr int64_t kSms = 152;             // for sizes that a caller asks for without a device

// ---------------------------------------------------------------- rows of up to 16368 columns
// The sums of a cluster's blocks, V of the 2 n columns at a time (V divides 2 n).
template <int V>
__device__ __forceinline__ void join_columns(const NormBackArgs& p, int n, int first, int step) {
    for (int c = first * V; c < 2 * n; c += step * V) {
        Pack<float, V> v[kCluster];
#pragma unroll
        for (int i = 0; i < kCluster; ++i) v[i] = load_pack<float, V>(p.part + static_cast<int64_t>(i) * 2 * n + c, p.bnd, 6);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kCluster; ++i) sum += v[i].v[k];
            if (c + k < n) store_one(p.dw + c + k, sum, p.bnd, 7);
            else store_one(p.db + c + k - n, sum, p.bnd, 8);
        }
    }
}

// With d = x - mean, q = dy rstd and g = q w (that is rstd dy w):
//   dx = g - d rstd^2 sum(g d) / n - sum(g) / n,  dw += q d,  db += dy
// Runs past a row's last have x = dy = 0 and are not stored; they add nothing to its sums,
// whose g is 0 there.
//
// The rows to come are on their way into a ring of `stages` rows in shared memory, in
// which each thread copies and reads only what is its own: no thread waits for
// another's copy, and a row's threads for one another only at its two sums.
template <typename T, typename D, int E, bool EDGE>
__global__ void __launch_bounds__(kRowThreads) norm_back_kernel(const NormBackArgs p, const Teams f, bool dy_vec, bool dx_vec, bool w_vec) {
    constexpr int W = 16 / sizeof(T), U = E / W, H = W / 2, XB = W * sizeof(T), DB = W * sizeof(D);
    constexpr bool KEEP = E <= 16;                         // a row's d and g in registers, and the weights
    extern __shared__ __align__(16) uint8_t s_mem[];
    __shared__ float s_sum[2][64];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int id = static_cast<int>(threadIdx.x) / f.team, t = static_cast<int>(threadIdx.x) - id * f.team;
    const uint32_t m = static_cast<uint32_t>(p.m), first = blockIdx.x + gridDim.x * id, step = gridDim.x * f.teams;
    const int all = static_cast<int>(blockDim.x);
    Ends end{0, static_cast<int>(p.n), -1};
    if constexpr (EDGE) end = ends_of<W>(static_cast<int>((f.at.base + static_cast<int64_t>(blockIdx.x) * f.at.stride) % W), static_cast<int>(p.n), t >= f.team - 32);
    const int n = end.tail;                                // of the runs
    const int c0 = end.head + t * W, cu = f.team * W;      // run u starts at column c0 + u * cu

    // [stage][U] runs of x and of dy, then (not KEEP) [E] weights, a thread's side by side;
    // then (EDGE) [stage][2][teams] words of the lanes that have a row's ends
    const int stage = all * U * (XB + DB);
    uint8_t* my_x = s_mem + threadIdx.x * XB;
    uint8_t* my_dy = s_mem + all * U * XB + threadIdx.x * DB;
    ulonglong2* my_w = reinterpret_cast<ulonglong2*>(s_mem + f.stages * stage) + threadIdx.x;     // + i * all
    uint32_t* my_end = reinterpret_cast<uint32_t*>(s_mem + f.stages * stage + (KEEP ? 0 : all * E * 4)) + id * 32 + (t & 31);
    const int end_row = f.teams * 32;                      // words
    for (int s = 0; s < f.stages; ++s)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            *reinterpret_cast<Pack<T, W>*>(my_x + s * stage + u * all * XB) = zero_pack<T, W>();
            *reinterpret_cast<Pack<D, W>*>(my_dy + s * stage + u * all * DB) = zero_pack<D, W>();
        }
    const OneOf<T> x_one(static_cast<const T*>(p.x) + first * p.sx, end.col, static_cast<int>(p.n), p.sx);
    const OneOf<D> dy_one(static_cast<const D*>(p.dy) + first * p.sdy, end.col, static_cast<int>(p.n), p.sdy);
    // (where ends take registers, rows are found by index; else step by step: 16384 x 7168 114.7 us and 120.8)
    const T* x_next = static_cast<const T*>(p.x) + first * p.sx;
    const D* dy_next = static_cast<const D*>(p.dy) + first * p.sdy;
    auto fetch = [&](int at, int stage_no, uint32_t row) { // that row into that stage, which begins at byte `at`
        if (row < m) {
            const T* x = EDGE ? static_cast<const T*>(p.x) + row * p.sx : x_next;
            const D* dy = EDGE ? static_cast<const D*>(p.dy) + row * p.sdy : dy_next;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                fetch_run<W>(my_x + at + u * all * XB, x, c0 + u * cu, n, true, p.bnd, 1);
                fetch_run<W>(my_dy + at + u * all * DB, dy, c0 + u * cu, n, !EDGE || dy_vec, p.bnd, 0);
            }
            if (EDGE && end.col >= 0) {
                x_one.fetch(my_end + 2 * stage_no * end_row, x + end.col, row, m, p.bnd, 1);
                dy_one.fetch(my_end + (2 * stage_no + 1) * end_row, dy + end.col, row, m, p.bnd, 0);
            }
        }
        copy_commit();                                     // a group for every row, also past the last
        x_next += step * p.sx;
        dy_next += step * p.sdy;
    };
    // what the first row needs besides, before the other stages: behind them it waits for the ring to fill
    fetch(0, 0, first);
    F2 w[KEEP ? E / 2 : H];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        F2* v = w + (KEEP ? u * H : 0);
        weight_run<W>(v, p.w, p.w_bf16, 1.0f, c0 + u * cu, n, !EDGE || (w_vec && end.head == 0), p.bnd, 4);
        if constexpr (!KEEP) {
#pragma unroll
            for (int i = 0; i < H / 2; ++i) my_w[(u * (H / 2) + i) * all] = make_ulonglong2(v[2 * i], v[2 * i + 1]);
        }
    }
    float mean = 0.0f, rstd = 0.0f;
    if (first < m) {
        mean = load_one(p.mean + first, p.bnd, 2, 0.0f);
        rstd = load_one(p.rstd + first, p.bnd, 3, 0.0f);
    }
    float end_w = 0.0f, end_dw = 0.0f, end_db = 0.0f;
    if (EDGE && end.col >= 0) end_w = weight_one(p.w, p.w_bf16, 1.0f, end.col, p.bnd, 4);
    for (int s = 1; s < f.stages; ++s) fetch(s * stage, s, first + s * step);
    auto weights = [&](int u, F2 (&v)[H]) {                // of run u
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = w[u * H + i];
        } else {
#pragma unroll
            for (int i = 0; i < H / 2; ++i) {
                const ulonglong2 two = my_w[(u * (H / 2) + i) * all];
                v[2 * i] = two.x;
                v[2 * i + 1] = two.y;
            }
        }
    };
    F2 dw[E / 2], db[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dw[e] = db[e] = 0ull;
    const float inv_n = 1.0f / static_cast<float>(p.n);
    int at = 0, turn = 0, stage_no = 0;
    T* dx_next = static_cast<T*>(p.dx) + first * p.sdx;
    for (uint32_t row = first; row < m; row += step, dx_next += step * p.sdx) {
        float mean2 = 0.0f, rstd2 = 0.0f;                  // the next row's
        if (row + step < m) {
            mean2 = load_one(p.mean + row + step, p.bnd, 2, 0.0f);
            rstd2 = load_one(p.rstd + row + step, p.bnd, 3, 0.0f);
        }
        copy_wait(f.stages);
        const F2 off = f2(-mean, -mean), r2 = f2(rstd, rstd);
        F2 d[KEEP ? E / 2 : 1], g[KEEP ? E / 2 : 1];
        F2 sg = 0ull, sgd = 0ull;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Pack<T, W> x = *reinterpret_cast<const Pack<T, W>*>(my_x + at + u * all * XB);
            const Pack<D, W> dy = *reinterpret_cast<const Pack<D, W>*>(my_dy + at + u * all * DB);
            F2 wu[H];
            weights(u, wu);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int e = u * H + i;
                const F2 v = pair_of<W>(dy, i), de = add2(pair_of<W>(x, i), off), q = mul2(v, r2), ge = mul2(q, wu[i]);
                dw[e] = fma2(q, de, dw[e]);
                db[e] = add2(db[e], v);
                sg = add2(sg, ge);
                sgd = fma2(ge, de, sgd);
                if constexpr (KEEP) {
                    d[e] = de;
                    g[e] = ge;
                }
            }
        }
        float a = sum2(sg), b = sum2(sgd), end_d = 0.0f, end_g = 0.0f;
        if (EDGE && end.col >= 0) {
            const float v = dy_one.value(my_end + (2 * stage_no + 1) * end_row), q = v * rstd;
            end_d = x_one.value(my_end + 2 * stage_no * end_row) - mean;
            end_g = q * end_w;
            end_dw = fmaf(q, end_d, end_dw);
            end_db += v;
            a += end_g;
            b = fmaf(end_g, end_d, b);
        }
        if constexpr (KEEP) fetch(at, stage_no, row + f.stages * step);
        sum_over_team(a, b, s_sum[turn], f.team, id);
        turn ^= 1;
        const float k1 = -a * inv_n, k2 = -rstd * rstd * (b * inv_n);
        const F2 k1k1 = f2(k1, k1), k2k2 = f2(k2, k2);
        asm volatile("" ::: "memory");                     // what is not kept is read again
        T* dx = EDGE ? static_cast<T*>(p.dx) + row * p.sdx : dx_next;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * cu;
            if (c >= n) continue;
            F2 o[H];
            if constexpr (KEEP) {
#pragma unroll
                for (int i = 0; i < H; ++i) o[i] = add2(g[u * H + i], fma2(d[u * H + i], k2k2, k1k1));
            } else {
                const Pack<T, W> x = *reinterpret_cast<const Pack<T, W>*>(my_x + at + u * all * XB);
                const Pack<D, W> dy = *reinterpret_cast<const Pack<D, W>*>(my_dy + at + u * all * DB);
                F2 wu[H];
                weights(u, wu);
#pragma unroll
                for (int i = 0; i < H; ++i)
                    o[i] = fma2(mul2(pair_of<W>(dy, i), r2), wu[i], fma2(add2(pair_of<W>(x, i), off), k2k2, k1k1));
            }
            store_run<W>(dx, o, c, n, !EDGE || dx_vec, p.bnd, 5);
        }
        if (EDGE && end.col >= 0) store_one(dx + end.col, from_f32<T>(end_g + fmaf(end_d, k2, k1)), p.bnd, 5);
        if constexpr (!KEEP) fetch(at, stage_no, row + f.stages * step);
        at += stage;
        if (++stage_no == f.stages) at = stage_no = 0;
        mean = mean2;
        rstd = rstd2;
    }
    if (p.dw == nullptr) return;
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.n;
    if ((EDGE && W > 4) || f.teams > 1) {
        // the block's teams in the rows' room: [team][E / 2][threads] pairs of dw and db, [team][32] of the ends'. (From here stores
        // are whole lines: 512 x 7167 13.5 us, 20.2 by each thread's runs, whose elements go one by one; but
        // 1003 x 4099 fp32, with runs of 4, 18.3 and 17.6.)
        ulonglong2* sums = reinterpret_cast<ulonglong2*>(s_mem);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E / 2; ++e) sums[(id * (E / 2) + e) * f.team + t] = make_ulonglong2(dw[e], db[e]);
        F2* end_sums = reinterpret_cast<F2*>(sums + all * (E / 2));
        if (EDGE && end.col >= 0) end_sums[id * 32 + (t & 31)] = f2(end_dw, end_db);
        __syncthreads();
        if (EDGE && id == 0 && end.col >= 0) {
            F2 v = end_sums[t & 31];
            for (int k = 1; k < f.teams; ++k) v = add2(v, end_sums[k * 32 + (t & 31)]);
            float a, b;
            unpack(v, a, b);
            store_one(part + end.col, a, p.bnd, 6);
            store_one(part + p.n + end.col, b, p.bnd, 6);
        }
        const int pairs = E / 2 * f.team;
        for (int j = threadIdx.x; j < pairs; j += all) {   // columns head + 2 j and the next, those of run j / H
            const int run = j / H, u = run / f.team, c = end.head + 2 * j, i = (u * H + j % H) * f.team + run - u * f.team;
            ulonglong2 v = sums[i];
            for (int k = 1; k < f.teams; ++k) {
                const ulonglong2 o = sums[k * pairs + i];
                v.x = add2(v.x, o.x);
                v.y = add2(v.y, o.y);
            }
            float a[4];
            unpack(v.x, a[0], a[1]);
            unpack(v.y, a[2], a[3]);
            if (c < n) {                                   // and c + 1 with it
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    store_one(part + c + k, a[k], p.bnd, 6);
                    store_one(part + p.n + c + k, a[2 + k], p.bnd, 6);
                }
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * cu;
            if (c >= n) continue;
            store_run<W>(part, dw + u * H, c, n, !EDGE, p.bnd, 6);
            store_run<W>(part + p.n, db + u * H, c, n, !EDGE, p.bnd, 6);
        }
        if (EDGE && end.col >= 0) {
            store_one(part + end.col, end_dw, p.bnd, 6);
            store_one(part + p.n + end.col, end_db, p.bnd, 6);
        }
    }
    if (f.cluster) {                                       // few rows: joined at once, by all blocks
        cluster_sync_all();
        const int cols = static_cast<int>(p.n);
        if (cols % 2 == 0) join_columns<4>(p, cols, static_cast<int>(blockIdx.x) * all + static_cast<int>(threadIdx.x), kCluster * all);
        else join_columns<1>(p, cols, static_cast<int>(blockIdx.x) * all + static_cast<int>(threadIdx.x), kCluster * all);
    }
}

// ---------------------------------------------------------------- any length
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
        LongSum s1, s2;
        for (int64_t i0 = threadIdx.x; i0 < p.n; i0 += kLongRun * kThreads) {
            const int count = long_run(i0, p.n, kThreads);
            float r1 = 0.0f, r2 = 0.0f;
#pragma unroll 8
            for (int j = 0; j < count; ++j) {
                const int64_t i = i0 + j * kThreads;
                float w[1];
                load_weights<1>(w, p.w, p.w_bf16, i, 1.0f, p.bnd, 4);
                const float g = __fmul_rn(to_f32(load_one(dy + i, p.bnd, 0, from_f32<D>(0.0f))), w[0]);
                r1 += g;
                r2 = fmaf(g, (to_f32(load_one(x + i, p.bnd, 1, from_f32<T>(0.0f))) - mean) * rstd, r2);
            }
            s1.add(r1);
            s2.add(r2);
        }
        float c[2] = {s1.value(), s2.value()};
        __syncthreads();
        sum_over_row<2, false>(c, s_sum);
        const float c1 = c[0] / n, c2 = c[1] / n;
        for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
            float w[1];
            load_weights<1>(w, p.w, p.w_bf16, i, 1.0f, p.bnd, 4);
            const float g = __fmul_rn(to_f32(load_one(dy + i, p.bnd, 0, from_f32<D>(0.0f))), w[0]);
            const float h = (to_f32(load_one(x + i, p.bnd, 1, from_f32<T>(0.0f))) - mean) * rstd;
            store_one(dx + i, from_f32<T>(rstd * fmaf(-h, c2, g - c1)), p.bnd, 5);
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
    LongSum dw, db;
    for (int64_t first = r0; first < r1; first += kLongRun) {
        const int count = long_run(first, r1, 1);
        float run_w = 0.0f, run_b = 0.0f;
#pragma unroll 8
        for (int j = 0; j < count; ++j) {
            const int64_t r = first + j;
            const float dy = to_f32(load_one(static_cast<const D*>(p.dy) + r * p.sdy + col, p.bnd, 0, from_f32<D>(0.0f)));
            const float x = to_f32(load_one(static_cast<const T*>(p.x) + r * p.sx + col, p.bnd, 1, from_f32<T>(0.0f)));
            run_w = fmaf(dy, (x - load_one(p.mean + r, p.bnd, 2, 0.0f)) * load_one(p.rstd + r, p.bnd, 3, 0.0f), run_w);
            run_b += dy;
        }
        dw.add(run_w);
        db.add(run_b);
    }
    float* part = p.part + static_cast<int64_t>(blockIdx.y) * 2 * p.n;
    store_one(part + col, dw.value(), p.bnd, 6);
    store_one(part + p.n + col, db.value(), p.bnd, 6);
}

// dw and db: the parts' sums, 32 columns by 16 shares of the parts per block, in a
// fixed order. At most 152 parts (10 of long rows): all of a thread's loads at once.
__global__ void __launch_bounds__(512) norm_dw_join_kernel(const NormBackArgs p, int parts) {
    __shared__ float s[16][33];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + tx;      // of 2 n
    float v[10];
#pragma unroll
    for (int i = 0; i < 10; ++i) v[i] = col < 2 * p.n && ty + 16 * i < parts ? load_one(p.part + (ty + 16 * i) * 2 * p.n + col, p.bnd, 6, 0.0f) : 0.0f;
#pragma unroll
    for (int i = 1; i < 10; ++i) v[0] += v[i];
    s[ty][tx] = v[0];
    __syncthreads();
    if (ty == 0 && col < 2 * p.n) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += s[i][tx];
        if (col < p.n) store_one(p.dw + col, sum, p.bnd, 7);
        else store_one(p.db + col - p.n, sum, p.bnd, 8);
    }
}

unsigned grid_of(int64_t n, int64_t most) { return static_cast<unsigned>(n < 1 ? 1 : (n < most ? n : most)); }

// Parts of the rows for the column sums of long rows: enough blocks for every SM to have four.
int64_t any_parts(int64_t m, int64_t n) {
    const int64_t cols = (n + kThreads - 1) / kThreads;
    int64_t parts = (kSms * 4 + cols - 1) / cols;
    if (parts > (m + 15) / 16) parts = (m + 15) / 16;
    return parts < 1 ? 1 : parts;
}

cudaError_t join(const NormBackArgs& a, int64_t parts, cudaStream_t st) {
    if (a.dw == nullptr) return cudaSuccess;
    return launch_after(norm_dw_join_kernel, dim3(static_cast<unsigned>((2 * a.n + 31) / 32)), 512, 0, st, a, static_cast<int>(parts));
}

// Most parts of the rows: the blocks of the kernel above, a multiple of 8 where rows
// start differently.
int64_t most_parts(int64_t m) {
    const int64_t least = m < kCluster ? kCluster : m;
    return least < kSms ? least : kSms;
}

template <typename T, typename D, int E>
cudaError_t back_e(const NormBackArgs& a, cudaStream_t st, int num_sms) {
    constexpr int W = 16 / sizeof(T);
    Teams f{};
    f.at = boundary_of(a.x, sizeof(T), a.sx, a.m, W);
    const Boundary dy_at = boundary_of(a.dy, sizeof(D), a.sdy, a.m, W);
    const bool dy_vec = same_boundary(f.at, dy_at),
               dx_vec = same_boundary(f.at, boundary_of(a.dx, sizeof(T), a.sdx, a.m, W)), w_vec = aligned_to(a.w, 16);
    const bool edge = f.at.base != 0 || f.at.stride != 0 || a.n % W != 0 || !dy_vec || !dx_vec || !w_vec;
    auto kern = edge ? norm_back_kernel<T, D, E, true> : norm_back_kernel<T, D, E, false>;
    f.team = runs_team_of(a.n, E, W);
    // With up to two rows to a team of eight blocks, these join their sums as a cluster: one launch less,
    // which takes the host longer than the rows' spread over the SMs saves (one row: 9.3 us of host time
    // with a second kernel, 5.8 without).
    f.cluster = a.dw != nullptr && a.m <= 2 * kCluster * (kRowThreads / f.team);
    const int64_t blocks = f.cluster ? kCluster : blocks_of(a.m, num_sms < kSms ? num_sms : kSms, f.at.stride == 0 && dy_at.stride == 0);
    f.teams = teams_of(a.m, blocks, f.team, kRowThreads);
    const int threads = f.team * f.teams, stage = threads * E * static_cast<int>(sizeof(T) + sizeof(D)), weights = E <= 16 ? 0 : threads * E * 4;
    const int ends = edge ? f.teams * 256 : 0;             // of a stage
    f.stages = (kNormRoom - weights) / (stage + ends);
    if (f.stages > 4) f.stages = 4;
    const int sums = a.dw != nullptr && ((edge && W > 4) || f.teams > 1) ? threads * E * 8 + f.teams * 256 : 0;
    const int rows = f.stages * (stage + ends) + weights, smem = sums > rows ? sums : rows;
    if (smem > 47 * 1024)                                  // 48 KB without being asked for
        if (cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), kNormRoom); e != cudaSuccess) return e;
    if (cudaError_t e = launch_cluster_after(kern, dim3(static_cast<unsigned>(blocks)), threads, f.cluster ? kCluster : 1, static_cast<size_t>(smem), st, a, f,
                                             dy_vec, dx_vec, w_vec);
        e != cudaSuccess || f.cluster)
        return e;
    return join(a, blocks, st);
}

// Elements per thread of a team.
template <typename T, typename D>
cudaError_t back_rows(const NormBackArgs& a, cudaStream_t st, int num_sms) {
    constexpr int W = 16 / sizeof(T);
    if (a.n <= 256 - W) return back_e<T, D, 8>(a, st, num_sms);
    if (a.n <= 8192 - W) return back_e<T, D, 16>(a, st, num_sms);
    return back_e<T, D, 32>(a, st, num_sms);
}

template <typename T, typename D>
cudaError_t back_t(const NormBackArgs& a, cudaStream_t st, int num_sms) {
    if (a.n > kNormLongest) {
        if (cudaError_t e = launch_after(norm_dx_any_kernel<T, D>, dim3(grid_of(a.m, static_cast<int64_t>(num_sms) * 8)), kThreads, 0, st, a);
            e != cudaSuccess || a.dw == nullptr)
            return e;
        const int64_t parts = any_parts(a.m, a.n), rows = (a.m + parts - 1) / parts;
        if (cudaError_t e = launch_after(norm_dw_any_kernel<T, D>, dim3(static_cast<unsigned>((a.n + kThreads - 1) / kThreads), static_cast<unsigned>(parts)),
                                         kThreads, 0, st, a, rows);
            e != cudaSuccess)
            return e;
        return join(a, parts, st);
    }
    return back_rows<T, D>(a, st, num_sms);
}

}  // namespace

size_t norm_back_workspace(int64_t m, int64_t n) {
    return static_cast<size_t>(n > kNormLongest ? any_parts(m, n) : most_parts(m)) * 2 * static_cast<size_t>(n) * sizeof(float);
}

cudaError_t launch_norm_back(const NormBackArgs& a, cudaStream_t st, int num_sms) {
    if (a.x_bf16) return a.dy_bf16 ? back_t<__nv_bfloat16, __nv_bfloat16>(a, st, num_sms) : back_t<__nv_bfloat16, float>(a, st, num_sms);
    return a.dy_bf16 ? back_t<float, __nv_bfloat16>(a, st, num_sms) : back_t<float, float>(a, st, num_sms);
}

}  // namespace ql
