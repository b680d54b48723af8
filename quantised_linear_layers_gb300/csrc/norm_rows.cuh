// What the layer norm kernels share: packed fp32 arithmetic, sums over the threads of a
// row, and rows that start anywhere.
//
// A row is a team's: `team` threads of whole warps. A thread has U runs of W elements, on
// boundaries of W elements and inside the row: run u of thread t those from column
// head + (u * team + t) * W on. What a row has before the first run and behind the last,
// up to W - 1 elements each, is the team's last warp's, an element to a lane (Ends).
#pragma once

#include "rows.cuh"

namespace ql {

constexpr int kNormRoom = 224 * 1024;     // shared memory of a block
constexpr int64_t kNormLongest = 16384 - 16;       // columns of a row in a team's registers
// Terms that a thread adds up one after the other where a sum may have any number of them; the
// runs' sums are added up with what each addition rounds off (Neumaier), so that the error does
// not grow with their number.
constexpr int kLongRun = 64;
struct LongSum {
    float all = 0.0f, off = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float t = all + v;
        off += fabsf(all) >= fabsf(v) ? (all - t) + v : (v - t) + all;
        all = t;
    }
    __device__ __forceinline__ float value() const { return fabsf(all) < INFINITY ? all + off : all; }
};
// Terms of the run that begins at first and goes on by `step`, up to end.
__device__ __forceinline__ int long_run(int64_t first, int64_t end, int step) {
    const int64_t count = (end - first + step - 1) / step;
    return count < kLongRun ? static_cast<int>(count) : kLongRun;
}

// ---------------------------------------------------------------- pairs of fp32
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(F2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(F2 v) {
    float a, b;
    unpack(v, a, b);
    return a + b;
}
// Elements 2i, 2i + 1 of a pack.
template <int W>
__device__ __forceinline__ F2 pair_of(const Pack<__nv_bfloat16, W>& p, int i) {
    const uint32_t u = reinterpret_cast<const uint32_t*>(&p)[i];
    return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <int W>
__device__ __forceinline__ F2 pair_of(const Pack<float, W>& p, int i) {
    return f2(p.v[2 * i], p.v[2 * i + 1]);
}
template <int W>
__device__ __forceinline__ void set_pair(Pack<__nv_bfloat16, W>& p, int i, F2 v) {
    float a, b;
    unpack(v, a, b);
    reinterpret_cast<__nv_bfloat162*>(&p)[i] = __floats2bfloat162_rn(a, b);
}
template <int W>
__device__ __forceinline__ void set_pair(Pack<float, W>& p, int i, F2 v) {
    unpack(v, p.v[2 * i], p.v[2 * i + 1]);
}

// ---------------------------------------------------------------- sums
// Two sums over a warp, in half the exchanges: lanes 0 to 15 get a's, the others b's.
__device__ __forceinline__ float sums_over_warp(float a, float b) {
    const bool high = (threadIdx.x & 16) != 0;
    float v = high ? b : a;
    v += __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Two sums over a team of at most 16 warps, the id-th of its block; every thread gets
// both. s: 64 floats of shared memory for a block's teams, free again after the team's
// next call with another s.
__device__ __forceinline__ void sum_over_team(float& a, float& b, float* s, int team, int id) {
    const int lane = threadIdx.x & 31;
    float v = sums_over_warp(a, b);
    if (team > 32) {
        const int warps = team >> 5;
        if ((lane & 15) == 0) s[(lane >> 4) * 32 + (threadIdx.x >> 5)] = v;
        named_bar_sync(static_cast<uint32_t>(id + 1), static_cast<uint32_t>(team));
        v = (lane & 15) < warps ? s[(lane >> 4) * 32 + id * warps + (lane & 15)] : 0.0f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    a = __shfl_sync(0xffffffffu, v, 0);
    b = __shfl_sync(0xffffffffu, v, 16);
}

// Four sums over such a team, eight lanes to each. s: 128 floats.
__device__ __forceinline__ void sum4_over_team(float (&a)[4], float* s, int team, int id) {
    const int lane = threadIdx.x & 31;
    const bool h16 = (lane & 16) != 0, h8 = (lane & 8) != 0;
    float v = h16 ? a[2] : a[0], u = h16 ? a[3] : a[1];
    v += __shfl_xor_sync(0xffffffffu, h16 ? a[0] : a[2], 16);
    u += __shfl_xor_sync(0xffffffffu, h16 ? a[1] : a[3], 16);
    const float other = __shfl_xor_sync(0xffffffffu, h8 ? v : u, 8);
    v = (h8 ? u : v) + other;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (team > 32) {
        const int warps = team >> 5;
        if ((lane & 7) == 0) s[(lane >> 3) * 32 + (threadIdx.x >> 5)] = v;
        named_bar_sync(static_cast<uint32_t>(id + 1), static_cast<uint32_t>(team));
        const float* of = s + (lane >> 3) * 32 + id * warps + (lane & 7);
        v = (lane & 7) < warps ? of[0] : 0.0f;
        if ((lane & 7) + 8 < warps) v += of[8];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __shfl_sync(0xffffffffu, v, 8 * i);
}

// ---------------------------------------------------------------- runs
// W elements from column c of a row on as pairs, zeros from column n on. vec: on a boundary.
template <int W, typename T, typename B>
__device__ __forceinline__ void load_run(F2* v, const T* row, int c, int n, bool vec, const B& bnd, int span) {
    Pack<T, W> p = zero_pack<T, W>();
    if (vec) {
        if (c < n) p = load_pack<T, W>(row + c, bnd, span);
    } else if (c < n) {
#pragma unroll
        for (int i = 0; i < W; ++i) p.v[i] = load_one(row + c + i, bnd, span, p.v[i]);
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) v[i] = pair_of<W>(p, i);
}
// And back, where c < n.
template <int W, typename T, typename B>
__device__ __forceinline__ void store_run(T* row, const F2* v, int c, int n, bool vec, const B& bnd, int span) {
    Pack<T, W> p;
#pragma unroll
    for (int i = 0; i < W / 2; ++i) set_pair<W>(p, i, v[i]);
    if (vec) {
        if (c < n) store_pack<T, W>(row + c, p, bnd, span);
    } else if (c < n) {
#pragma unroll
        for (int i = 0; i < W; ++i) store_one(row + c + i, p.v[i], bnd, span);
    }
}
// A run of weights of bf16 or fp32 that may be missing (`other`), and one of them.
template <int W, typename B>
__device__ __forceinline__ void weight_run(F2* v, const void* p, bool bf16, float other, int c, int n, bool vec, const B& bnd, int span) {
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) v[i] = f2(other, other);
    } else if (bf16) {
        load_run<W>(v, static_cast<const __nv_bfloat16*>(p), c, n, vec, bnd, span);
    } else {
        load_run<W>(v, static_cast<const float*>(p), c, n, vec, bnd, span);
    }
}
template <typename B>
__device__ __forceinline__ float weight_one(const void* p, bool bf16, float other, int c, const B& bnd, int span) {
    float w[1];
    load_weights<1>(w, p, bf16, c, other, bnd, span);
    return w[0];
}

// A row of n >= W columns whose first is `shift` past a boundary: whole runs of the columns
// [head, tail), and the lane's column of the others, or -1.
struct Ends {
    int head, tail, col;
};
template <int W>
__device__ __forceinline__ Ends ends_of(int shift, int n, bool last_warp) {
    Ends e;
    e.head = shift == 0 ? 0 : W - shift;
    e.tail = e.head + (n - e.head) / W * W;
    const int lane = static_cast<int>(threadIdx.x & 31), c = lane < W ? e.head - W + lane : e.tail + lane - W;
    e.col = last_warp && lane < 2 * W && c >= 0 && c < n && (c < e.head || c >= e.tail) ? c : -1;
    return e;
}

// Where a tensor's rows start past boundaries of w elements: row r at (base + r * stride) % w.
struct Boundary {
    int base, stride;
};
inline Boundary boundary_of(const void* p, int64_t es, int64_t stride, int64_t m, int w) {
    return Boundary{static_cast<int>(reinterpret_cast<uintptr_t>(p) / static_cast<uintptr_t>(es) % static_cast<uintptr_t>(w)),
                    m > 1 ? static_cast<int>(((stride % w) + w) % w) : 0};
}
inline bool same_boundary(const Boundary& a, const Boundary& b) { return a.base == b.base && a.stride == b.stride; }
// Threads of a team for rows of n columns, E elements each.
inline int team_of(int64_t n, int e) { return static_cast<int>((n + 32 * e - 1) / (32 * e)) * 32; }

// ---------------------------------------------------------------- rows through shared memory
// A run into a thread's own place in shared memory, where c < n.
template <int W, typename T, typename B>
__device__ __forceinline__ void fetch_run(void* place, const T* row, int c, int n, bool vec, const B& bnd, int span) {
    T* to = static_cast<T*>(place);
    if (vec) {
        if (c < n && QL_IN(bnd, span, row + c, W * sizeof(T))) copy_async<W * sizeof(T)>(to, row + c);
    } else if (c < n) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (QL_IN(bnd, span, row + c + i, sizeof(T))) {
                if constexpr (sizeof(T) == 4) copy_async<4>(to + i, row + c + i);
                else to[i] = row[c + i];
            }
    }
}
// Column c of a tensor's rows by a lane with a word of its own, where it comes in the word of
// memory that it is in: with a neighbour of bf16, which may be the row before's or behind's
// (or what lies between them), but not past the tensor. first: a row of the lane's, n its
// columns, stride that between rows; all the lane's rows start alike.
template <typename T>
struct OneOf {
    bool high, before, behind;                             // the second half; with a neighbour of another row, or (both) none
    __device__ __forceinline__ OneOf(const T* first, int c, int n, int64_t stride) {
        high = sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(first + c) & 2) != 0;
        before = sizeof(T) == 2 && high && c == 0;
        behind = sizeof(T) == 2 && !high && c == n - 1;
        if ((before || behind) && stride <= 0) before = behind = true;
    }
    template <typename B>
    __device__ __forceinline__ void fetch(uint32_t* word, const T* p, uint32_t row, uint32_t m, const B& bnd, int span) const {
        if constexpr (sizeof(T) == 4) {
            if (QL_IN(bnd, span, p, 4)) copy_async<4>(word, p);
        } else if ((before && row == 0) || (behind && row == m - 1) || (before && behind)) {
            reinterpret_cast<T*>(word)[high] = load_one(p, bnd, span, from_f32<T>(0.0f));
        } else if (QL_IN(bnd, span, p - high, 4)) {
            copy_async<4>(word, p - high);
        }
    }
    __device__ __forceinline__ float value(const uint32_t* word) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(*word);
        else return __uint_as_float(high ? *word & 0xffff0000u : *word << 16);
    }
};

// How the rows go to the teams of warps of the blocks. Every row of a block has the same
// shift (row = block + blocks * (team + teams * i), blocks a multiple of 8 unless all
// rows start alike, x's and dy's), so a thread's columns stay its own.
struct Teams {
    int team, teams, stages;
    Boundary at;
    bool cluster;              // the blocks are one cluster
};
// And for rows in runs of w with Ends.
inline int runs_team_of(int64_t n, int e, int w) { return n < w ? 32 : team_of(n / w * w, e); }
// Blocks of a launch over m rows (alike: all start alike), `most` at most (a multiple of
// 8), and their teams of `team` threads, `threads` at most in all: rows first to blocks,
// then to teams.
inline int64_t blocks_of(int64_t m, int64_t most, bool alike) {
    if (alike) return m < most ? m : most;
    const int64_t blocks = (m < 8 ? 8 : m) / 8 * 8;
    return blocks < most ? blocks : most / 8 * 8;
}
inline int teams_of(int64_t m, int64_t blocks, int team, int threads) {
    const int64_t rows = (m + blocks - 1) / blocks;
    return static_cast<int>(rows < threads / team ? rows : threads / team);
}

}  // namespace ql
