// The exchange of rows with the experts: the order of the slots (token, j) by
// expert (a stable counting sort), rows to their places, and the weighted sums
// back, with the gradients of both.
#include "gemm.cuh"
#include "route.cuh"
#include "rows.cuh"

namespace ql {
namespace {

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanRoom = kRouteMaxExperts + 2;            // and a place for no expert

// The expert of a slot; `experts` for none.
__device__ __forceinline__ int expert_of(const PlanArgs& p, int64_t slot) {
    const int e = load_one(p.chosen + slot, p.bnd, 0, -1);
    if (e >= 0 && e < p.experts) return e;
    if (e != -1) atomicOr(p.dev_status, kDevErrBadIndex);
    return p.experts;
}

// The lanes of a warp with this lane's expert, bit by bit. (A match of whole values goes over
// the distinct ones: 1.9 us for two of 32 over 256 experts.)
__device__ __forceinline__ uint32_t same_expert(int e, int bits) {
    uint32_t same = 0xffffffffu;
    for (int i = 0; i < bits; ++i) {
        const bool set = (e >> i & 1) != 0;
        const uint32_t with = __ballot_sync(0xffffffffu, set);
        same &= set ? with : ~with;
    }
    return same;
}

// counts[chunk][expert]: how many slots of the chunk name the expert.
__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(const PlanArgs p) {
    __shared__ int s_count[kPlanRoom];
    pdl_launch_dependents();
    pdl_wait_prior();
    for (int e = threadIdx.x; e <= p.experts; e += kPlanThreads) s_count[e] = 0;
    __syncthreads();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.chunk;
    const int64_t last = first + p.chunk < p.slots ? first + p.chunk : p.slots;
    for (int64_t i = first + threadIdx.x; i < last; i += kPlanThreads) atomicAdd(&s_count[expert_of(p, i)], 1);
    __syncthreads();
    int32_t* out = p.counts + static_cast<int64_t>(blockIdx.x) * p.experts;
    for (int e = threadIdx.x; e < p.experts; e += kPlanThreads) store_one(out + e, s_count[e], p.bnd, 3);
}

// Places of a chunk's slots: an expert's first row, its slots in the chunks before,
// in the warps before and in the warp before the slot. The warps have equal runs of
// the chunk's slots, so the order among an expert's slots is the slots' own. Every
// chunk adds up the counts of all of them: no chunk waits for another.
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanArgs p) {
    __shared__ __align__(16) uint16_t s_warp[kPlanWarps][kPlanRoom];   // slots of a warp, then of the warps before
    __shared__ int s_total[kRouteMaxExperts], s_before[kRouteMaxExperts];
    __shared__ int s_sum[kPlanWarps];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = lane; i < (p.experts + 2) / 2; i += 32) reinterpret_cast<uint32_t*>(s_warp[warp])[i] = 0;
    for (int e = threadIdx.x; e < kRouteMaxExperts; e += kPlanThreads) s_total[e] = s_before[e] = 0;
    __syncthreads();
    const int64_t run = p.chunk / kPlanWarps;              // a multiple of 32
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.chunk + warp * run;
    const int64_t last = first + run < p.slots ? first + run : p.slots;
    const uint32_t below = (1u << lane) - 1u;
    const int bits = 32 - __clz(p.experts);                // of 0 .. experts
    int e = p.experts;                                     // of the lane's last slot
    uint32_t same = 0u;
    for (int64_t i = first; i < last; i += 32) {
        e = i + lane < last ? expert_of(p, i + lane) : p.experts;
        same = same_expert(e, bits);
        if ((same & below) == 0) s_warp[warp][e] = static_cast<uint16_t>(s_warp[warp][e] + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    for (int of = threadIdx.x; of < p.experts; of += kPlanThreads) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < kPlanWarps; ++w) {
            const int c = s_warp[w][of];
            s_warp[w][of] = static_cast<uint16_t>(sum);
            sum += c;
        }
        if (p.counts == nullptr) s_total[of] = sum;         // one chunk
    }
    if (p.counts != nullptr) {
        int room = 32;                                     // threads side by side over the experts
        while (room < p.experts) room *= 2;
        const int of = threadIdx.x & (room - 1), share = threadIdx.x / room, shares = kPlanThreads / room;
        if (of < p.experts) {
            int total = 0, before = 0;
#pragma unroll 8
            for (int c = share; c < static_cast<int>(gridDim.x); c += shares) {
                const int v = load_one(p.counts + static_cast<int64_t>(c) * p.experts + of, p.bnd, 3, 0);
                total += v;
                if (c < static_cast<int>(blockIdx.x)) before += v;
            }
            atomicAdd(&s_total[of], total);
            atomicAdd(&s_before[of], before);
        }
    }
    __syncthreads();
    // experts' first rows: a sum over the experts before
    const int mine = threadIdx.x < p.experts ? s_total[threadIdx.x] : 0;
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    int ahead = lane < warp ? s_sum[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    const int start = ahead + sum - mine;
    if (threadIdx.x < p.experts) s_before[threadIdx.x] += start;
    if (blockIdx.x == 0 && threadIdx.x <= p.experts) store_one(p.offsets + threadIdx.x, start, p.bnd, 1);
    __syncthreads();
    for (int64_t i = first; i < last; i += 32) {
        if (run > 32) {                                    // else they are those of the first time
            e = i + lane < last ? expert_of(p, i + lane) : p.experts;
            same = same_expert(e, bits);
        }
        const int at = s_warp[warp][e];
        __syncwarp();
        if ((same & below) == 0) s_warp[warp][e] = static_cast<uint16_t>(at + __popc(same));
        __syncwarp();
        if (i + lane < last) store_one(p.rows + i + lane, e < p.experts ? s_before[e] + at + __popc(same & below) : -1, p.bnd, 2);
    }
}

// ---------------------------------------------------------------- rows there and back
// A token is a team's: a power of two of threads, up to a block. A thread has runs of W
// columns: whole 16-byte vectors, or (SPREAD) elements a team apart, which take any
// boundary and any length and are whole lines all the same. What hides the memory's
// latency is threads: each has few loads, all at once, and is soon gone.
constexpr int kThreads = 128;
constexpr int kSlots = 8;                                  // of a token at a time

// Columns of run u of a team's thread.
template <int W, bool SPREAD>
__device__ __forceinline__ int64_t column(int u, int i, int lane, int team) {
    return SPREAD ? (static_cast<int64_t>(u) * W + i) * team + lane : (static_cast<int64_t>(u) * team + lane) * W + i;
}
template <typename T, int W, bool SPREAD, typename B>
__device__ __forceinline__ Pack<T, W> load_columns(const T* row, int u, int lane, int team, int64_t n, const B& b, int span) {
    if constexpr (!SPREAD) {
        return load_pack<T, W>(row + column<W, false>(u, 0, lane, team), b, span);
    } else {
        Pack<T, W> v = zero_pack<T, W>();
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int64_t c = column<W, true>(u, i, lane, team);
            if (c < n) v.v[i] = load_one(row + c, b, span, v.v[i]);
        }
        return v;
    }
}
template <typename T, int W, bool SPREAD, typename B>
__device__ __forceinline__ void store_columns(T* row, const Pack<T, W>& v, int u, int lane, int team, int64_t n, const B& b, int span) {
    if constexpr (!SPREAD) {
        store_pack<T, W>(row + column<W, false>(u, 0, lane, team), v, b, span);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int64_t c = column<W, true>(u, i, lane, team);
            if (c < n) store_one(row + c, v.v[i], b, span);
        }
    }
}

// The rows of K slots of a token from slot j0 on: -1 for none, and for what lies outside
// [0, all).
template <int K, typename B>
__device__ __forceinline__ void rows_of(int32_t (&r)[K], const int32_t* rows, int64_t t, int j0, int k, int64_t all, const B& b, int span) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
        r[j] = j0 + j < k ? load_one(rows + t * k + j0 + j, b, span, -1) : -1;
        if (r[j] >= all) r[j] = -1;
    }
}
template <int K, typename B>
__device__ __forceinline__ void weights_of(float (&w)[K], const float* weights, int64_t t, int j0, int k, const B& b, int span) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j] = weights == nullptr ? 1.0f : (j0 + j < k ? load_one(weights + t * k + j0 + j, b, span, 0.0f) : 0.0f);
}

// A row is read once and written k times (4096 x 8 of 7168 bf16: 80 us, 0.97 of a copy's
// rate). Row t k + j of xs is token t's to clear if no slot has it.
template <typename T, int W, bool SPREAD>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchArgs p, int team, unsigned pieces) {
    constexpr int U = 4, K = 4;
    pdl_launch_dependents();
    pdl_wait_prior();
    const unsigned group = blockIdx.x / pieces;
    const int lane = threadIdx.x & (team - 1), u0 = static_cast<int>(blockIdx.x - group * pieces) * U;
    const int64_t t = static_cast<int64_t>(group) * (kThreads / team) + threadIdx.x / team, all = p.m * p.k;
    if (t >= p.m) return;
    const T* x = static_cast<const T*>(p.x) + t * p.sx;
    Pack<T, W> v[U];
    int32_t r[K];
    rows_of<K>(r, p.rows, t, 0, p.k, all, p.bnd, 1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v[u] = zero_pack<T, W>();
        if (column<W, SPREAD>(u0 + u, 0, lane, team) < p.n) v[u] = load_columns<T, W, SPREAD>(x, u0 + u, lane, team, p.n, p.bnd, 0);
    }
    const int64_t used = load_one(p.offsets + p.experts, p.bnd, 2, 0);
    for (int j0 = 0; j0 < p.k; j0 += K) {
        int32_t next[K];
        if (j0 + K < p.k) rows_of<K>(next, p.rows, t, j0 + K, p.k, all, p.bnd, 1);
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (r[j] >= 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (column<W, SPREAD>(u0 + u, 0, lane, team) < p.n)
                        store_columns<T, W, SPREAD>(static_cast<T*>(p.xs) + r[j] * p.sxs, v[u], u0 + u, lane, team, p.n, p.bnd, 3);
#pragma unroll
        for (int j = 0; j < K; ++j) r[j] = next[j];
    }
    if (t * p.k + p.k > used)
        for (int j = 0; j < p.k; ++j)
            if (t * p.k + j >= used)
                for (int u = u0; u < u0 + U; ++u)
                    if (column<W, SPREAD>(u, 0, lane, team) < p.n)
                        store_columns<T, W, SPREAD>(static_cast<T*>(p.xs) + (t * p.k + j) * p.sxs, zero_pack<T, W>(), u, lane, team, p.n, p.bnd, 3);
}

// Runs of a thread: enough loads for few slots, sums that registers hold.
__host__ __device__ constexpr int combine_runs(int k) { return k == 1 ? 4 : (k == 2 ? 2 : 1); }

// A thread adds up its columns' k terms in fp32 in the order of j: U runs of K slots are on
// their way at a time.
template <typename T, int W, int K, bool SPREAD>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs p, int team, unsigned pieces) {
    constexpr int U = combine_runs(K);
    pdl_launch_dependents();
    pdl_wait_prior();
    const unsigned group = blockIdx.x / pieces;
    const int lane = threadIdx.x & (team - 1), u0 = static_cast<int>(blockIdx.x - group * pieces) * U;
    const int64_t t = static_cast<int64_t>(group) * (kThreads / team) + threadIdx.x / team, all = p.m * p.k;
    if (t >= p.m) return;
    float sum[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < W; ++i) sum[u][i] = 0.0f;
        if (p.add != nullptr && column<W, SPREAD>(u0 + u, 0, lane, team) < p.n) {
            const Pack<T, W> a = load_columns<T, W, SPREAD>(static_cast<const T*>(p.add) + t * p.sadd, u0 + u, lane, team, p.n, p.bnd, 3);
#pragma unroll
            for (int i = 0; i < W; ++i) sum[u][i] = to_f32(a.v[i]);
        }
    }
    for (int j0 = 0; j0 < p.k; j0 += K) {
        int32_t r[K];
        float w[K];
        rows_of<K>(r, p.rows, t, j0, p.k, all, p.bnd, 1);
        weights_of<K>(w, p.weights, t, j0, p.k, p.bnd, 2);
        Pack<T, W> v[U][K];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (r[j] >= 0 && column<W, SPREAD>(u0 + u, 0, lane, team) < p.n)
                    v[u][j] = load_columns<T, W, SPREAD>(static_cast<const T*>(p.ys) + r[j] * p.sys, u0 + u, lane, team, p.n, p.bnd, 0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (r[j] >= 0)
#pragma unroll
                    for (int i = 0; i < W; ++i) sum[u][i] = fmaf(w[j], to_f32(v[u][j].v[i]), sum[u][i]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (column<W, SPREAD>(u0 + u, 0, lane, team) < p.n) {
            Pack<T, W> o;
#pragma unroll
            for (int i = 0; i < W; ++i) o.v[i] = from_f32<T>(sum[u][i]);
            store_columns<T, W, SPREAD>(static_cast<T*>(p.y) + t * p.sy, o, u0 + u, lane, team, p.n, p.bnd, 4);
        }
}

// For up to K of a token's slots at a time a team goes over dy[t] once, writes their rows
// of dys and sums up their dots. Teams are parts of a warp, or (BLOCK) a block.
template <typename T, int W, int K, bool SPREAD, bool BLOCK>
__global__ void __launch_bounds__(kThreads) combine_back_kernel(const CombineBackArgs p, int team) {
    constexpr int U = K >= 4 ? 1 : 4 / K;
    __shared__ float s_sum[BLOCK ? K * 32 : 1];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int lane = threadIdx.x & (team - 1), runs = static_cast<int>((p.n + team * W - 1) / (team * W));
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / team) + threadIdx.x / team, all = p.m * p.k;
    const bool here = t < p.m;                             // a warp's teams sum up together
    const int64_t used = load_one(p.offsets + p.experts, p.bnd, 3, 0);
    const T* dy = static_cast<const T*>(p.dy) + t * p.sdy;
    for (int j0 = 0; j0 < p.k; j0 += K) {
        int32_t r[K];
        float w[K], dot[K];
        rows_of<K>(r, p.rows, t, j0, here ? p.k : 0, all, p.bnd, 2);
        weights_of<K>(w, p.weights, t, j0, here ? p.k : 0, p.bnd, 4);
#pragma unroll
        for (int j = 0; j < K; ++j) dot[j] = 0.0f;
        for (int u0 = 0; u0 < runs && here; u0 += U) {
            Pack<T, W> g[U], v[U][K];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (column<W, SPREAD>(u0 + u, 0, lane, team) < p.n) {
                    g[u] = load_columns<T, W, SPREAD>(dy, u0 + u, lane, team, p.n, p.bnd, 0);
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        if (r[j] >= 0) v[u][j] = load_columns<T, W, SPREAD>(static_cast<const T*>(p.ys) + r[j] * p.sys, u0 + u, lane, team, p.n, p.bnd, 1);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (column<W, SPREAD>(u0 + u, 0, lane, team) < p.n)
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        if (r[j] >= 0) {
                            Pack<T, W> o;
#pragma unroll
                            for (int i = 0; i < W; ++i) {
                                const float d = to_f32(g[u].v[i]);
                                dot[j] = fmaf(d, to_f32(v[u][j].v[i]), dot[j]);
                                o.v[i] = from_f32<T>(d * w[j]);
                            }
                            store_columns<T, W, SPREAD>(static_cast<T*>(p.dys) + r[j] * p.sdys, o, u0 + u, lane, team, p.n, p.bnd, 5);
                        }
        }
        if constexpr (BLOCK) {
            if (j0 > 0) __syncthreads();                   // the last sums have been read
            sum_over_row<K, false>(dot, s_sum);
        } else {
            for (int o = team >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int j = 0; j < K; ++j) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        }
        if (here && lane == 0)
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (j0 + j < p.k) store_one(p.dweights + t * p.k + j0 + j, dot[j], p.bnd, 6);
    }
    if (here && t * p.k + p.k > used)
        for (int j = 0; j < p.k; ++j)
            if (t * p.k + j >= used)
                for (int u = 0; u < runs; ++u)
                    if (column<W, SPREAD>(u, 0, lane, team) < p.n)
                        store_columns<T, W, SPREAD>(static_cast<T*>(p.dys) + (t * p.k + j) * p.sdys, zero_pack<T, W>(), u, lane, team, p.n, p.bnd, 5);
}

// ---------------------------------------------------------------- many tokens
// The same for many tokens: a team is a warp or a block and goes from token to token, with
// the runs to come on their way into a ring of S in shared memory, in which each thread
// copies and reads only what is its own. A token's rows are known one token ahead. For sums of
// many slots "token" is one of its 2^split pieces of columns, so that all teams have about as
// much to do.
constexpr int kRingThreads = 256;
constexpr int ring_stages(int k) { return k >= 8 ? 3 : (k >= 4 ? 5 : 8); }

struct RingArgs {
    const void *one, *many;    // a row of each token: add (or null), dy; the experts' rows: ys
    int64_t m, n, s_one, s_many;
    int k, split;
    const int32_t* rows;
    const float* weights;      // or null: 1
    void* out;                 // y, or dys
    int64_t s_out;
    const int32_t* offsets;    // back: past offsets[experts] dys is zero
    int experts;
    float* dweights;
    BoundsOf<7> bnd;           // one, many, rows, weights, out, offsets, dweights
};

template <typename T, int K, bool BACK, bool BLOCK>
__global__ void __launch_bounds__(kRingThreads, 2) exchange_ring_kernel(const RingArgs p) {
    constexpr int W = 16 / sizeof(T), S = ring_stages(K), L = K + 1, TEAM = BLOCK ? kRingThreads : 32;
    extern __shared__ __align__(16) uint8_t s_ring[];      // [S][L][threads] runs: the token's if there is one, the experts'
    __shared__ float s_sum[2][BACK && BLOCK ? K * 32 : 1];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int lane = threadIdx.x & (TEAM - 1), runs = static_cast<int>((p.n + TEAM * W - 1) / (TEAM * W));
    const int split = !BACK && K > 2 ? p.split : 0, piece = (runs + (1 << split) - 1) >> split;       // runs of a piece; none is empty
    const int64_t items = p.m << split;
    const int64_t all = p.m * p.k, step = static_cast<int64_t>(gridDim.x) * (kRingThreads / TEAM);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kRingThreads / TEAM) + threadIdx.x / TEAM;
    uint8_t* mine = s_ring + threadIdx.x * 16;
    auto slot = [&](int s, int l) { return mine + (s * L + l) * kRingThreads * 16; };
    const int64_t used = BACK ? load_one(p.offsets + p.experts, p.bnd, 5, 0) : 0;

    // the copies' place in the sequence of runs
    auto run_of = [&](int64_t i) { return static_cast<int>(i & ((1 << split) - 1)) * piece; };
    auto end_of = [&](int run) { return run + piece < runs ? run + piece : runs; };
    int64_t f_item = first;
    int f_run = run_of(first), f_end = end_of(f_run);
    int32_t f_rows[K], f_next[K];
    auto rows_at = [&](int32_t (&r)[K], int64_t i) { rows_of<K>(r, p.rows, i >> split, 0, i < items ? p.k : 0, all, p.bnd, 2); };
    rows_at(f_rows, first);
    rows_at(f_next, first + step);
    auto fetch = [&](int s) {
        const int64_t c = (static_cast<int64_t>(f_run) * TEAM + lane) * W;
        if (f_item < items && c < p.n) {
            const T* one = static_cast<const T*>(p.one) + (f_item >> split) * p.s_one + c;
            if (p.one != nullptr && QL_IN(p.bnd, 0, one, 16)) copy_async<16>(slot(s, 0), one);
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (f_rows[j] >= 0) {
                    const T* many = static_cast<const T*>(p.many) + f_rows[j] * p.s_many + c;
                    if (QL_IN(p.bnd, 1, many, 16)) copy_async<16>(slot(s, 1 + j), many);
                }
        }
        copy_commit();                                     // a group for every run, also past the last
        if (++f_run == f_end) {
            f_item += step;
            f_run = run_of(f_item);
            f_end = end_of(f_run);
#pragma unroll
            for (int j = 0; j < K; ++j) f_rows[j] = f_next[j];
            rows_at(f_next, f_item + step);
        }
    };
    int32_t next[K];
    float w_next[K];                                       // (behind the copies they would wait for the ring to fill)
#pragma unroll
    for (int j = 0; j < K; ++j) next[j] = f_rows[j];
    weights_of<K>(w_next, p.weights, first >> split, 0, first < items ? p.k : 0, p.bnd, 3);
    for (int s = 0; s < S; ++s) fetch(s);
    int s = 0, turn = 0;
    for (int64_t item = first; item < items; item += step) {
        const int64_t t = item >> split;
        int32_t r[K];
        float w[K], dot[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            r[j] = next[j];
            w[j] = w_next[j];
            dot[j] = 0.0f;
        }
        rows_at(next, item + step);
        weights_of<K>(w_next, p.weights, (item + step) >> split, 0, item + step < items ? p.k : 0, p.bnd, 3);
        const int u0 = run_of(item), u1 = end_of(u0);
        for (int u = u0; u < u1; ++u) {
            copy_wait<S - 1>();
            const int64_t c = (static_cast<int64_t>(u) * TEAM + lane) * W;
            if (c < p.n) {
                Pack<T, W> one = zero_pack<T, W>();
                if (p.one != nullptr) one = *reinterpret_cast<const Pack<T, W>*>(slot(s, 0));
                float sum[W];
#pragma unroll
                for (int i = 0; i < W; ++i) sum[i] = to_f32(one.v[i]);
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (r[j] >= 0) {
                        const Pack<T, W> v = *reinterpret_cast<const Pack<T, W>*>(slot(s, 1 + j));
                        if constexpr (BACK) {
                            Pack<T, W> o;
#pragma unroll
                            for (int i = 0; i < W; ++i) {
                                dot[j] = fmaf(sum[i], to_f32(v.v[i]), dot[j]);
                                o.v[i] = from_f32<T>(sum[i] * w[j]);
                            }
                            store_pack<T, W>(static_cast<T*>(p.out) + r[j] * p.s_out + c, o, p.bnd, 4);
                        } else {
#pragma unroll
                            for (int i = 0; i < W; ++i) sum[i] = fmaf(w[j], to_f32(v.v[i]), sum[i]);
                        }
                    }
                if constexpr (!BACK) {
                    Pack<T, W> o;
#pragma unroll
                    for (int i = 0; i < W; ++i) o.v[i] = from_f32<T>(sum[i]);
                    store_pack<T, W>(static_cast<T*>(p.out) + t * p.s_out + c, o, p.bnd, 4);
                }
            }
            fetch(s);                                      // what it copies over has been read
            if (++s == S) s = 0;
        }
        if constexpr (BACK) {
            sum_over_row<K, !BLOCK>(dot, s_sum[turn]);
            turn ^= 1;                                     // the next token's sums go elsewhere
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (j < p.k) store_one(p.dweights + t * p.k + j, dot[j], p.bnd, 6);
            if (t * p.k + p.k > used)
                for (int j = 0; j < p.k; ++j)
                    if (t * p.k + j >= used)
                        for (int64_t c = lane * W; c < p.n; c += TEAM * W)
                            store_pack<T, W>(static_cast<T*>(p.out) + (t * p.k + j) * p.s_out + c, zero_pack<T, W>(), p.bnd, 4);
        }
    }
}

// The team for rows of n columns, `most` threads at most.
int team_of(int64_t n, int w, int most) {
    int team = 1;
    while (team < most && static_cast<int64_t>(team) * w < n) team *= 2;
    return team;
}
// Pieces of a row of n columns, and blocks for m tokens: those of one token follow one
// another, so that a row's pieces are on their way together (the other way round 4096 x 8
// rows of 7168 took 171 us to combine).
unsigned pieces_of(int64_t n, int w, int team, int runs) {
    const int64_t each = static_cast<int64_t>(team) * w * runs;
    return static_cast<unsigned>((n + each - 1) / each);
}
dim3 blocks_of(int64_t m, int team, unsigned pieces) {
    const int64_t per = kThreads / team;
    return dim3(static_cast<unsigned>((m + per - 1) / per * pieces));
}

template <typename T, bool SPREAD>
cudaError_t dispatch_s(const DispatchArgs& a, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    const int team = team_of(a.n, W, kThreads);
    const unsigned pieces = pieces_of(a.n, W, team, 4);
    return launch_after(dispatch_kernel<T, W, SPREAD>, blocks_of(a.m, team, pieces), kThreads, 0, st, a, team, pieces);
}
template <typename T, int K, bool SPREAD>
cudaError_t combine_k(const CombineArgs& a, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    const int team = team_of(a.n, W, kThreads);
    const unsigned pieces = pieces_of(a.n, W, team, combine_runs(K));
    return launch_after(combine_kernel<T, W, K, SPREAD>, blocks_of(a.m, team, pieces), kThreads, 0, st, a, team, pieces);
}
template <typename T, int K, bool SPREAD>
cudaError_t combine_back_k(const CombineBackArgs& a, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    if (a.n > 32 * 4 * W)
        return launch_after(combine_back_kernel<T, W, K, SPREAD, true>, dim3(static_cast<unsigned>(a.m)), kThreads, 0, st, a, kThreads);
    const int team = team_of(a.n, W, 32), per = kThreads / team;
    return launch_after(combine_back_kernel<T, W, K, SPREAD, false>, dim3(static_cast<unsigned>((a.m + per - 1) / per)), kThreads, 0, st, a, team);
}
// Slots at a time: k's own number where it is small.
#define QL_BY_SLOTS(F, T, SPREAD, a, ...)                               \
    ((a).k == 1 ? F<T, 1, SPREAD>(a, __VA_ARGS__)                       \
                : ((a).k == 2 ? F<T, 2, SPREAD>(a, __VA_ARGS__)         \
                              : ((a).k <= 4 ? F<T, 4, SPREAD>(a, __VA_ARGS__) : F<T, kSlots, SPREAD>(a, __VA_ARGS__))))

// Two blocks of ring on every SM, with a token to every warp at least; with fewer, a
// token to a block if it has work for one. Measured, ring by warps / by blocks / no ring, us:
//   sums       4096 x 8 of 7168 85 / 84 / 136, 4096 x 2 of 4096 18.7 / 22.9 / 21.9, 16384 x 1 of 4096 51 / 66 / 53,
//              8192 x 2 of 1024 12.7 / - / 18.5
//   gradients  163 / 163 / 177, 30.2 / 35.1 / 39.4, 71 / 100 / 116, 17.0 / - / 19.4
// fewer tokens, by blocks / no ring:
//   sums       1500 x 8 of 7168 34 / 52, 400 x 8 of 7168 13.2 / 16.8, 512 x 8 of 4096 10.2 / 12.6, 2400 x 2 of 8192 22.4 / 25.0,
//              1024 x 2 of 4096 7.3 / 5.6
//   gradients  63 / 73, 20.2 / 21.3, 15.5 / 21.2, 32.4 / 41.8, 12.0 / 12.4
template <typename T, int K, bool BACK>
bool ring_k(RingArgs a, cudaStream_t st, int num_sms, cudaError_t& e) {
    constexpr int smem = ring_stages(K) * (K + 1) * kRingThreads * 16;
    const int64_t blocks = static_cast<int64_t>(num_sms) * 2;
    const bool by_warps = a.m >= blocks * (kRingThreads / 32);
    if (!by_warps && (a.m < blocks || a.k * a.n * static_cast<int64_t>(sizeof(T)) < 32 * 1024)) return false;
    const int64_t teams = blocks * (by_warps ? kRingThreads / 32 : 1), run = (by_warps ? 32 : kRingThreads) * 16 / static_cast<int64_t>(sizeof(T));
    const int64_t runs = (a.n + run - 1) / run;
    // pieces: 4096 x 8 of 7168 85 us, by whole tokens 88, 3000 x 4 of 2048 14.4 and 15.7; but with fewer
    // slots their looking up costs more: 4096 x 2 of 4096 20.5 and 18.7
    a.split = 0;
    if (!BACK && K > 2)
        while (a.split < 3 && (a.m << a.split) < 6 * teams && runs >> a.split >= 4 && runs % (2 << a.split) == 0) ++a.split;
    auto kern = by_warps ? exchange_ring_kernel<T, K, BACK, false> : exchange_ring_kernel<T, K, BACK, true>;
    e = smem > 46 * 1024 ? ensure_smem_attr(reinterpret_cast<const void*>(kern), smem) : cudaSuccess;
    if (e == cudaSuccess) e = launch_after(kern, dim3(static_cast<unsigned>(blocks)), kRingThreads, smem, st, a);
    return true;
}
template <typename T, bool BACK>
bool ring(const RingArgs& a, cudaStream_t st, int num_sms, cudaError_t& e) {
    constexpr int W = 16 / sizeof(T);
    if (a.k > 8 || a.n < 32 * W) return false;
    if (a.k == 1) return ring_k<T, 1, BACK>(a, st, num_sms, e);
    if (a.k == 2) return ring_k<T, 2, BACK>(a, st, num_sms, e);
    if (a.k <= 4) return ring_k<T, 4, BACK>(a, st, num_sms, e);
    return ring_k<T, 8, BACK>(a, st, num_sms, e);
}

template <typename T>
cudaError_t dispatch_t(const DispatchArgs& a, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    const bool vec = a.n % W == 0 && rows_aligned(a.x, sizeof(T), a.sx, a.m, 16) && rows_aligned(a.xs, sizeof(T), a.sxs, a.m * a.k, 16);
    return vec ? dispatch_s<T, false>(a, st) : dispatch_s<T, true>(a, st);
}
template <typename T>
cudaError_t combine_t(const CombineArgs& a, cudaStream_t st, int num_sms) {
    constexpr int W = 16 / sizeof(T);
    const bool vec = a.n % W == 0 && rows_aligned(a.ys, sizeof(T), a.sys, a.m * a.k, 16) && rows_aligned(a.y, sizeof(T), a.sy, a.m, 16) &&
                     (a.add == nullptr || rows_aligned(a.add, sizeof(T), a.sadd, a.m, 16));
    cudaError_t e;
    if (vec && ring<T, false>(RingArgs{a.add, a.ys, a.m, a.n, a.sadd, a.sys, a.k, 0, a.rows, a.weights, a.y, a.sy, nullptr, 0, nullptr,
                                       {{a.bnd.s[3], a.bnd.s[0], a.bnd.s[1], a.bnd.s[2], a.bnd.s[4], Span{0, 0}, Span{0, 0}}, a.bnd.status}},
                              st, num_sms, e))
        return e;
    return vec ? QL_BY_SLOTS(combine_k, T, false, a, st) : QL_BY_SLOTS(combine_k, T, true, a, st);
}
template <typename T>
cudaError_t combine_back_t(const CombineBackArgs& a, cudaStream_t st, int num_sms) {
    constexpr int W = 16 / sizeof(T);
    const bool vec = a.n % W == 0 && rows_aligned(a.ys, sizeof(T), a.sys, a.m * a.k, 16) && rows_aligned(a.dy, sizeof(T), a.sdy, a.m, 16) &&
                     rows_aligned(a.dys, sizeof(T), a.sdys, a.m * a.k, 16);
    cudaError_t e;
    if (vec && ring<T, true>(RingArgs{a.dy, a.ys, a.m, a.n, a.sdy, a.sys, a.k, 0, a.rows, a.weights, a.dys, a.sdys, a.offsets, a.experts, a.dweights,
                                      {{a.bnd.s[0], a.bnd.s[1], a.bnd.s[2], a.bnd.s[4], a.bnd.s[5], a.bnd.s[3], a.bnd.s[6]}, a.bnd.status}},
                             st, num_sms, e))
        return e;
    return vec ? QL_BY_SLOTS(combine_back_k, T, false, a, st) : QL_BY_SLOTS(combine_back_k, T, true, a, st);
}

}  // namespace

// Slots per chunk: whole rounds of every warp, and no more than 128 chunks while a
// warp's counts fit their 16 bits (65536 x 8 slots over 64 experts: 64 chunks 20.1 us, 128
// 13.4, 256 18.4). One block takes 1.4 us for every round more: 512 x 8 slots 8.0 us alone,
// 5.0 by chunks.
int64_t plan_chunk(int64_t slots) {
    int64_t rounds = (slots + 128 * kPlanThreads - 1) / (128 * kPlanThreads);
    if (rounds < 1) rounds = 1;
    if (rounds > 60) rounds = 60;
    return rounds * kPlanThreads;
}
size_t plan_workspace(int64_t slots, int experts) {
    const int64_t chunk = plan_chunk(slots);
    return slots <= chunk ? 0 : static_cast<size_t>((slots + chunk - 1) / chunk) * static_cast<size_t>(experts) * sizeof(int32_t);
}

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st) {
    const unsigned chunks = a.slots <= a.chunk ? 1u : static_cast<unsigned>((a.slots + a.chunk - 1) / a.chunk);
    if (chunks > 1)
        if (cudaError_t e = launch_after(plan_count_kernel, dim3(chunks), kPlanThreads, 0, st, a); e != cudaSuccess) return e;
    return launch_after(plan_place_kernel, dim3(chunks), kPlanThreads, 0, st, a);
}

cudaError_t launch_dispatch(const DispatchArgs& a, cudaStream_t st) {
    return a.es == 2 ? dispatch_t<__nv_bfloat16>(a, st) : dispatch_t<float>(a, st);
}
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t st, int num_sms) {
    return a.bf16 ? combine_t<__nv_bfloat16>(a, st, num_sms) : combine_t<float>(a, st, num_sms);
}
cudaError_t launch_combine_back(const CombineBackArgs& a, cudaStream_t st, int num_sms) {
    return a.bf16 ? combine_back_t<__nv_bfloat16>(a, st, num_sms) : combine_back_t<float>(a, st, num_sms);
}

}  // namespace ql
