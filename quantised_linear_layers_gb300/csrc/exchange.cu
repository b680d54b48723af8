// The exchange of rows with the experts: the order of the slots (token, j) by
// expert (a stable counting sort), rows to their places, and the weighted sums
// back, with the gradients of both.
#include "route.cuh"

#include "rows.cuh"

namespace ql {
namespace {

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanRoom = kRouteMaxExperts + 1;            // and a place for no expert

// The expert of a slot; `experts` for none.
__device__ __forceinline__ int expert_of(const PlanArgs& p, int64_t slot) {
    const int e = load_one(p.chosen + slot, p.bnd, 0, -1);
    if (e >= 0 && e < p.experts) return e;
    if (e != -1) atomicOr(p.dev_status, kDevErrBadIndex);
    return p.experts;
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
    __shared__ uint16_t s_warp[kPlanWarps][kPlanRoom];     // slots of a warp, then of the warps before
    __shared__ int s_total[kRouteMaxExperts], s_before[kRouteMaxExperts];
    __shared__ int s_sum[kPlanWarps];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kPlanWarps * kPlanRoom; i += kPlanThreads) (&s_warp[0][0])[i] = 0;
    for (int e = threadIdx.x; e < kRouteMaxExperts; e += kPlanThreads) s_total[e] = s_before[e] = 0;
    __syncthreads();
    const int64_t run = p.chunk / kPlanWarps;              // a multiple of 32
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.chunk + warp * run;
    const int64_t last = first + run < p.slots ? first + run : p.slots;
    const uint32_t below = (1u << lane) - 1u;
    for (int64_t i = first; i < last; i += 32) {
        const int e = i + lane < last ? expert_of(p, i + lane) : p.experts;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        if ((same & below) == 0) s_warp[warp][e] = static_cast<uint16_t>(s_warp[warp][e] + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kPlanThreads) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < kPlanWarps; ++w) {
            const int c = s_warp[w][e];
            s_warp[w][e] = static_cast<uint16_t>(sum);
            sum += c;
        }
        if (p.counts == nullptr) s_total[e] = sum;         // one chunk
    }
    if (p.counts != nullptr) {
        int room = 32;                                     // threads side by side over the experts
        while (room < p.experts) room *= 2;
        const int e = threadIdx.x & (room - 1), share = threadIdx.x / room, shares = kPlanThreads / room;
        if (e < p.experts) {
            int total = 0, before = 0;
#pragma unroll 8
            for (int c = share; c < static_cast<int>(gridDim.x); c += shares) {
                const int v = load_one(p.counts + static_cast<int64_t>(c) * p.experts + e, p.bnd, 3, 0);
                total += v;
                if (c < static_cast<int>(blockIdx.x)) before += v;
            }
            atomicAdd(&s_total[e], total);
            atomicAdd(&s_before[e], before);
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
    int ahead = 0;
    for (int w = 0; w < warp; ++w) ahead += s_sum[w];
    const int start = ahead + sum - mine;
    if (threadIdx.x < p.experts) s_before[threadIdx.x] += start;
    if (blockIdx.x == 0 && threadIdx.x <= p.experts) store_one(p.offsets + threadIdx.x, start, p.bnd, 1);
    __syncthreads();
    for (int64_t i = first; i < last; i += 32) {
        const int e = i + lane < last ? expert_of(p, i + lane) : p.experts;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int at = s_warp[warp][e];
        __syncwarp();
        if ((same & below) == 0) s_warp[warp][e] = static_cast<uint16_t>(at + __popc(same));
        __syncwarp();
        if (i + lane < last) store_one(p.rows + i + lane, e < p.experts ? s_before[e] + at + __popc(same & below) : -1, p.bnd, 2);
    }
}

// ---------------------------------------------------------------- rows there and back
constexpr int kThreads = 128;

// A row that `rows` names, or -1: what lies outside [0, all) is none.
template <typename B>
__device__ __forceinline__ int64_t row_at(const int32_t* rows, int64_t slot, int64_t all, const B& b, int span) {
    const int64_t r = load_one(rows + slot, b, span, -1);
    return r < all ? r : -1;
}

// A block has a token and a piece of its columns, held in registers and written to
// each of the token's k rows. E: an element, or 16 bytes of them (n and strides then
// count those). Row t k + j of xs is this token's to clear if no slot has it.
template <typename E>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchArgs p) {
    constexpr int U = 4;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int64_t t = blockIdx.x, all = p.m * p.k;
    const int64_t c0 = static_cast<int64_t>(blockIdx.y) * (kThreads * U) + threadIdx.x;
    const E* x = static_cast<const E*>(p.x) + t * p.sx;
    E v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + u * kThreads;
        v[u] = c < p.n ? load_one(x + c, p.bnd, 0, E{}) : E{};
    }
    const int64_t used = load_one(p.offsets + p.experts, p.bnd, 2, 0);
    for (int j = 0; j < p.k; ++j) {
        const int64_t r = row_at(p.rows, t * p.k + j, all, p.bnd, 1);
        if (r >= 0) {
            E* xs = static_cast<E*>(p.xs) + r * p.sxs;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * kThreads < p.n) store_one(xs + c0 + u * kThreads, v[u], p.bnd, 3);
        }
        if (t * p.k + j >= used) {
            E* xs = static_cast<E*>(p.xs) + (t * p.k + j) * p.sxs;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * kThreads < p.n) store_one(xs + c0 + u * kThreads, E{}, p.bnd, 3);
        }
    }
}

// A block has a token and a piece of its columns; a thread W columns, whose k terms it
// adds up in fp32 in the order of j, eight loads at a time.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs p) {
    constexpr int J = 8;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int64_t t = blockIdx.x, all = p.m * p.k;
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x) * W;
    if (c >= p.n) return;
    float sum[W];
#pragma unroll
    for (int i = 0; i < W; ++i) sum[i] = 0.0f;
    if (p.add != nullptr) {
        const Pack<T, W> a = load_pack<T, W>(static_cast<const T*>(p.add) + t * p.sadd + c, p.bnd, 3);
#pragma unroll
        for (int i = 0; i < W; ++i) sum[i] = to_f32(a.v[i]);
    }
    for (int j0 = 0; j0 < p.k; j0 += J) {
        Pack<T, W> v[J];
        float w[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t r = j0 + j < p.k ? row_at(p.rows, t * p.k + j0 + j, all, p.bnd, 1) : -1;
            w[j] = r < 0 ? 0.0f : (p.weights != nullptr ? load_one(p.weights + t * p.k + j0 + j, p.bnd, 2, 0.0f) : 1.0f);
            v[j] = r < 0 ? zero_pack<T, W>() : load_pack<T, W>(static_cast<const T*>(p.ys) + r * p.sys + c, p.bnd, 0);
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < W; ++i) sum[i] = fmaf(w[j], to_f32(v[j].v[i]), sum[i]);
    }
    Pack<T, W> o;
#pragma unroll
    for (int i = 0; i < W; ++i) o.v[i] = from_f32<T>(sum[i]);
    store_pack<T, W>(static_cast<T*>(p.y) + t * p.sy + c, o, p.bnd, 4);
}

// A block has a token: for up to eight of its slots at a time it goes over dy[t] once,
// writes their rows of dys and sums up their dots.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) combine_back_kernel(const CombineBackArgs p) {
    constexpr int J = 8;
    __shared__ float s_sum[J * 32];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int64_t t = blockIdx.x, all = p.m * p.k;
    const T* dy = static_cast<const T*>(p.dy) + t * p.sdy;
    const int64_t used = load_one(p.offsets + p.experts, p.bnd, 3, 0);
    for (int j0 = 0; j0 < p.k; j0 += J) {
        int64_t r[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            r[j] = j0 + j < p.k ? row_at(p.rows, t * p.k + j0 + j, all, p.bnd, 2) : -1;
            w[j] = r[j] < 0 ? 0.0f : load_one(p.weights + t * p.k + j0 + j, p.bnd, 4, 0.0f);
            dot[j] = 0.0f;
        }
        for (int64_t c = static_cast<int64_t>(threadIdx.x) * W; c < p.n; c += kThreads * W) {
            const Pack<T, W> g = load_pack<T, W>(dy + c, p.bnd, 0);
            Pack<T, W> v[J];
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (r[j] >= 0) v[j] = load_pack<T, W>(static_cast<const T*>(p.ys) + r[j] * p.sys + c, p.bnd, 1);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (r[j] >= 0) {
                    Pack<T, W> o;
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float d = to_f32(g.v[i]);
                        dot[j] = fmaf(d, to_f32(v[j].v[i]), dot[j]);
                        o.v[i] = from_f32<T>(d * w[j]);
                    }
                    store_pack<T, W>(static_cast<T*>(p.dys) + r[j] * p.sdys + c, o, p.bnd, 5);
                }
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (j0 + j < p.k && t * p.k + j0 + j >= used)
                    store_pack<T, W>(static_cast<T*>(p.dys) + (t * p.k + j0 + j) * p.sdys + c, zero_pack<T, W>(), p.bnd, 5);
        }
        __syncthreads();                                   // the last slots' sums have been read
        sum_over_row<J, false>(dot, s_sum);
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (threadIdx.x == j && j0 + j < p.k) store_one(p.dweights + t * p.k + j0 + j, dot[j], p.bnd, 6);
    }
}

unsigned pieces(int64_t n, int64_t each) { return static_cast<unsigned>((n + each - 1) / each); }

template <typename T>
cudaError_t combine_t(const CombineArgs& a, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    const bool vec = a.n % W == 0 && rows_aligned(a.ys, sizeof(T), a.sys, a.m * a.k, 16) && rows_aligned(a.y, sizeof(T), a.sy, a.m, 16) &&
                     (a.add == nullptr || rows_aligned(a.add, sizeof(T), a.sadd, a.m, 16));
    if (vec)
        return launch_after(combine_kernel<T, W>, dim3(static_cast<unsigned>(a.m), pieces(a.n, kThreads * W)), kThreads, 0, st, a);
    return launch_after(combine_kernel<T, 1>, dim3(static_cast<unsigned>(a.m), pieces(a.n, kThreads)), kThreads, 0, st, a);
}
template <typename T>
cudaError_t combine_back_t(const CombineBackArgs& a, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    const bool vec = a.n % W == 0 && rows_aligned(a.ys, sizeof(T), a.sys, a.m * a.k, 16) && rows_aligned(a.dy, sizeof(T), a.sdy, a.m, 16) &&
                     rows_aligned(a.dys, sizeof(T), a.sdys, a.m * a.k, 16);
    if (vec) return launch_after(combine_back_kernel<T, W>, dim3(static_cast<unsigned>(a.m)), kThreads, 0, st, a);
    return launch_after(combine_back_kernel<T, 1>, dim3(static_cast<unsigned>(a.m)), kThreads, 0, st, a);
}
template <typename E>
cudaError_t dispatch_e(DispatchArgs a, int64_t per, cudaStream_t st) {
    a.n /= per;
    a.sx /= per;
    a.sxs /= per;
    return launch_after(dispatch_kernel<E>, dim3(static_cast<unsigned>(a.m), pieces(a.n, kThreads * 4)), kThreads, 0, st, a);
}

}  // namespace

// Slots per chunk: whole rounds of every warp, and no more than 128 chunks while a
// warp's counts fit their 16 bits.
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

cudaError_t launch_dispatch(const DispatchArgs& a, cudaStream_t st, int num_sms) {
    (void)num_sms;
    if ((a.n * a.es) % 16 == 0 && rows_aligned(a.x, a.es, a.sx, a.m, 16) && rows_aligned(a.xs, a.es, a.sxs, a.m * a.k, 16)) {
        DispatchArgs v = a;
        if (a.m <= 1) v.sx = 0;
        if (a.m * a.k <= 1) v.sxs = 0;
        return dispatch_e<uint4>(v, 16 / a.es, st);
    }
    return a.es == 2 ? dispatch_e<uint16_t>(a, 1, st) : dispatch_e<uint32_t>(a, 1, st);
}
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t st, int num_sms) {
    (void)num_sms;
    return a.bf16 ? combine_t<__nv_bfloat16>(a, st) : combine_t<float>(a, st);
}
cudaError_t launch_combine_back(const CombineBackArgs& a, cudaStream_t st) {
    return a.bf16 ? combine_back_t<__nv_bfloat16>(a, st) : combine_back_t<float>(a, st);
}

}  // namespace ql
