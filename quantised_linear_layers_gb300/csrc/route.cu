// Routing: which experts a token goes to, with which weights, and the gradient.
//
// A warp has a token; a lane has NV consecutive experts in registers. Choices are
// compared as unsigned integers in the order of the numbers that they stand for:
// 0 for an expert out of reach (logit or bias -inf), 1 for a NaN. Each of k rounds
// takes the largest key of the warp, the lowest index first.
//
// The choice is what 64 bits say. Without a bias experts are compared by their
// logits, since both scores rise with them: exact. With one, or where a group's
// score is a sum, fp32 scores with a bound on their error decide wherever the gaps
// that matter are wider than it; the other tokens are done again in 64 bits.
#include "route.cuh"

#include "rows.cuh"

namespace ql {
namespace {

constexpr int kWarps = 4;
constexpr uint32_t kAll = 0xffffffffu;
constexpr uint32_t kUnreached = 0u, kNanKey = 1u;

__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);          // -0 is 0
    return u ^ (static_cast<int32_t>(u) < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ (static_cast<int32_t>(key) < 0 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// e / size for e < 512: magic = ceil(2^20 / size); e size < 2^20.
__device__ __forceinline__ int over(int e, int magic) { return (e * magic) >> 20; }

// A token's logits, NV to a lane; -inf past the last.
template <typename T, int NV, bool VEC>
__device__ __forceinline__ void load_row(float (&l)[NV], const T* row, int experts, const Bounds& bnd, int span) {
    const int e0 = (threadIdx.x & 31) * NV;
    if constexpr (VEC) {                                   // NV elements or none
        if (e0 < experts) {
            const Pack<T, NV> v = load_pack<T, NV>(row + e0, bnd, span);
#pragma unroll
            for (int i = 0; i < NV; ++i) l[i] = to_f32(v.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) l[i] = -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            l[i] = e0 + i < experts ? to_f32(load_one(row + e0 + i, bnd, span, from_f32<T>(0.0f))) : -INFINITY;
    }
}

// The k best of a token in 64 bits: lane j gets the j-th one's index, or -1.
// c: 512 doubles of shared memory, the warp's own.
template <int NV>
__device__ __noinline__ int choose_exact(const RouteArgs& p, const float (&l)[NV], const float (&b)[NV], float top, int magic,
                                         double* c) {
    const int lane = threadIdx.x & 31;
    const double lowest = -1e300;
    double total = 1.0;
    double v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = p.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l[i]))) : exp(static_cast<double>(l[i]) - static_cast<double>(top));
    if (!p.sigmoid) {
        total = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i) total += v[i];
        total = warp_sum(total);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool reached = l[i] != -INFINITY && b[i] != -INFINITY;
        double x = v[i] / total + static_cast<double>(b[i]);
        if (x != x) x = lowest;
        c[lane * NV + i] = reached ? x : -INFINITY;
        v[i] = !reached ? -INFINITY : (p.bias != nullptr ? x : static_cast<double>(l[i]));
    }
    __syncwarp();
    if (p.kept < p.groups) {
        const int size = p.experts / p.groups;
        double score = -INFINITY;
        if (lane < p.groups) {
            double best = -INFINITY, next = -INFINITY;
            for (int i = 0; i < size; ++i) {
                const double x = c[lane * size + i];
                if (x > best) {
                    next = best;
                    best = x;
                } else if (x > next) {
                    next = x;
                }
            }
            score = p.group_best > 1 && next != -INFINITY ? best + next : best;
        }
        uint32_t kept = 0;
        for (int r = 0; r < p.kept; ++r) {
            double s = (kept >> lane) & 1u ? -INFINITY : score;
            int at = lane;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const double s2 = __shfl_xor_sync(kAll, s, o);
                const int at2 = __shfl_xor_sync(kAll, at, o);
                if (s2 > s || (s2 == s && at2 < at)) {
                    s = s2;
                    at = at2;
                }
            }
            if (s == -INFINITY) break;
            kept |= 1u << at;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (((kept >> (over(lane * NV + i, magic) & 31)) & 1u) == 0u) v[i] = -INFINITY;
    }
    int mine = -1;
    for (int r = 0; r < p.k; ++r) {
        double s = -INFINITY;
        int at = 1 << 20;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (v[i] > s) {
                s = v[i];
                at = lane * NV + i;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double s2 = __shfl_xor_sync(kAll, s, o);
            const int at2 = __shfl_xor_sync(kAll, at, o);
            if (s2 > s || (s2 == s && at2 < at)) {
                s = s2;
                at = at2;
            }
        }
        if (s == -INFINITY) break;
        if (lane == r) mine = at;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (at == lane * NV + i) v[i] = -INFINITY;
    }
    return mine;
}

template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs p) {
    __shared__ double s_row[kWarps][NV * 32];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= p.m) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.sl;
    float l[NV], b[NV];
    load_row<T, NV, VEC>(l, row, p.experts, p.bnd, 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        b[i] = p.bias != nullptr && e < p.experts ? load_one(p.bias + e, p.bnd, 1, 0.0f) : 0.0f;
    }
    const bool grouped = p.kept < p.groups, sums = grouped && p.group_best > 1;
    const bool biased = p.bias != nullptr, scored = biased || sums;
    const int size = p.experts / p.groups;
    const int magic = ((1 << 20) + size - 1) / size;

    bool nan = false;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        nan |= l[i] != l[i] || b[i] != b[i];
        top = fmaxf(top, l[i]);
    }
    nan = __any_sync(kAll, nan);
    // row sums of the softmax are only needed where a score is
    const bool whole = !p.sigmoid && (scored || !p.renormalise);
    float total = 1.0f;
    if (whole) top = warp_max(top);
    const float base = top == -INFINITY ? 0.0f : top;

    uint32_t key[NV];
    float s[NV];
    float bound = 0.0f;                                    // of a choice's error
    if (whole || scored) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            s[i] = p.sigmoid ? 1.0f / (1.0f + expf(-l[i])) : expf(l[i] - base);
            sum += s[i];
        }
        if (!p.sigmoid) {
            total = warp_sum(sum);
            const float inv = 1.0f / total;
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] *= inv;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool reached = l[i] != -INFINITY && b[i] != -INFINITY;
        const float c = biased ? s[i] + b[i] : l[i];
        key[i] = !reached ? kUnreached : (c != c ? kNanKey : key_of(c));
    }
    if (scored) {
        // relative to the largest score: expf 2^-22, 1 + e and the division 2^-24 each, a
        // softmax's sum at most 21 roundings; one rounding of c, of s + |b| at most
        const float unit = p.sigmoid ? 0x1p-20f : 0x1p-18f;
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > kNanKey) most = fmaxf(most, fmaf(s[i], unit, fabsf(b[i]) * 0x1p-23f));
        bound = warp_max(most);
    }

    bool unsure = false;
    if (grouped) {
        // scores of the groups: lane g has that of group g
        uint32_t group = kUnreached;
        float* c = reinterpret_cast<float*>(s_row[warp]);
        uint32_t* ck = reinterpret_cast<uint32_t*>(c);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint32_t v = key[i];
            if (sums && !biased) v = v <= kNanKey ? v : key_of(s[i]);
            ck[lane * NV + i] = v;
        }
        __syncwarp();
        if (lane < p.groups) {
            uint32_t best = 0, next = 0;
            const uint32_t* of = ck + lane * size;
            for (int i = 0, at = lane; i < size; ++i, ++at) {
                while (at >= size) at -= size;             // lanes start at different banks
                const uint32_t v = of[at];
                next = max(next, min(best, v));
                best = max(best, v);
            }
            group = best;
            if (p.group_best > 1 && next > kNanKey) group = key_of(value_of(best) + value_of(next));
        }
        uint32_t kept = 0, last = 0;
        for (int r = 0; r <= p.kept; ++r) {
            const uint32_t v = (kept >> lane) & 1u ? 0u : group;
            const uint32_t best = __reduce_max_sync(kAll, v);
            if (r == p.kept) {                             // the best that stays out
                if (scored && best > kNanKey) unsure = value_of(last) - value_of(best) <= 6.0f * bound;      // two sums of two
                break;
            }
            if (best == 0) break;
            kept |= 1u << (__ffs(__ballot_sync(kAll, v == best)) - 1);
            last = best;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (((kept >> (over(lane * NV + i, magic) & 31)) & 1u) == 0u) key[i] = kUnreached;
    }

    int mine = -1;                                         // lane j: the j-th choice
    uint32_t my_key = 0;
    for (int r = 0; r < p.k; ++r) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) best = max(best, key[i]);
        const uint32_t most = __reduce_max_sync(kAll, best);
        if (most == 0) break;
        const int from = __ffs(__ballot_sync(kAll, best == most)) - 1;
        int at = 0;
        if (lane == from) {
            bool found = false;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (!found && key[i] == most) {
                    found = true;
                    key[i] = 0;
                    at = lane * NV + i;
                }
        }
        at = __shfl_sync(kAll, at, from);
        if (lane == r) {
            mine = at;
            my_key = most;
        }
    }
    float lg = mine >= 0 ? to_f32(load_one(row + mine, p.bnd, 0, from_f32<T>(0.0f))) : -INFINITY;
    if (biased) {
        // gaps between choices next to one another, and from the last to what stays out;
        // the same logit and bias are a tie in any precision
        const float b1 = mine >= 0 ? load_one(p.bias + mine, p.bnd, 1, 0.0f) : 0.0f;
        const uint32_t key2 = __shfl_down_sync(kAll, my_key, 1);
        const float lg2 = __shfl_down_sync(kAll, lg, 1), b2 = __shfl_down_sync(kAll, b1, 1);
        if (lane < p.k - 1 && key2 > kNanKey && value_of(my_key) - value_of(key2) <= 3.0f * bound && (lg != lg2 || b1 != b2))
            unsure = true;
        const uint32_t last = __shfl_sync(kAll, my_key, p.k - 1);
        const float llast = __shfl_sync(kAll, lg, p.k - 1), blast = __shfl_sync(kAll, b1, p.k - 1);
        if (last > kNanKey) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (key[i] > kNanKey && value_of(last) - value_of(key[i]) <= 3.0f * bound && (l[i] != llast || b[i] != blast))
                    unsure = true;
        }
    }
    if (__any_sync(kAll, unsure) && !nan) {
        __syncwarp();
        if (!biased) {
#pragma unroll
            for (int i = 0; i < NV; ++i) b[i] = 0.0f;
        }
        mine = choose_exact<NV>(p, l, b, whole ? base : 0.0f, magic, s_row[warp]);
        lg = mine >= 0 ? to_f32(load_one(row + mine, p.bnd, 0, from_f32<T>(0.0f))) : -INFINITY;
    }

    float w;
    if (p.renormalise) {
        // shares of the chosen: every term is taken relative to the largest, so that
        // none of them underflows with it
        const float most = warp_max(lg);
        const float ref = p.sigmoid ? fminf(most, 0.0f) : (most == -INFINITY ? 0.0f : most);
        float e = 0.0f;
        if (mine >= 0) {
            if (!p.sigmoid) e = expf(lg - ref);
            else e = lg <= 0.0f ? expf(lg - ref) / (1.0f + expf(lg)) : 1.0f / (1.0f + expf(-lg));
        }
        const float all = warp_sum(e);
        w = mine >= 0 ? e / all * p.scale : 0.0f;
    } else if (mine < 0) {
        w = 0.0f;
    } else {
        w = (p.sigmoid ? 1.0f / (1.0f + expf(-lg)) : expf(lg - base) / total) * p.scale;
    }
    if (nan && mine >= 0) w = __int_as_float(0x7fffffff);
    if (lane < p.k) {
        store_one(p.weights + t * p.k + lane, w, p.bnd, 2);
        store_one(p.chosen + t * p.k + lane, mine, p.bnd, 3);
    }
}

// Gradient with respect to the logits. With dw' = scale dw:
//   softmax          ds_j = dw'_j at the chosen, dl = s (ds - sum ds s): every expert
//   renormalised     q the chosen's shares, dl_j = q_j (dw'_j - sum q dw') for a softmax,
//                    times 1 - s_j for a sigmoid: the chosen alone
//   sigmoid          dl_j = dw'_j s_j (1 - s_j): the chosen alone
// The warp gathers what its lanes have for the chosen in a row of shared memory, slot
// by slot, so that an expert named twice gets both.
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) route_back_kernel(const RouteBackArgs p) {
    __shared__ float s_row[kWarps][NV * 32];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= p.m) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.sl;
    int e = -1;
    float g = 0.0f, lg = -INFINITY;
    if (lane < p.k) {
        e = load_one(p.chosen + t * p.k + lane, p.bnd, 2, -1);
        if (e < 0 || e >= p.experts) e = -1;
    }
    if (e >= 0) {
        g = load_one(p.dweights + t * p.k + lane, p.bnd, 0, 0.0f) * p.scale;
        lg = to_f32(load_one(row + e, p.bnd, 1, from_f32<T>(0.0f)));
    }
    const bool dense = !p.sigmoid && !p.renormalise;
    float l[NV], base = 0.0f, total = 1.0f;
    if (dense) {
        load_row<T, NV, VEC>(l, row, p.experts, p.bnd, 1);
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) top = fmaxf(top, l[i]);
        top = warp_max(top);
        base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            l[i] = expf(l[i] - base);
            sum += l[i];
        }
        total = warp_sum(sum);
        if (total == 0.0f) total = 1.0f;                   // no expert within reach
    }
    float v = 0.0f, mean = 0.0f;
    if (p.renormalise) {
        const float most = warp_max(lg);
        const float ref = p.sigmoid ? fminf(most, 0.0f) : (most == -INFINITY ? 0.0f : most);
        float q = 0.0f, rest = 1.0f;                       // rest: 1 - s
        if (e >= 0) {
            if (!p.sigmoid) {
                q = expf(lg - ref);
            } else {
                const float a = expf(-fabsf(lg)), small = a / (1.0f + a), large = 1.0f / (1.0f + a);
                q = lg <= 0.0f ? expf(lg - ref) * large : large;
                rest = lg <= 0.0f ? large : small;
            }
        }
        const float all = warp_sum(q);
        q = all == 0.0f ? 0.0f : q / all;
        mean = warp_sum(e >= 0 ? q * g : 0.0f);
        if (e >= 0) v = q * rest * (g - mean);
    } else if (p.sigmoid) {
        const float a = expf(-fabsf(lg)), one = 1.0f / (1.0f + a);
        if (e >= 0) v = g * a * one * one;                 // s (1 - s)
    } else {
        v = g;
        mean = warp_sum(e >= 0 ? g * (expf(lg - base) / total) : 0.0f);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) s_row[warp][lane * NV + i] = 0.0f;
    __syncwarp();
    for (int j = 0; j < p.k; ++j) {
        if (lane == j && e >= 0) s_row[warp][e] += v;
        __syncwarp();
    }
    T* out = static_cast<T*>(p.dlogits) + t * p.sd;
    float d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        d[i] = s_row[warp][lane * NV + i];
        if (dense) d[i] = l[i] / total * (d[i] - mean);
    }
    if constexpr (VEC) {
        if (lane * NV < p.experts) {
            Pack<T, NV> o;
#pragma unroll
            for (int i = 0; i < NV; ++i) o.v[i] = from_f32<T>(d[i]);
            store_pack<T, NV>(out + lane * NV, o, p.bnd, 3);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane * NV + i < p.experts) store_one(out + lane * NV + i, from_f32<T>(d[i]), p.bnd, 3);
    }
}

unsigned blocks(int64_t m) { return static_cast<unsigned>((m + kWarps - 1) / kWarps); }

// Lanes of NV elements whose loads are whole.
bool vec_rows(const void* p, int64_t es, int64_t stride, int64_t m, int experts, int nv) {
    const int64_t bytes = es * nv < 16 ? es * nv : 16;
    return experts % nv == 0 && rows_aligned(p, es, stride, m, bytes);
}

template <typename T, int NV>
cudaError_t route_nv(const RouteArgs& a, cudaStream_t st) {
    if (vec_rows(a.logits, sizeof(T), a.sl, a.m, a.experts, NV))
        return launch_after(route_kernel<T, NV, true>, dim3(blocks(a.m)), kWarps * 32, 0, st, a);
    return launch_after(route_kernel<T, NV, false>, dim3(blocks(a.m)), kWarps * 32, 0, st, a);
}
template <typename T>
cudaError_t route_t(const RouteArgs& a, cudaStream_t st) {
    if (a.experts <= 32) return route_nv<T, 1>(a, st);
    if (a.experts <= 64) return route_nv<T, 2>(a, st);
    if (a.experts <= 128) return route_nv<T, 4>(a, st);
    if (a.experts <= 256) return route_nv<T, 8>(a, st);
    return route_nv<T, 16>(a, st);
}

template <typename T, int NV>
cudaError_t back_nv(const RouteBackArgs& a, cudaStream_t st) {
    if (vec_rows(a.logits, sizeof(T), a.sl, a.m, a.experts, NV) && vec_rows(a.dlogits, sizeof(T), a.sd, a.m, a.experts, NV))
        return launch_after(route_back_kernel<T, NV, true>, dim3(blocks(a.m)), kWarps * 32, 0, st, a);
    return launch_after(route_back_kernel<T, NV, false>, dim3(blocks(a.m)), kWarps * 32, 0, st, a);
}
template <typename T>
cudaError_t back_t(const RouteBackArgs& a, cudaStream_t st) {
    if (a.experts <= 32) return back_nv<T, 1>(a, st);
    if (a.experts <= 64) return back_nv<T, 2>(a, st);
    if (a.experts <= 128) return back_nv<T, 4>(a, st);
    if (a.experts <= 256) return back_nv<T, 8>(a, st);
    return back_nv<T, 16>(a, st);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
    return a.bf16 ? route_t<__nv_bfloat16>(a, st) : route_t<float>(a, st);
}
cudaError_t launch_route_back(const RouteBackArgs& a, cudaStream_t st) {
    return a.bf16 ? back_t<__nv_bfloat16>(a, st) : back_t<float>(a, st);
}

}  // namespace ql
