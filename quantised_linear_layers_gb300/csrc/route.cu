// Routing: which experts a token goes to, with which weights, and the gradient.
//
// A warp has a token; a lane has NV consecutive experts in registers. Choices are
// compared as unsigned integers in the order of the numbers that they stand for:
// 0 for an expert out of reach (logit or bias -inf), 1 for a NaN. Each of k rounds
// takes the largest key of the warp, the lowest index first; the outcome is looked over.
//
// The choice is what 64 bits say. Without a bias experts are compared by their
// logits, since both scores rise with them: exact. With one, or where a group's
// score is a sum, fp32 scores with a bound on their error decide wherever the gaps
// that matter are wider than it; the other tokens are done again in 64 bits.
//
// Bound by instructions, 500 to 1000 a token (memory would take 16384 x 256 fp32 2.6 us): 8 of
// 256 experts for 16384 tokens 11.9 us, with a bias 13.4, by groups of sums 18.3, the
// gradient 7 to 10; of 512 31, 43 and 44 (sixteen keys a lane, some of them spilled: 35 to 40
// with the registers of four blocks an SM instead of eight); one token 3 us, a launch.
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
// Of unsigned integers by exchanges too. __reduce_max_sync is one instruction, but as it is
// compiled here it has given a maximum of values that lanes no longer had (the last round's,
// once in 100000 tokens of up to 32 experts, on other tokens every time): it is used only
// where the outcome is looked over (8 % less time than by exchanges alone).
__device__ __forceinline__ uint32_t warp_max(uint32_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ uint32_t warp_min(uint32_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// e / size for e < 512: magic = ceil(2^20 / size); e size < 2^20.
__device__ __forceinline__ int over(int e, int magic) { return (e * magic) >> 20; }

// NV words of a lane to or from its run of a warp's.
template <int NV, typename E>
__device__ __forceinline__ void store_words(E* to, const E (&k)[NV]) {
    if constexpr (NV % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
            Pack<E, 4> v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v.v[j] = k[i + j];
            *reinterpret_cast<Pack<E, 4>*>(to + i) = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) to[i] = k[i];
    }
}
template <int NV, typename E>
__device__ __forceinline__ void load_words(E (&k)[NV], const E* from) {
    if constexpr (NV % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
            const Pack<E, 4> v = *reinterpret_cast<const Pack<E, 4>*>(from + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) k[i + j] = v.v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) k[i] = from[i];
    }
}

// A row's elements, NV to a lane; `other` past the last. VEC: a lane's are one vector or
// none; else they come as whole lines by way of buf, NV * 32 floats of the warp's own.
template <typename T, int NV, bool VEC>
__device__ __forceinline__ void load_row(float (&l)[NV], const T* row, int experts, float other, float* buf, const Bounds& bnd, int span) {
    const int lane = threadIdx.x & 31, e0 = lane * NV;
    if constexpr (VEC) {
        if (e0 < experts) {
            const Pack<T, NV> v = load_pack<T, NV>(row + e0, bnd, span);
#pragma unroll
            for (int i = 0; i < NV; ++i) l[i] = to_f32(v.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) l[i] = other;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = i * 32 + lane;
            l[i] = e < experts ? to_f32(load_one(row + e, bnd, span, from_f32<T>(0.0f))) : other;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NV; ++i) buf[i * 32 + lane] = l[i];
        __syncwarp();
        load_words<NV>(l, buf + e0);
        __syncwarp();
    }
}

// Terms of the chosen's shares, and their sum: s itself, or where they would underflow s
// over the largest of them. Lanes with `on` have a chosen expert's logit.
__device__ __forceinline__ float share_terms(bool sigmoid, bool on, float l, float& e) {
    float most = 0.0f;
    if (!sigmoid || !__any_sync(kAll, on && !(l < -64.0f))) {
        most = warp_max(on ? l : -INFINITY);
        if (most == -INFINITY) most = 0.0f;
    }
    e = 0.0f;
    if (on) {
        if (!sigmoid) {
            e = expf(l - most);
        } else if (most < 0.0f) {
            e = expf(l - most);                            // s = e^l to all of fp32's digits
        } else {
            const float a = expf(-fabsf(l));
            e = (l < 0.0f ? a : 1.0f) / (1.0f + a);
        }
    }
    return warp_sum(e);
}

// Lane j has the token's j-th expert and its logit, or -1: weights and experts.
template <bool SIGMOID>
__device__ __forceinline__ void put_weights(const RouteArgs& p, int64_t t, int mine, float lg, float top, float total, bool nan) {
    float w = 0.0f;
    if (p.renormalise) {
        const float all = share_terms(SIGMOID, mine >= 0, lg, w);
        w = mine >= 0 ? w / all * p.scale : 0.0f;
    } else if (mine >= 0) {
        w = (SIGMOID ? 1.0f / (1.0f + expf(-lg)) : expf(lg - top) / total) * p.scale;
    }
    if (nan && mine >= 0) w = __int_as_float(0x7fffffff);
    const int lane = threadIdx.x & 31;
    if (lane < p.k) {
        store_one(p.weights + t * p.k + lane, w, p.bnd, 2);
        store_one(p.chosen + t * p.k + lane, mine, p.bnd, 3);
    }
}

// ---------------------------------------------------------------- the choice
// Sorts a lane's keys, largest first (Batcher's odd-even merges).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int d = p; d >= 1; d /= 2)
#pragma unroll
            for (int j = d % p; j + d < N; j += 2 * d)
#pragma unroll
                for (int i = 0; i < d; ++i)
                    if (i + j + d < N && (i + j) / (2 * p) == (i + j + d) / (2 * p)) {
                        const uint32_t a = k[i + j], b = k[i + j + d];
                        k[i + j] = max(a, b);
                        k[i + j + d] = min(a, b);
                    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// A choice c = s + b is off by what its score is (`off` at most) and by its own rounding, 2^-24
// of it, whatever the other experts' biases are. c1 is greater than c2 in earnest where it
// seems so by more than this: c2's rounding is 2^-24 (|c1| + c1 - c2) at most.
__device__ __forceinline__ float wide_of(float c1, float off) { return 2.05f * fmaf(fabsf(c1), 0x1p-24f, off); }
// The least key that is not surely below one.
__device__ __forceinline__ uint32_t near_key(uint32_t key, float off) {
    const float v = value_of(key) - wide_of(value_of(key), off);
    return v == v ? key_of(v) : kNanKey + 1;
}
// Whether the choice with key k1 is not surely greater than the one with k2.
__device__ __forceinline__ bool close_keys(uint32_t k1, uint32_t k2, float off) {
    return !(value_of(k1) - value_of(k2) > wide_of(value_of(k1), off));
}

// By how much the choice with logit l1 and bias b1 is greater than the one with l2, b2, told
// by differences, which fp32 has to a share of themselves, and how far off that may be. With
// hi the greater logit and x = lo - hi, never positive,
//   s(hi) - s(lo) = s(hi) (1 - s(lo)) (1 - e^x) for a sigmoid, s(hi) (1 - e^x) for a softmax
// against b2 - b1. x's rounding moves 1 - e^x by 2^-24 of itself (x e^x / (1 - e^x) is 1 at
// most; for the lesser logit first it would go whole into the exponential). expf is within 2^-22
// of itself, which moves the sigmoid's factors by 1 - s(hi) and s(lo) of it, together by no more
// than all of it; expm1f is within 2^-23, and divisions, products and sums add 2^-24 each:
// 12 * 2^-24 for the sigmoid; for the softmax 9 * 2^-24, the 37 * 2^-24 of its total (below) and
// the rounding of hi - top. `off` has a third more, for the roundings of `by` and of itself;
// db's own is 2^-24 of it. What underflows or overflows on the way is below 2^-126.
template <bool SIGMOID>
__device__ __forceinline__ void add_difference(float l1, float b1, float l2, float b2, float top, float total, float& by, float& off) {
    const bool up = l1 < l2;
    const float hi = up ? l2 : l1, lo = up ? l1 : l2;
    const float gap = -expm1f(lo - hi) * (SIGMOID ? 1.0f / ((1.0f + expf(-hi)) * (1.0f + expf(lo))) : expf(hi - top) / total);
    const float ds = up ? -gap : gap, db = b2 - b1;
    by += ds - db;
    off += gap * (SIGMOID ? 0x1p-20f : fmaf(top - hi, 0x1.2p-24f, 0x1p-18f)) + fabsf(db) * 0x1p-22f + 0x1p-126f;
}
template <bool SIGMOID>
__device__ __forceinline__ bool surely_greater(float l1, float b1, float l2, float b2, float top, float total) {
    float by = 0.0f, off = 0.0f;
    add_difference<SIGMOID>(l1, b1, l2, b2, top, total, by, off);
    return by > off;
}

// The largest of keys[first .. first + size), the lowest place first; every lane gets both.
// It is taken out.
__device__ __forceinline__ int take_best(uint32_t* keys, int first, int size, uint32_t& best) {
    uint32_t mine = kUnreached;
    int at = 0x7fffffff;
#pragma unroll 1
    for (int e = first + static_cast<int>(threadIdx.x & 31); e < first + size; e += 32)
        if (keys[e] > mine) {
            mine = keys[e];
            at = e;
        }
    best = warp_max(mine);
    at = static_cast<int>(warp_min(mine == best ? static_cast<uint32_t>(at) : 0x7fffffffu));
    __syncwarp();
    if (best != kUnreached && (threadIdx.x & 31) == 0) keys[at] = kUnreached;
    __syncwarp();
    return at;
}
// Whether group a's score is surely greater than group z's, by the differences of their best
// experts, whom no other of their groups is near. Takes those out of keys.
template <typename T, bool SIGMOID>
__device__ __noinline__ bool surely_greater_group(const RouteArgs& p, const T* row, uint32_t* keys, int a, int z, float score_off, float top, float total) {
    const int size = p.experts / p.groups;
    float by = 0.0f, off = 0.0f;
    uint32_t ka = kUnreached, kz = kUnreached;
#pragma unroll 1
    for (int r = 0; r < p.group_best; ++r) {
        const int ea = take_best(keys, a * size, size, ka), ez = take_best(keys, z * size, size, kz);
        if (ka <= kNanKey || kz <= kNanKey) return false;
        add_difference<SIGMOID>(to_f32(load_one(row + ea, p.bnd, 0, from_f32<T>(0.0f))), p.bias != nullptr ? load_one(p.bias + ea, p.bnd, 1, 0.0f) : 0.0f,
                                to_f32(load_one(row + ez, p.bnd, 0, from_f32<T>(0.0f))), p.bias != nullptr ? load_one(p.bias + ez, p.bnd, 1, 0.0f) : 0.0f,
                                top, total, by, off);
    }
    if (p.bias != nullptr) {                               // without one the keys are the logits'
        uint32_t ra, rz;
        take_best(keys, a * size, size, ra);
        take_best(keys, z * size, size, rz);
        if ((ra > kNanKey && close_keys(ka, ra, score_off)) || (rz > kNanKey && close_keys(kz, rz, score_off))) return false;
    }
    return by > off;
}

// The k best of a token's keys, the lowest index first, without the sorted runs: lane j gets the
// j-th, its key, and all lanes the last one's key (kUnreached: fewer than k); `head` is the
// largest of the lane's own nv that stay out. list: k ints.
__device__ __noinline__ int choose_again(uint32_t* keys, int* list, int k, int nv, uint32_t& my_key, uint32_t& last, uint32_t& head) {
    const int lane = threadIdx.x & 31;
    my_key = kUnreached;
    __syncwarp();
    for (int r = 0; r < k; ++r) {
        const int at = take_best(keys, 0, nv * 32, last);
        if (last == kUnreached) break;
        if (lane == r) {
            my_key = last;
            list[r] = at;
        }
    }
    head = kUnreached;
    for (int i = 0; i < nv; ++i) head = max(head, keys[lane * nv + i]);
    __syncwarp();
    int mine = -1;
    if (my_key != kUnreached) {
        mine = list[lane];
        keys[mine] = my_key;
    }
    __syncwarp();
    return mine;
}

// ---------------------------------------------------------------- what fp32 leaves open
// Choices in 64 bits: -inf out of reach.
template <typename T, bool SIGMOID>
struct Choice64 {
    const RouteArgs& p;
    const T* row;
    double top, total;
    __device__ __forceinline__ float logit(int e) const { return to_f32(load_one(row + e, p.bnd, 0, from_f32<T>(0.0f))); }
    __device__ __forceinline__ float bias(int e) const { return p.bias != nullptr ? load_one(p.bias + e, p.bnd, 1, 0.0f) : 0.0f; }
    __device__ __forceinline__ double of(float l, float b) const {
        if (l == -INFINITY || b == -INFINITY) return -INFINITY;
        const double x = static_cast<double>(l), s = SIGMOID ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / total;
        return s + static_cast<double>(b);
    }
    __device__ void prepare(float most) {
        top = static_cast<double>(most);
        total = 1.0;
        if (!SIGMOID) {
            total = 0.0;
            for (int e = threadIdx.x & 31; e < p.experts; e += 32) total += exp(static_cast<double>(logit(e)) - top);
            total = warp_sum(total);
        }
    }
};
// The largest of a warp's values and the lowest place that has it.
__device__ __forceinline__ void best_of_warp(double& v, int& at) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const double v2 = __shfl_xor_sync(kAll, v, o);
        const int at2 = __shfl_xor_sync(kAll, at, o);
        if (v2 > v || (v2 == v && at2 < at)) {
            v = v2;
            at = at2;
        }
    }
}

// A token whose choice hangs on gaps within the bounds: one in 17000 of random ones, so the kernel ends
// with this call and keeps no register for it. keys: its experts' keys; sure: the
// groups that stay; open: those of which the best join them; top, total: its softmax's. A
// warp has few lanes for 64 bits (16 cycles an instruction): they see only the open groups, and
// of the experts those near the border, if differences do not tell those apart.
// list: 64 ints of shared memory.
template <typename T, bool SIGMOID>
__device__ __noinline__ void route_open(const RouteArgs& p, int64_t t, uint32_t* keys, int* list, float score_off, float top, float total, uint32_t sure,
                                        uint32_t open) {
    const int lane = threadIdx.x & 31, size = p.experts / p.groups;
    Choice64<T, SIGMOID> c64{p, static_cast<const T*>(p.logits) + t * p.sl};
    bool ready = false;
    uint32_t kept = sure;
    if (open != 0) {
        c64.prepare(top);
        ready = true;
        double mine = -INFINITY;                           // lane g: group g's score
        for (uint32_t left = open; left != 0; left &= left - 1) {
            const int g = __ffs(left) - 1;
            double best = -INFINITY, next = -INFINITY;
            for (int i = lane; i < size; i += 32) {
                const double c = c64.of(c64.logit(g * size + i), c64.bias(g * size + i));
                next = fmax(next, fmin(best, c));
                best = fmax(best, c);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const double b2 = __shfl_xor_sync(kAll, best, o), n2 = __shfl_xor_sync(kAll, next, o);
                next = fmax(fmin(best, b2), fmax(next, n2));
                best = fmax(best, b2);
            }
            if (lane == g) mine = p.group_best > 1 && next != -INFINITY ? best + next : best;
        }
        for (int need = p.kept - __popc(sure); need > 0; --need) {
            double v = mine;
            int at = lane;
            best_of_warp(v, at);
            if (v == -INFINITY) break;
            kept |= 1u << at;
            if (lane == at) mine = -INFINITY;
        }
        for (int e = lane; e < p.experts; e += 32)
            if (((kept >> (e / size & 31)) & 1u) == 0u) keys[e] = kUnreached;
        __syncwarp();
    }
    // the k best by keys, then whatever is near the last of them
    int count = 0, first = 0;                              // first: of those near
    uint32_t last = kUnreached;
    for (int r = 0; r < p.k; ++r) {
        uint32_t best = kUnreached;
        int at = 0x7fffffff;
        for (int e = lane; e < p.experts; e += 32)
            if (keys[e] > best) {
                best = keys[e];
                at = e;
            }
        const uint32_t most = warp_max(best);
        if (most == kUnreached) break;
        at = static_cast<int>(warp_min(best == most ? static_cast<uint32_t>(at) : 0x7fffffffu));
        __syncwarp();
        if (lane == 0) {
            keys[at] = kUnreached;
            list[r] = at;
        }
        __syncwarp();
        last = most;
        count = r + 1;
    }
    first = count;
    bool few = true;
    if (p.bias != nullptr && count == p.k && last > kNanKey) {
        const uint32_t least = near_key(last, score_off);
        for (int e0 = 0; e0 < p.experts && few; e0 += 32) {
            const bool near = e0 + lane < p.experts && keys[e0 + lane] >= least;
            const uint32_t all = __ballot_sync(kAll, near);
            few = count + __popc(all) <= 32;
            if (few && near) list[count + __popc(all & ((1u << lane) - 1u))] = e0 + lane;
            count += __popc(all);
        }
        __syncwarp();
    }
    int mine = -1;
    float lg = -INFINITY;
    if (few) {
        const int e = lane < count ? list[lane] : -1;
        const float l = e >= 0 ? c64.logit(e) : -INFINITY, b = e >= 0 ? c64.bias(e) : 0.0f;
        mine = lane < first ? e : -1;
        if (p.bias != nullptr) {                           // without one the keys are the logits'
            // the chosen against the one before, the others against the last chosen
            const int to = lane < first ? lane - 1 : first - 1;
            const float l1 = __shfl_sync(kAll, l, to & 31), b1 = __shfl_sync(kAll, b, to & 31);
            const bool told = lane == 0 || e < 0 || (l == l1 && b == b1) || surely_greater<SIGMOID>(l1, b1, l, b, top, total);
            if (!__all_sync(kAll, told)) {
                if (!ready) c64.prepare(top);
                const double c = e >= 0 ? c64.of(l, b) : -INFINITY;
                int rank = 0;
                for (int i = 0; i < count; ++i) {
                    const double c2 = __shfl_sync(kAll, c, i);
                    const int e2 = __shfl_sync(kAll, e, i);
                    rank += c2 > c || (c2 == c && e2 < e);
                }
                __syncwarp();
                if (e >= 0 && rank < p.k) list[32 + rank] = e;
                __syncwarp();
                mine = lane < first ? list[32 + lane] : -1;
            }
        }
    } else {
        // more than a warp's worth: every round in 64 bits, those that were taken by keys among them
        if (lane < first) keys[list[lane]] = last;
        __syncwarp();
        const uint32_t least = near_key(last, score_off);
        if (!ready) c64.prepare(top);
        for (int r = 0; r < p.k; ++r) {
            double v = -INFINITY;
            int at = 1 << 20;
            for (int e = lane; e < p.experts; e += 32)
                if (keys[e] >= least) {
                    const double c = c64.of(c64.logit(e), c64.bias(e));
                    if (c > v) {
                        v = c;
                        at = e;
                    }
                }
            best_of_warp(v, at);
            if (v == -INFINITY) break;
            if (lane == r) mine = at;
            if (lane == 0) keys[at] = kUnreached;
            __syncwarp();
        }
    }
    if (mine >= 0) lg = c64.logit(mine);
    put_weights<SIGMOID>(p, t, mine, lg, top, total, false);
}

// A token's k best take k rounds: the lanes' keys are sorted once, a round takes the
// largest of the lanes' next ones, the lowest lane first, and that lane goes on to its
// next. Which expert it was follows from the key and its place among the lane's, all
// rounds at once.
template <typename T, int NV, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kWarps * 32, 8) route_kernel(const __grid_constant__ RouteArgs p) {
    // a warp's keys as they are, and sorted, lane by lane, with a last 0
    __shared__ __align__(16) uint32_t s_keys[kWarps][NV * 32], s_sorted[kWarps][NV * 32 + 32];
    __shared__ int s_list[kWarps][64];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= p.m) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.sl;
    const bool grouped = p.kept < p.groups, sums = grouped && p.group_best > 1;
    const bool biased = p.bias != nullptr, scored = biased || sums;
    const bool whole = !SIGMOID && (scored || !p.renormalise);         // the softmax over all experts is needed
    const int size = p.experts / p.groups;
    const int magic = ((1 << 20) + size - 1) / size;
    const int e0 = lane * NV;
    auto in = [&](int i) { return VEC ? e0 < p.experts : e0 + i < p.experts; };

    float l[NV], b[NV];
    float* buf = reinterpret_cast<float*>(s_keys[warp]);
    load_row<T, NV, VEC>(l, row, p.experts, 0.0f, buf, p.bnd, 0);
    float odd = 0.0f;                                      // NaN if anything is not finite
#pragma unroll
    for (int i = 0; i < NV; ++i) odd = fmaf(l[i], 0.0f, odd);
    if (biased) {
        if (VEC && aligned_to(p.bias, 16)) load_row<float, NV, true>(b, p.bias, p.experts, 0.0f, buf, p.bnd, 1);
        else load_row<float, NV, false>(b, p.bias, p.experts, 0.0f, buf, p.bnd, 1);
#pragma unroll
        for (int i = 0; i < NV; ++i) odd = fmaf(b[i], 0.0f, odd);
    }
    const bool special = __any_sync(kAll, odd != 0.0f);

    float top = 0.0f, total = 1.0f, s[NV];
    if (SIGMOID) {
        if (scored) {
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] = rcp_fast(1.0f + exp2_fast(l[i] * -1.442695041f));      // e^x as 2^(x log2 e)
        }
    } else if (whole) {
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) top = fmaxf(top, in(i) ? l[i] : -INFINITY);
        top = warp_max(top);
        if (top == -INFINITY) top = 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            s[i] = exp2_fast((l[i] - top) * 1.442695041f);
            sum += in(i) ? s[i] : 0.0f;
        }
        total = warp_sum(sum);
        const float inv = 1.0f / total;
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] *= inv;
    }
    uint32_t key[NV];
    if (biased) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = key_of(s[i] + b[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = key_of(l[i]);
    }
    bool nan = false;
    if (special) {
#pragma unroll 1
        for (int i = 0; i < NV; ++i) {
            float li = l[0], bi = biased ? b[0] : 0.0f;
            uint32_t k = key[0];
#pragma unroll
            for (int j = 1; j < NV; ++j)
                if (j == i) {
                    li = l[j];
                    bi = biased ? b[j] : 0.0f;
                    k = key[j];
                }
            if (e0 + i < p.experts) nan |= li != li || bi != bi || (!SIGMOID && li == INFINITY);
            if (k > key_of(INFINITY) || k < key_of(-INFINITY)) k = kNanKey;            // a NaN of either sign
            if (li == -INFINITY || bi == -INFINITY) k = kUnreached;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j == i) key[j] = k;
        }
        nan = __any_sync(kAll, nan);
    }
    if (p.experts < NV * 32) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = in(i) ? key[i] : kUnreached;
    }
    // How far a score in fp32 may be off. 2^(x log2 e) is within 2^-22 + 1.5 |x| 2^-24 of e^x
    // (the approximation; the product and the constant in it): by that a sigmoid moves by
    // 0.29 * 2^-22 at most, the sum and the reciprocal add 2^-24 and 2^-23 of it: 1.04 * 2^-22
    // (measured over 2^30 logits in [-60, 60]: 0.49 * 2^-22). A
    // softmax's term at x below the largest is off by (2 + 1.13 x) 2^-23 exp(-x), 2^-22 at
    // most, its sum of up to 512 by 21 roundings and 2^-20 of itself, so s by 2^-18.5 of
    // the largest.
    const float score_off = SIGMOID ? 0x1.4p-22f : 0x1p-18f / total;

    if (grouped) {
        uint32_t best = 0, next = 0;
        const int lanes = size / NV;
        if (lanes * NV == size && (lanes & (lanes - 1)) == 0) {        // a group is a power of two of lanes
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint32_t v = sums && !biased && key[i] > kNanKey ? key_of(s[i]) : key[i];
                next = max(next, min(best, v));
                best = max(best, v);
            }
            for (int o = 1; o < lanes; o <<= 1) {
                const uint32_t b2 = __shfl_xor_sync(kAll, best, o), n2 = __shfl_xor_sync(kAll, next, o);
                next = max(min(best, b2), max(next, n2));
                best = max(best, b2);
            }
            best = __shfl_sync(kAll, best, (lane * lanes) & 31);
            next = __shfl_sync(kAll, next, (lane * lanes) & 31);
        } else {
            // through shared memory, `per` lanes to a group
            uint32_t* keys = s_keys[warp];
#pragma unroll
            for (int i = 0; i < NV; ++i) keys[e0 + i] = sums && !biased && key[i] > kNanKey ? key_of(s[i]) : key[i];
            __syncwarp();
            int per = 1;
            while (2 * per * p.groups <= 32) per *= 2;
            const int g = lane / per;
            if (g < p.groups)
                for (int i = lane & (per - 1); i < size; i += per) {
                    const uint32_t v = keys[g * size + i];
                    next = max(next, min(best, v));
                    best = max(best, v);
                }
            for (int o = 1; o < per; o <<= 1) {
                const uint32_t b2 = __shfl_xor_sync(kAll, best, o), n2 = __shfl_xor_sync(kAll, next, o);
                next = max(min(best, b2), max(next, n2));
                best = max(best, b2);
            }
            best = __shfl_sync(kAll, best, (lane * per) & 31);
            next = __shfl_sync(kAll, next, (lane * per) & 31);
            __syncwarp();
        }
        // lane g has group g's
        uint32_t group = lane < p.groups ? best : kUnreached;
        if (sums && lane < p.groups && next > kNanKey) group = key_of(value_of(best) + value_of(next));
        auto best_groups = [&](auto max_of) {
            uint32_t kept = 0;
            for (int r = 0; r < p.kept; ++r) {
                const uint32_t v = (kept >> lane) & 1u ? kUnreached : group;
                const uint32_t most = max_of(v);
                if (most == kUnreached) break;
                const uint32_t all = __ballot_sync(kAll, v == most);
                kept |= all & (0u - all);                  // the first of them
            }
            return kept;
        };
        uint32_t kept = 0;
        // (with scores a wrong group among them shows below: its bounds meet those of a better one that stays out)
        if (scored && !nan) kept = best_groups([](uint32_t v) { return __reduce_max_sync(kAll, v); });
        if (__popc(kept) != p.kept) kept = best_groups([](uint32_t v) { return warp_max(v); });
        if (scored && !nan) {
            // what a group's score may be: its choices' errors, its sum's rounding and that of the ends
            const bool in_reach = group > kNanKey, stays = ((kept >> lane) & 1u) != 0u;
            const float score = value_of(group);
            const float off = fmaf(fabsf(value_of(best)) + (sums && next > kNanKey ? fabsf(value_of(next)) : 0.0f), 0x1.8p-23f, 2.1f * score_off);
            const float low = score - off, high = score + off;
            const uint32_t least = low == low ? key_of(low) : kNanKey + 1, most = high == high ? key_of(high) : kAll;
            // the groups near the border between the best that stays out and the last that stays
            uint32_t last = __reduce_min_sync(kAll, stays ? least : kAll), out = kUnreached;
            if (__any_sync(kAll, stays ? least < last : in_reach && most >= last)) {
                out = warp_max(in_reach && !stays ? most : kUnreached);
                last = warp_min(stays ? least : kAll);
            }
            if (out >= last) {
                const bool above = stays && least > out, near = in_reach && !above && most >= last;
                const uint32_t sure = __ballot_sync(kAll, above), open = __ballot_sync(kAll, near);
                store_words<NV>(s_keys[warp] + e0, key);
                __syncwarp();
                const uint32_t kept_near = open & kept, out_near = open & ~kept;
                const bool told = __popc(kept_near) == 1 && __popc(out_near) == 1 &&
                                  surely_greater_group<T, SIGMOID>(p, row, s_keys[warp], __ffs(kept_near) - 1, __ffs(out_near) - 1, score_off, top, total);
                if (!told) {
                    __syncwarp();
                    store_words<NV>(s_keys[warp] + e0, key);
                    __syncwarp();
                    route_open<T, SIGMOID>(p, t, s_keys[warp], s_list[warp], score_off, top, total, sure, open);
                    return;
                }
                __syncwarp();
            }
        }
        if (lanes * NV == size) {                          // a lane's experts are of one group
            if (((kept >> (over(e0, magic) & 31)) & 1u) == 0u) {
#pragma unroll
                for (int i = 0; i < NV; ++i) key[i] = kUnreached;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (((kept >> (over(e0 + i, magic) & 31)) & 1u) == 0u) key[i] = kUnreached;
        }
    }

    uint32_t* keys = s_keys[warp];
    uint32_t* sorted = s_sorted[warp];
    store_words<NV>(keys + e0, key);
    sort_keys<NV>(key);
#pragma unroll
    for (int i = 1; i < NV; ++i) sorted[i * 32 + lane] = key[i];
    sorted[NV * 32 + lane] = kUnreached;
    __syncwarp();
    uint32_t head = key[0], my_key = kUnreached, last = kUnreached;
    int place = lane;                                      // of the lane's next key in `sorted`
    int* places = s_list[warp];                            // of the choices
    const uint32_t below = (1u << lane) - 1u;
    for (int r = 0; r < p.k; ++r) {
        last = __reduce_max_sync(kAll, head);
        if (last == kUnreached) break;
        const bool has = head == last;
        const uint32_t all = __ballot_sync(kAll, has);
        if (lane == r) my_key = last;
        if (has && (all & below) == 0) {                   // the first of them
            places[r] = place;
            place += 32;
            head = sorted[place];
        }
    }
    __syncwarp();
    int mine = -1;                                         // lane j: the j-th choice
    if (my_key != kUnreached) {
        // the (place - greater ones)-th of its lane's experts with that key
        const int my_place = places[lane], first = (my_place & 31) * NV;
        int skip = my_place >> 5;
        uint32_t of[NV];
        load_words<NV>(of, keys + first);
#pragma unroll
        for (int i = 0; i < NV; ++i) skip -= of[i] > my_key;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (of[i] == my_key && skip-- == 0) mine = first + i;
    }
    // looked over: every choice is an expert's, behind the one before, and before all that stay out
    uint32_t key2 = __shfl_down_sync(kAll, my_key, 1);
    const int mine2 = __shfl_down_sync(kAll, mine, 1), mine_last = __shfl_sync(kAll, mine, p.k - 1);
    bool wrong = my_key != kUnreached && mine < 0;
    wrong |= lane < p.k - 1 && key2 != kUnreached && !(my_key > key2 || (my_key == key2 && mine < mine2));
    wrong |= head > last || (head == last && last != kUnreached && e0 + NV <= mine_last);
    if (__any_sync(kAll, wrong)) {
        uint32_t k1, k2, k3;
        mine = choose_again(keys, places, p.k, NV, k1, k2, k3);
        my_key = k1;
        last = k2;
        head = k3;
        key2 = __shfl_down_sync(kAll, my_key, 1);
    }
    float lg = mine >= 0 ? to_f32(load_one(row + mine, p.bnd, 0, from_f32<T>(0.0f))) : -INFINITY;
    if (biased && !nan) {
        // gaps between choices next to one another, and from the last to what stays out
        const bool ahead = lane < p.k - 1 && key2 > kNanKey && close_keys(my_key, key2, score_off);
        const uint32_t least = near_key(last, score_off);
        const bool near = last > kNanKey && head >= least;
        if (__any_sync(kAll, ahead || near)) {
            // the same logit and bias are a tie in any precision; others by their differences
            const float b1 = mine >= 0 ? load_one(p.bias + mine, p.bnd, 1, 0.0f) : 0.0f;
            const float lg2 = __shfl_down_sync(kAll, lg, 1), b2 = __shfl_down_sync(kAll, b1, 1);
            const float llast = __shfl_sync(kAll, lg, p.k - 1), blast = __shfl_sync(kAll, b1, p.k - 1);
            // my own next in line, then my lane's experts that stay out against the last choice
            float l1 = lg, bb1 = b1, l2 = lg2, bb2 = b2;
            bool ask = ahead, unsure = false;
#pragma unroll 1
            for (int i = -1; i < (near ? NV : 0); ++i) {
                if (i >= 0) {
                    const int e = e0 + i;
                    ask = keys[e] >= least && keys[e] <= last;
                    if (!ask) continue;
                    l1 = llast;
                    bb1 = blast;
                    l2 = to_f32(load_one(row + e, p.bnd, 0, from_f32<T>(0.0f)));
                    bb2 = load_one(p.bias + e, p.bnd, 1, 0.0f);
                }
                if (ask && (l1 != l2 || bb1 != bb2)) unsure |= !surely_greater<SIGMOID>(l1, bb1, l2, bb2, top, total);
            }
            if (__any_sync(kAll, unsure)) {
                __syncwarp();
                route_open<T, SIGMOID>(p, t, keys, s_list[warp], score_off, top, total, kAll, 0u);
                return;
            }
        }
    }
    put_weights<SIGMOID>(p, t, mine, lg, top, total, nan);
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
    __shared__ __align__(16) float s_row[kWarps][NV * 32];
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
        load_row<T, NV, VEC>(l, row, p.experts, -INFINITY, s_row[warp], p.bnd, 1);
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
        float q;
        const float all = share_terms(p.sigmoid, e >= 0, lg, q);
        q = all == 0.0f ? 0.0f : q / all;
        float rest = 1.0f;                                 // 1 - s
        if (p.sigmoid) {
            const float a = expf(-fabsf(lg));
            rest = (lg < 0.0f ? 1.0f : a) / (1.0f + a);
        }
        mean = warp_sum(e >= 0 ? q * g : 0.0f);
        if (e >= 0) v = q * rest * (g - mean);
    } else if (p.sigmoid) {
        const float a = expf(-fabsf(lg)), one = 1.0f / (1.0f + a);
        if (e >= 0) v = g * a * one * one;                 // s (1 - s)
    } else {
        v = g;
        mean = warp_sum(e >= 0 ? g * (expf(lg - base) / total) : 0.0f);
    }
    float d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = 0.0f;
    store_words<NV>(s_row[warp] + lane * NV, d);
    __syncwarp();
    for (int j = 0; j < p.k; ++j) {
        if (lane == j && e >= 0) s_row[warp][e] += v;
        __syncwarp();
    }
    T* out = static_cast<T*>(p.dlogits) + t * p.sd;
    load_words<NV>(d, s_row[warp] + lane * NV);
    if (dense) {
        const float inv = 1.0f / total;
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = l[i] * inv * (d[i] - mean);
    }
    if constexpr (VEC) {
        if (lane * NV < p.experts) {
            Pack<T, NV> o;
#pragma unroll
            for (int i = 0; i < NV; ++i) o.v[i] = from_f32<T>(d[i]);
            store_pack<T, NV>(out + lane * NV, o, p.bnd, 3);
        }
    } else {                                               // as whole lines
        __syncwarp();
        store_words<NV>(s_row[warp] + lane * NV, d);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * 32 + lane < p.experts) store_one(out + i * 32 + lane, from_f32<T>(s_row[warp][i * 32 + lane]), p.bnd, 3);
    }
}

unsigned blocks(int64_t m) { return static_cast<unsigned>((m + kWarps - 1) / kWarps); }

// Lanes of NV elements whose loads are whole.
bool vec_rows(const void* p, int64_t es, int64_t stride, int64_t m, int experts, int nv) {
    const int64_t bytes = es * nv < 16 ? es * nv : 16;
    return experts % nv == 0 && rows_aligned(p, es, stride, m, bytes);
}

template <typename T, int NV, bool SIGMOID>
cudaError_t route_s(const RouteArgs& a, cudaStream_t st) {
    if (vec_rows(a.logits, sizeof(T), a.sl, a.m, a.experts, NV))
        return launch_after(route_kernel<T, NV, true, SIGMOID>, dim3(blocks(a.m)), kWarps * 32, 0, st, a);
    return launch_after(route_kernel<T, NV, false, SIGMOID>, dim3(blocks(a.m)), kWarps * 32, 0, st, a);
}
template <typename T, int NV>
cudaError_t route_nv(const RouteArgs& a, cudaStream_t st) {
    return a.sigmoid ? route_s<T, NV, true>(a, st) : route_s<T, NV, false>(a, st);
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
