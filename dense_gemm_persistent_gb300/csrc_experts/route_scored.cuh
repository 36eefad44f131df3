// route_scored.cuh -- dgemm_route_scored: the experts of one token by scores, a balance
// bias and groups. Part of route.cu, whose kernels group the chosen pairs.
//
// Per token, by one warp (lane l holds the VPL experts from l * VPL on):
//     s = sigmoid(x) or softmax(x),  c = s + bias
//     worth of a group = max c, or the sum of its two largest c
//     chosen: the k largest c of the groups_kept groups of most worth
//     weight = s / sum s (over the chosen) * scale
// The order decides integers, so it has to be that of the values, not of their FP32 roundings.
// The FP32 pass knows its error (Margin): where two values that decide are nearer than
// that and not the same by their inputs, the token is done again in FP64 -- only its k + 1
// best experts where just their order is open, else all of them. Without a bias and without
// sums the logits' order is the values', and nothing has to be told apart.
// That the pass knows its error also makes it cheap: a lane's keys give up their last bits for the
// expert's place in the lane, so that they differ, are sorted once, and a round of the selection
// looks at the first and moves the winner's up.
// FP64 is slow on this chip (two fused multiply-adds a clock and SM, long latency), and one token that waits for it holds
// up the call: 16001 tokens took 60 us while some 3 of them did all of their 256 experts in FP64,
// with an average SM busy for 25. Hence the shorter ways: a border between two groups needs their
// two best experts each, an open order the chosen ones.
#pragma once

namespace {

struct ScoredParams : RouteParams {
    const float* bias;          // [E], or null
    int softmax, groups, per_group, kept, top2;
    int lanes_per_group;        // a group is this many whole lanes (a power of two), or 0
    int by_logit;               // the logits' order is the choice values'
    float scale;
};

constexpr unsigned kAll = 0xffffffffu;
constexpr unsigned kNone = 0x007fffffu;   // ordered(-infinity): what must not be chosen; every number is above it

// How far an FP32 score is off, in units of the largest there can be (sigmoid 1, softmax 1 / its sum), so that a value far
// down the list is covered too. Sigmoid: s (1 - s) of exp's relative error (2^-22, and |x| 2^-23.5 for its
// rounded argument: 8e-8 in all), and 2 ulp of the quotient. Softmax: exp the same way, and a sum of up to 1024
// terms, 37 deep. kTiny: scores that underflow. kSum: relative error of an addition.
struct Margin {
    static constexpr float kSigmoid = 6e-7f, kSoftmax = 4e-6f, kTiny = 1e-37f, kSum = 6.1e-8f;
};

__device__ __forceinline__ float logit_at(const RouteParams& p, int t, int e) {
    const int64_t at = static_cast<int64_t>(t) * p.E + e;
    const float x = p.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at])
                           : static_cast<const float*>(p.logits)[at];
    return x > -INFINITY ? fminf(x, FLT_MAX) : -INFINITY;            // (NaN too)
}
__device__ __forceinline__ float bias_at(const ScoredParams& p, int e) {
    const float b = p.bias ? __ldg(p.bias + e) : 0.0f;
    return b > -INFINITY ? fminf(b, FLT_MAX) : -INFINITY;
}

__device__ __forceinline__ unsigned long long ordered64(double x) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered64(unsigned long long o) {
    return __longlong_as_double(static_cast<long long>((o >> 63) ? (o & 0x7FFFFFFFFFFFFFFFull) : ~o));
}
// e^y in FP64, straight-line so that several run side by side: y = n ln 2 + r with ln 2 = 355/512 + a rest, whose first
// product is exact (Cody and Waite), e^r by its Taylor series to r^13 (the next term is 4e-18). y is cut
// off at +-708: e^y stays a normal number.
__device__ __forceinline__ double exp64(double y) {
    y = fmin(fmax(y, -708.0), 708.0);
    const double n = rint(y * 1.4426950408889634);
    const double r = fma(n, 0.00021219444005469057, fma(n, -355.0 / 512.0, y));
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __longlong_as_double(__double_as_longlong(p) + (static_cast<long long>(n) << 52));
}
// 1 / d for d >= 1, up to e^709: Newton's iteration on the significand, from the FP32 quotient (2^-23, 2^-46, 2^-92).
__device__ __forceinline__ double inverse64(double d) {
    const long long bits = __double_as_longlong(d), exponent = (bits >> 52) - 1023;
    const double m = __longlong_as_double(bits - (exponent << 52));                  // in [1, 2)
    double q = static_cast<double>(1.0f / static_cast<float>(m));
    q = fma(q, fma(-m, q, 1.0), q);
    q = fma(q, fma(-m, q, 1.0), q);
    return __longlong_as_double(__double_as_longlong(q) - (exponent << 52));
}
__device__ __forceinline__ double sigmoid64(float x) { return inverse64(1.0 + exp64(-static_cast<double>(x))); }

// e^x and 1 / x by the special function unit (2^-22 relative beside the argument's rounding, 1 ulp; small numbers are 0).
__device__ __forceinline__ float exp_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}
__device__ __forceinline__ float inverse_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Top two of the union of (a1 >= a2) and (b1 >= b2), into a.
template <class T>
__device__ __forceinline__ void merge_two(T& a1, T& a2, T b1, T b2) {
    a2 = max(min(a1, b1), max(a2, b2));
    a1 = max(a1, b1);
}

// Bit g: group g is kept. Lane g (below G) holds the order-preserving worth of group g, kNone where nothing may be chosen.
// in, out: the groups at the border, the last one kept and the first one not; before: the worth of the last but one kept.
struct Border {
    unsigned kept, left;                // groups kept; of this lane: its worth while its group is neither kept nor `out`
    unsigned in, out;                   // one bit each, 0: none
    unsigned worth_in, worth_out, before;
};
__device__ __forceinline__ Border keep_groups(const ScoredParams& p, unsigned worth) {
    const unsigned me = 1u << (threadIdx.x & 31);
    Border b{0, 0, 0, 0, kNone, kNone, kAll};
    auto best = [&](unsigned& m) {
        m = __reduce_max_sync(kAll, worth);
        unsigned who = __ballot_sync(kAll, worth == m);
        who &= 0u - who;                // (the lowest)
        if (who == me) worth = kNone;
        return m > kNone ? who : 0u;
    };
    for (int r = 0; r < p.kept; ++r) {
        unsigned m;
        const unsigned g = best(m);
        if (!g) break;
        b.kept |= g;
        b.in = g;
        if (r > 0) b.before = b.worth_in;
        b.worth_in = m;
    }
    b.out = best(b.worth_out);
    b.left = worth;
    return b;
}

// The sum of a row's softmax in FP64, and its largest logit.
template <int VPL>
__device__ __noinline__ double softmax_sum64(const ScoredParams& p, int t, int lane, float xmax) {
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        const float x = e < p.E && bias_at(p, e) > -INFINITY ? logit_at(p, t, e) : -INFINITY;
        const double v = exp64(static_cast<double>(fmaxf(x, -FLT_MAX)) - xmax);
        total += x > -INFINITY ? v : 0.0;
    }
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    return total;
}

// An expert's choice value in FP64; inv: one over the row's softmax_sum64.
__device__ __forceinline__ double choice64(const ScoredParams& p, int t, int e, float xmax, double inv) {
    const float x = logit_at(p, t, e);
    const double s = p.softmax ? exp64(static_cast<double>(x) - xmax) * inv : sigmoid64(x);
    return s + bias_at(p, e);
}

// The whole token in FP64: lane j keeps the j-th choice.
template <int VPL>
__device__ __noinline__ int choose64(const ScoredParams& p, int t, int lane, float xmax, double inv) {
    unsigned long long key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        const bool may = e < p.E && logit_at(p, t, min(e, p.E - 1)) > -INFINITY && bias_at(p, min(e, p.E - 1)) > -INFINITY;
        const double c = choice64(p, t, min(e, p.E - 1), xmax, inv);
        key[i] = may ? ordered64(c + 0.0) : 0;
    }
    if (p.groups > 1) {
        unsigned long long worth = 0;
        for (int g = 0; g < p.groups; ++g) {
            unsigned long long m1 = 0, m2 = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (static_cast<unsigned>(lane * VPL + i - g * p.per_group) < static_cast<unsigned>(p.per_group))
                    merge_two(m1, m2, key[i], 0ull);
            for (int o = 16; o > 0; o >>= 1)
                merge_two(m1, m2, __shfl_xor_sync(kAll, m1, o), __shfl_xor_sync(kAll, m2, o));
            if (lane == g) worth = p.top2 && m2 != 0 ? ordered64(unordered64(m1) + unordered64(m2) + 0.0) : m1;
        }
        int better = 0;
        for (int g = 0; g < p.groups; ++g) {
            const unsigned long long o = __shfl_sync(kAll, worth, g);
            better += o > worth || (o == worth && g < lane);
        }
        const unsigned kept = __ballot_sync(kAll, worth != 0 && better < p.kept);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (!((kept >> min((lane * VPL + i) / p.per_group, 31)) & 1)) key[i] = 0;
    }
    int my_id = -1;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long best = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
        unsigned long long m = best;
        for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
        if (m == 0) break;
        const int src = __ffs(__ballot_sync(kAll, best == m)) - 1;     // lanes in the experts' order: the lowest
        int at = 0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool hit = key[i] == m && !found;
            at = hit ? i : at;
            if (hit && lane == src) key[i] = 0;
            found = found || hit;
        }
        const int e = __shfl_sync(kAll, lane * VPL + at, src);
        my_id = lane == j ? e : my_id;
    }
    return my_id;
}

// The first `count` lanes hold the best experts, whose order alone is open; lane j < n gets the j-th of them.
__device__ __noinline__ int order64(const ScoredParams& p, int t, int id, int count, int n, int lane, float xmax, double inv) {
    const unsigned long long key = lane < count ? ordered64(choice64(p, t, id, xmax, inv) + 0.0) : 0;
    int place = 0;
    for (int j = 0; j < count; ++j) {
        const unsigned long long o = __shfl_sync(kAll, key, j);
        const int other = __shfl_sync(kAll, id, j);
        place += o > key || (o == key && other < id);
    }
    int mine = -1;
    for (int j = 0; j < count; ++j) {
        const int at = __shfl_sync(kAll, place, j), other = __shfl_sync(kAll, id, j);
        mine = at == lane && lane < n ? other : mine;
    }
    return mine;
}

// Which of two groups a and b is worth more, by its two best experts in lanes 0, 1 and 2, 3 (id < 0: it has no second).
__device__ __noinline__ bool second_group64(const ScoredParams& p, int t, int id, int lane, int a, int b, float xmax, double inv) {
    const double c = lane < 4 && id >= 0 ? choice64(p, t, id, xmax, inv) : 0.0;
    const double sum = c + __shfl_down_sync(kAll, c, 1);
    const double wa = __shfl_sync(kAll, sum, 0), wb = __shfl_sync(kAll, sum, 2);
    return wb > wa || (wb == wa && b < a);
}

// One key a lane's expert, up to kNone: not to be chosen. BY_LOGIT: the logit (BF16: its 16 bits over the complement of the expert,
// so that keys differ); else the choice value, whose last bits are the complement of the expert's place in the lane.
template <int VPL, bool BF16, bool BY_LOGIT>
struct Selection {
    static constexpr bool UNIQUE = !BY_LOGIT || BF16;       // a lane's keys differ
    static constexpr bool SORTED = UNIQUE && VPL <= 8;
    static constexpr unsigned PLACE = BY_LOGIT ? 0u : VPL - 1;
    unsigned key[VPL];

    __device__ __forceinline__ void start(int lane) {
        if constexpr (BY_LOGIT && BF16) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (key[i] > kNone) key[i] = (key[i] & 0xFFFF0000u) | (0xFFFFu - static_cast<unsigned>(lane * VPL + i));
        } else if constexpr (!BY_LOGIT) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                key[i] = (key[i] & ~PLACE) | (PLACE - i);
        }
        if constexpr (SORTED) {     // odd-even merge sort, largest first
#pragma unroll
            for (int p2 = 1; p2 < VPL; p2 *= 2)
#pragma unroll
                for (int d = p2; d >= 1; d /= 2)
#pragma unroll
                    for (int j = d % p2; j + d < VPL; j += 2 * d)
#pragma unroll
                        for (int i = 0; i < d; ++i)
                            if (i + j + d < VPL && (i + j) / (2 * p2) == (i + j + d) / (2 * p2)) {
                                const unsigned hi = max(key[i + j], key[i + j + d]), lo = min(key[i + j], key[i + j + d]);
                                key[i + j] = hi;
                                key[i + j + d] = lo;
                            }
        }
    }
    // Takes the largest: its key without the place (up to kNone: nothing is left); the lane that had it writes it and its
    // expert to `to`. Lanes are in the experts'
    // order, so of equal keys the first lane's is the lowest expert's.
    __device__ __forceinline__ unsigned take(int lane, uint2* to) {
        unsigned best = key[0];
        if constexpr (!SORTED) {
#pragma unroll
            for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
        }
        const unsigned m = __reduce_max_sync(kAll, best & ~PLACE);
        const unsigned who = __ballot_sync(kAll, (best & ~PLACE) == m);
        const bool won = (who & ((2u << lane) - 1)) == 1u << lane;         // (the first of them)
        if constexpr (SORTED) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = won ? (i + 1 < VPL ? key[i + 1] : 0) : key[i];
        } else if constexpr (UNIQUE) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = won && key[i] == best ? 0 : key[i];
        }
        unsigned e;
        if constexpr (BY_LOGIT && BF16) {
            e = 0xFFFFu - (m & 0xFFFFu);
        } else if constexpr (!BY_LOGIT) {
            e = lane * VPL + (PLACE - (best & PLACE));
        } else {
            int at = 0;
            bool found = !won;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const bool hit = key[i] == m && !found;
                at = hit ? i : at;
                key[i] = hit ? 0 : key[i];
                found = found || hit;
            }
            e = lane * VPL + at;
        }
        if (won) *to = make_uint2(m, e);
        return m;
    }
};

template <int VPL, bool BF16, bool BY_LOGIT>
__device__ __forceinline__ void route_scored_token(const ScoredParams& p, int t, int lane, const float* bias, uint2* won, int* sid) {
    // logits (masked: -inf or NaN)
    float x[VPL];
    {
        const int64_t at = static_cast<int64_t>(t) * p.E + lane * VPL;
        constexpr int BYTES = VPL * (BF16 ? 2 : 4), WORDS = (BYTES + 3) / 4, VEC = BYTES < 16 ? BYTES : 16;
        const char* src = static_cast<const char*>(p.logits) + at * (BF16 ? 2 : 4);
        if (p.E % VPL == 0) {      // (whole lanes: every lane's experts start on a vector)
            uint32_t w[WORDS];
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = 0xFFFFFFFFu;                // NaN
            if (lane * VPL < p.E) {
                if constexpr (VEC == 16) {
#pragma unroll
                    for (int i = 0; i < WORDS; i += 4) {
                        const uint4 v = *reinterpret_cast<const uint4*>(src + 4 * i);
                        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
                    }
                } else if constexpr (VEC == 8) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    w[0] = v.x, w[1] = v.y;
                } else {
                    w[0] = *reinterpret_cast<const uint32_t*>(src);
                }
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                x[i] = BF16 ? __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16) : __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                x[i] = lane * VPL + i >= p.E ? -INFINITY
                       : BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src)[i])
                              : reinterpret_cast<const float*>(src)[i];
        }
    }
    float b[VPL];
    if constexpr (!BY_LOGIT) {
#pragma unroll
        for (int i = 0; i < VPL; i += 2) {
            const float2 v = *reinterpret_cast<const float2*>(bias + lane * VPL + i);
            b[i] = v.x, b[i + 1] = v.y;
        }
    }
    Selection<VPL, BF16, BY_LOGIT> pick;
    float xmax = 0.0f, inv_total = 1.0f;
    if (p.softmax) {
        unsigned m = kNone;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            x[i] = x[i] > -INFINITY && (BY_LOGIT || b[i] > -INFINITY) ? fminf(x[i], FLT_MAX) : -INFINITY;
            m = max(m, ordered(x[i]));
        }
        m = __reduce_max_sync(kAll, m);
        xmax = m > kNone ? unordered(m) : 0.0f;
        if (!BY_LOGIT || !p.renorm) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) sum += exp_fast(x[i] - xmax);
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            inv_total = 1.0f / sum;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if constexpr (BY_LOGIT) {
            pick.key[i] = x[i] > -INFINITY ? ordered(fminf(x[i], FLT_MAX) + 0.0f) : kNone;
        } else {
            const float s = p.softmax ? exp_fast(x[i] - xmax) * inv_total : inverse_fast(1.0f + exp_fast(-x[i]));
            // (a bias of -infinity stands for one that is NaN too)
            pick.key[i] = ordered((x[i] > -INFINITY ? s : -INFINITY) + b[i] + 0.0f);
        }
    }
    // twice the most that a score is off
    const float off = 2.0f * (p.softmax ? Margin::kSoftmax * inv_total : Margin::kSigmoid) + Margin::kTiny;
    bool whole = false;           // the token has to be done in FP64 altogether
    auto inverse_sum = [&]() { return p.softmax ? 1.0 / softmax_sum64<VPL>(p, t, lane, xmax) : 0.0; };
    if (p.groups > 1) {
        unsigned m1 = kNone, m2 = kNone;
        if (p.lanes_per_group) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) merge_two(m1, m2, pick.key[i], kNone);
            for (int o = 1; o < p.lanes_per_group; o <<= 1)
                merge_two(m1, m2, __shfl_xor_sync(kAll, m1, o), __shfl_xor_sync(kAll, m2, o));
            const int first = min(lane * p.lanes_per_group, 31);
            m1 = __shfl_sync(kAll, m1, first);
            m2 = __shfl_sync(kAll, m2, first);
        } else {
            for (int g = 0; g < p.groups; ++g) {
                unsigned a1 = kNone, a2 = kNone;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    merge_two(a1, a2, static_cast<unsigned>(lane * VPL + i - g * p.per_group) <
                                              static_cast<unsigned>(p.per_group) ? pick.key[i] : kNone, kNone);
                for (int o = 16; o > 0; o >>= 1)
                    merge_two(a1, a2, __shfl_xor_sync(kAll, a1, o), __shfl_xor_sync(kAll, a2, o));
                if (lane == g) m1 = a1, m2 = a2;
            }
        }
        if (lane >= p.groups) m1 = m2 = kNone;
        // (two finite numbers: a sum below FP32's range is the lowest there is, not kNone; the margin then sends it to FP64)
        const unsigned worth = p.top2 && m2 > kNone ? ordered(fmaxf(unordered(m1) + unordered(m2), -FLT_MAX) + 0.0f) : m1;
        const Border at = keep_groups(p, worth);
        unsigned kept = at.kept;
        if (!BY_LOGIT && at.out) {
            // (the values that were added may be larger than their sum)
            float size = 0.0f;
            if (m1 > kNone) size = fabsf(unordered(m1)) + (m2 > kNone ? fabsf(unordered(m2)) : 0.0f);
            size = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size)));
            const float margin = 2.0f * off + 4.0f * Margin::kSum * size;
            auto near = [&](unsigned a, unsigned b) { return b > kNone && !(unordered(a) - unordered(b) > margin); };      // (inf - inf too)
            if (near(at.worth_in, at.worth_out)) {
                // one border between two groups, and no third expert that might be one of a group's two best?
                whole = (at.before != kAll && near(at.before, at.worth_out)) || near(at.worth_in, __reduce_max_sync(kAll, at.left));
                int id = -1;
                for (int r = 0; r < 2 && !whole; ++r) {
                    const int g = __ffs(r ? at.out : at.in) - 1;
                    unsigned second = kNone;
                    int found[2] = {-1, -1};        // this lane's experts of the group that are taken
                    for (int n = 0; n < 3; ++n) {
                        unsigned best = kNone;
                        int best_e = -1;
#pragma unroll
                        for (int i = 0; i < VPL; ++i) {
                            const int e = lane * VPL + i;
                            const bool in = static_cast<unsigned>(e - g * p.per_group) < static_cast<unsigned>(p.per_group);
                            if (in && e != found[0] && e != found[1] && pick.key[i] > best) best = pick.key[i], best_e = e;
                        }
                        const unsigned m = __reduce_max_sync(kAll, best);
                        if (n == (p.top2 ? 2 : 1)) {
                            whole = whole || near(second, m);
                            break;
                        }
                        second = m;
                        if (m <= kNone) break;
                        const int e = __shfl_sync(kAll, best_e, __ffs(__ballot_sync(kAll, best == m)) - 1);
                        found[n] = e;
                        if (lane == 2 * r + n) id = e;
                    }
                }
                if (!whole && second_group64(p, t, id, lane, __ffs(at.in), __ffs(at.out), xmax, inverse_sum())) kept ^= at.in | at.out;
            }
        }
        if (p.lanes_per_group) {
            const bool keep = (kept >> min(lane / p.lanes_per_group, 31)) & 1;
#pragma unroll
            for (int i = 0; i < VPL; ++i) pick.key[i] = keep ? pick.key[i] : kNone;
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (!((kept >> min((lane * VPL + i) / p.per_group, 31)) & 1)) pick.key[i] = kNone;
        }
    }
    // the k largest, and where FP32 values decide the two behind them
    int n = 0;
    pick.start(lane);
    while (n < p.k && pick.take(lane, won + n) > kNone) ++n;
    __syncwarp();
    const uint2 mine = lane < n ? won[lane] : make_uint2(kNone, 0xFFFFFFFFu);
    const unsigned my_key = mine.x;
    int my_id = static_cast<int>(mine.y);
    __syncwarp();
    float xj = lane < n ? logit_at(p, t, my_id) : 0.0f;
    if constexpr (!BY_LOGIT) {
        unsigned behind = kNone;
        int behind_id = -1;
        if (n == p.k) {
            behind = pick.take(lane, won);
            __syncwarp();
            behind_id = static_cast<int>(won->y);
        }
        // The border's neighbours by their keys, which are short of up to VPL units in the last place.
        auto near = [&](unsigned k1, unsigned k2) {
            const float c1 = unordered(k1), c2 = unordered(k2);
            return k2 > kNone && c1 - c2 <= off + (Margin::kSum * (1 + 2 * VPL)) * (fabsf(c1) + fabsf(c2));
        };
        unsigned next_key = __shfl_down_sync(kAll, my_key, 1);
        if (lane == n - 1) next_key = behind;
        const bool tight = lane < n && near(my_key, next_key);
        if (whole) {
            my_id = choose64<VPL>(p, t, lane, xmax, inverse_sum());
            xj = my_id >= 0 ? logit_at(p, t, my_id) : 0.0f;
        } else if (__any_sync(kAll, tight)) {
            // the same by their inputs? Then they are equal, and in order
            const bool more = behind > kNone;
            const float bj = lane < n ? bias_at(p, my_id) : 0.0f, xe = more ? logit_at(p, t, behind_id) : 0.0f;
            const float be = more ? bias_at(p, behind_id) : 0.0f;
            float xn = __shfl_down_sync(kAll, xj, 1), bn = __shfl_down_sync(kAll, bj, 1);
            int next_id = __shfl_down_sync(kAll, my_id, 1);
            if (lane == n - 1) xn = xe, bn = be, next_id = behind_id;
            const bool open = __any_sync(kAll, tight && !(xj == xn && bj == bn && my_id < next_id));
            // Who else may be among the first k? What is near the last of them: what is not lies below all of them.
            const unsigned last = __shfl_sync(kAll, my_key, n - 1);
            const bool one = near(last, behind);
            bool several = false, all = open && one && n >= 32;
            if (one) {
                __syncwarp();
                several = near(last, pick.take(lane, won));
                __syncwarp();
            }
            if (several && !open) {       // in order as they are if all of them are the last one's equals
                const float xl = __shfl_sync(kAll, xj, n - 1), bl = __shfl_sync(kAll, bj, n - 1);
                auto differs = [&](int e) { return !(logit_at(p, t, e) == xl && bias_at(p, e) == bl); };
                bool other = differs(static_cast<int>(won->y));
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (near(last, pick.key[i])) other = other || differs(lane * VPL + (pick.PLACE - (pick.key[i] & pick.PLACE)));
                all = __any_sync(kAll, other);
            }
            if (all || open) {
                const double inv = inverse_sum();
                if (all || several) my_id = choose64<VPL>(p, t, lane, xmax, inv);
                else my_id = order64(p, t, lane == n && one ? behind_id : my_id, one ? n + 1 : n, n, lane, xmax, inv);
                xj = my_id >= 0 ? logit_at(p, t, my_id) : 0.0f;
            }
        }
    }
    // The weights are made of expf (2 ulp) and __fdividef (2 ulp up to 2^126, beyond it 0; full quotients: 16001 tokens of 256 experts
    // 34.3 us, not 33.5), but for the softmax's sum over the row without renormalize: that is the selection's, of special-function
    // exponentials, off by up to (VPL + 20) 2^-24.
    const bool chosen = my_id >= 0;
    float w = 0.0f, least = FLT_MIN;
    // the largest logit of the chosen
    auto largest = [&]() { return unordered(max(__reduce_max_sync(kAll, chosen ? ordered(xj) : 0u), kNone + 1)); };
    if (p.softmax) {              // over it: exact where the row's largest is far away
        const float over = p.renorm ? largest() : xmax;
        if (chosen) w = expf(xj - over) * (p.renorm ? 1.0f : inv_total);
    } else if (p.renorm && !__any_sync(kAll, chosen && xj > -20.0f)) {
        // All scores are small, perhaps too small for FP32 though their parts of the sum are not (eight logits of -88: 6e-39
        // each, 1/8 each): exponentials over the largest logit too, and `least` in the same units, by a half exponential
        // squared (e^89 is infinite before 2^-126 is taken of it).
        const float over = largest(), half = expf(-0.5f * over) * 0x1p-63f;
        least = half * half;
        if (chosen) w = expf(xj - over);                  // (1 + e^x is 1)
    } else if (chosen) {
        w = __fdividef(1.0f, 1.0f + expf(-xj));
    }
    if (p.renorm) {
        float sum = w;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        w = __fdividef(w, fmaxf(sum, least));
    }
    if (lane < p.k) {
        const int64_t at = static_cast<int64_t>(t) * p.k + lane;
        p.ids[at] = my_id;
        p.weights[at] = chosen ? w * p.scale : 0.0f;
        sid[lane] = my_id;
    }
}

__host__ __device__ constexpr int scored_threads(int vpl) { return vpl <= 8 ? 768 : 384; }

template <int VPL, bool BF16, bool BY_LOGIT>
__global__ void __launch_bounds__(scored_threads(VPL), 2) route_select_scored(const __grid_constant__ ScoredParams p) {
    extern __shared__ __align__(16) unsigned long long mask[];            // [E]
    int* total = reinterpret_cast<int*>(mask + p.E);        // [E] (one chunk)
    int* sid = total + p.E;                                 // [CHUNK][k]
    __shared__ __align__(16) float bias[32 * VPL];          // -infinity where there is no expert, or its bias is NaN
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    __shared__ uint2 won[scored_threads(VPL) / 32][DGEMM_MAX_TOPK];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int t0 = blockIdx.x * p.chunk, n = min(p.chunk, p.T - t0);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0;
    for (int e = threadIdx.x; e < 32 * VPL; e += blockDim.x) bias[e] = e < p.E ? bias_at(p, e) : -INFINITY;
    __syncthreads();
    for (int i = warp; i < n; i += warps) {
        route_scored_token<VPL, BF16, BY_LOGIT>(p, t0 + i, lane, bias, won[warp], sid + i * p.k);
        __syncwarp();
        if (lane < p.k && sid[i * p.k + lane] >= 0) atomicOr(&mask[sid[i * p.k + lane]], 1ull << i);
    }
    __syncthreads();
    finish_chunk(p, mask, total, sid, t0, n);
}

template <int VPL>
cudaError_t launch_scored(const ScoredParams& p, cudaStream_t s) {
    const int most = scored_threads(VPL) / 32, warps = std::max(std::min(most, p.chunk), std::min(most, (p.E + 31) / 32));
    dg::host::Launch l(static_cast<unsigned>(p.chunks), 1, 32u * warps, static_cast<size_t>(p.E) * 12 + CHUNK * p.k * 4, s);
    if (p.by_logit)
        return p.bf16 ? cudaLaunchKernelEx(&l.cfg, route_select_scored<VPL, true, true>, p)
                      : cudaLaunchKernelEx(&l.cfg, route_select_scored<VPL, false, true>, p);
    return p.bf16 ? cudaLaunchKernelEx(&l.cfg, route_select_scored<VPL, true, false>, p)
                  : cudaLaunchKernelEx(&l.cfg, route_select_scored<VPL, false, false>, p);
}

}  // namespace
