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

// Relative error of an FP32 score (expf: 2 ulp; sum, quotient; softmax also its sum of up to 1024
// terms, 37 deep, and its rounded argument), absolute part for scores that underflow, and
// relative error of an addition. Scores are bounded by the largest one there can be, so that
// a value far down the list is covered too.
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
__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v) {
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// Top two of the union of (a1 >= a2) and (b1 >= b2), into a.
template <class T>
__device__ __forceinline__ void merge_two(T& a1, T& a2, T b1, T b2) {
    a2 = max(min(a1, b1), max(a2, b2));
    a1 = max(a1, b1);
}

// Bit g: group g is kept. Lane g (below G) holds the order-preserving worth of group g, 0 for
// a group that has nothing to choose. The values at the border are left in `in` and `out`.
template <class T>
__device__ __forceinline__ unsigned keep_groups(const ScoredParams& p, T worth, int lane, T* in, T* out) {
    int better = 0;
    for (int g = 0; g < p.groups; ++g) {
        const T o = __shfl_sync(kAll, worth, g);
        better += o > worth || (o == worth && g < lane);
    }
    const bool keep = worth != 0 && better < p.kept;
    T a = keep ? worth : ~T(0), b = keep ? T(0) : worth;
    for (int o = 16; o > 0; o >>= 1) {
        a = min(a, __shfl_xor_sync(kAll, a, o));
        b = max(b, __shfl_xor_sync(kAll, b, o));
    }
    *in = a;
    *out = b;
    return __ballot_sync(kAll, keep);
}

// The whole token in FP64: lane j keeps the j-th choice.
template <int VPL>
__device__ __noinline__ int choose64(const ScoredParams& p, int t, int lane) {
    unsigned long long key[VPL];
    double xmax = 0.0, total = 1.0;
    if (p.softmax) {
        unsigned long long top = 0;
        for (int i = 0; i < VPL; ++i) {
            const int e = lane * VPL + i;
            const float x = e < p.E && bias_at(p, e) > -INFINITY ? logit_at(p, t, e) : -INFINITY;
            if (x > -INFINITY) top = max(top, ordered64(x));
        }
        top = warp_max64(top);
        if (top == 0) return -1;
        xmax = unordered64(top);
        total = 0.0;
        for (int i = 0; i < VPL; ++i) {
            const int e = lane * VPL + i;
            const float x = e < p.E && bias_at(p, e) > -INFINITY ? logit_at(p, t, e) : -INFINITY;
            if (x > -INFINITY) total += exp(x - xmax);
        }
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    }
    for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        const float x = e < p.E ? logit_at(p, t, e) : -INFINITY, b = e < p.E ? bias_at(p, e) : 0.0f;
        const double s = p.softmax ? exp(x - xmax) / total : 1.0 / (1.0 + exp(-static_cast<double>(x)));
        key[i] = x > -INFINITY && b > -INFINITY ? ordered64(s + b + 0.0) : 0;
    }
    if (p.groups > 1) {
        unsigned long long worth = 0;
        for (int g = 0; g < p.groups; ++g) {
            unsigned long long m1 = 0, m2 = 0;
            for (int i = 0; i < VPL; ++i)
                if (static_cast<unsigned>(lane * VPL + i - g * p.per_group) < static_cast<unsigned>(p.per_group))
                    merge_two(m1, m2, key[i], 0ull);
            for (int o = 16; o > 0; o >>= 1)
                merge_two(m1, m2, __shfl_xor_sync(kAll, m1, o), __shfl_xor_sync(kAll, m2, o));
            if (lane == g) worth = p.top2 && m2 != 0 ? ordered64(unordered64(m1) + unordered64(m2) + 0.0) : m1;
        }
        unsigned long long in, out;
        const unsigned kept = keep_groups(p, worth, lane, &in, &out);
        for (int i = 0; i < VPL; ++i)
            if (!((kept >> min((lane * VPL + i) / p.per_group, 31)) & 1)) key[i] = 0;
    }
    int my_id = -1;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long best = 0;
        for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
        const unsigned long long m = warp_max64(best);
        if (m == 0) break;
        const int src = __ffs(__ballot_sync(kAll, best == m)) - 1;     // lanes in the experts' order: the lowest
        int at = VPL - 1;
        for (int i = VPL - 1; i >= 0; --i) at = key[i] == m ? i : at;
        const int e = __shfl_sync(kAll, lane * VPL + at, src);
        if (lane == src) key[at] = 0;
        my_id = lane == j ? e : my_id;
    }
    return my_id;
}

// Sigmoid scores: the first `count` lanes hold the best experts, whose order alone is open; lane
// j < n gets the j-th of them.
__device__ __noinline__ int order64(const ScoredParams& p, int t, int id, int count, int n, int lane) {
    unsigned long long key = 0;
    if (lane < count) {
        const double x = logit_at(p, t, id);
        key = ordered64(1.0 / (1.0 + exp(-x)) + bias_at(p, id) + 0.0);
    }
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

template <int VPL, bool BF16>
__device__ __forceinline__ void route_scored_token(const ScoredParams& p, int t, int lane, int* sid) {
    // logits (masked: -inf)
    float x[VPL];
    {
        const int64_t at = static_cast<int64_t>(t) * p.E + lane * VPL;
        constexpr int BYTES = VPL * (BF16 ? 2 : 4), WORDS = (BYTES + 3) / 4, VEC = BYTES < 16 ? BYTES : 16;
        const char* src = static_cast<const char*>(p.logits) + at * (BF16 ? 2 : 4);
        if (VPL > 1 && p.E % VPL == 0) {      // (whole lanes: every lane's experts start on a vector)
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
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = x[i] > -INFINITY ? fminf(x[i], FLT_MAX) : -INFINITY;
    // choice values as order-preserving keys, 0: not to be chosen
    unsigned key[VPL];
    float xmax = 0.0f, inv_total = 1.0f;
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane * VPL + i < p.E && !(__ldg(p.bias + lane * VPL + i) > -INFINITY)) x[i] = -INFINITY;
    }
    if (p.softmax) {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = fmaxf(m, x[i]);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        xmax = m > -INFINITY ? m : 0.0f;
    }
    if (p.by_logit) {
        if (p.softmax && !p.renorm) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) sum += expf(x[i] - xmax);
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            inv_total = 1.0f / sum;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = x[i] > -INFINITY ? ordered(x[i] + 0.0f) : 0;
    } else {
        float s[VPL];
        if (p.softmax) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                s[i] = expf(x[i] - xmax);
                sum += s[i];
            }
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            inv_total = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < VPL; ++i) s[i] *= inv_total;
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) s[i] = __fdividef(1.0f, 1.0f + expf(-x[i]));
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const float b = p.bias && lane * VPL + i < p.E ? fminf(__ldg(p.bias + lane * VPL + i), FLT_MAX) : 0.0f;
            key[i] = x[i] > -INFINITY ? ordered(s[i] + b + 0.0f) : 0;
        }
    }
    // twice the most that a score (at most 1, or the softmax's largest) is off
    const float off = 2.0f * (p.softmax ? Margin::kSoftmax * inv_total : Margin::kSigmoid) + Margin::kTiny;
    bool open = false;            // FP32 cannot tell which groups are kept
    if (p.groups > 1) {
        unsigned m1 = 0, m2 = 0, worth = 0;
        if (p.lanes_per_group) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) merge_two(m1, m2, key[i], 0u);
            for (int o = 1; o < p.lanes_per_group; o <<= 1)
                merge_two(m1, m2, __shfl_xor_sync(kAll, m1, o), __shfl_xor_sync(kAll, m2, o));
            const int first = min(lane * p.lanes_per_group, 31);
            m1 = __shfl_sync(kAll, m1, first);
            m2 = __shfl_sync(kAll, m2, first);
            if (lane >= p.groups) m1 = m2 = 0;
        } else {
            for (int g = 0; g < p.groups; ++g) {
                unsigned a1 = 0, a2 = 0;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    merge_two(a1, a2, static_cast<unsigned>(lane * VPL + i - g * p.per_group) <
                                              static_cast<unsigned>(p.per_group) ? key[i] : 0u, 0u);
                for (int o = 16; o > 0; o >>= 1)
                    merge_two(a1, a2, __shfl_xor_sync(kAll, a1, o), __shfl_xor_sync(kAll, a2, o));
                if (lane == g) m1 = a1, m2 = a2;
            }
        }
        worth = p.top2 && m2 != 0 ? ordered(unordered(m1) + unordered(m2) + 0.0f) : m1;
        unsigned in, out;
        const unsigned kept = keep_groups(p, worth, lane, &in, &out);
        if (!p.by_logit && out != 0 && in != kAll) {
            const float a = unordered(in), b = unordered(out);
            float size = 0.0f;          // the values that were added may be larger than their sum
            if (lane < p.groups && worth != 0) size = fabsf(unordered(m1)) + (m2 != 0 ? fabsf(unordered(m2)) : 0.0f);
            for (int o = 16; o > 0; o >>= 1) size = fmaxf(size, __shfl_xor_sync(kAll, size, o));
            open = a - b <= 2.0f * off + 4.0f * Margin::kSum * size;
        }
        if (p.lanes_per_group) {
            const bool keep = (kept >> min(lane / p.lanes_per_group, 31)) & 1;
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = keep ? key[i] : 0;
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (!((kept >> min((lane * VPL + i) / p.per_group, 31)) & 1)) key[i] = 0;
        }
    }
    // the k largest, and where FP32 values decide the two behind them
    int my_id = -1, n = 0;
    unsigned my_key = 0;
    unsigned behind = 0, behind2 = 0;
    int behind_id = -1;
    auto take = [&](unsigned& m) {
        unsigned best = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
        m = __reduce_max_sync(kAll, best);
        // (lanes are in the experts' order, so the first one that holds it has the lowest expert)
        const int src = __ffs(__ballot_sync(kAll, best == m)) - 1;
        const unsigned mine = lane == src ? m : 0u;     // 0: nothing of this lane (its keys may be 0 already)
        int at = 0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool hit = key[i] == mine && !found;
            at = hit ? i : at;
            key[i] = hit ? 0 : key[i];
            found = found || hit;
        }
        return __shfl_sync(kAll, lane * VPL + at, src);
    };
    for (int j = 0; j < p.k; ++j) {
        unsigned m;
        const int e = take(m);
        if (m == 0) break;
        n = j + 1;
        my_id = lane == j ? e : my_id;
        my_key = lane == j ? m : my_key;
    }
    float xj = lane < n ? logit_at(p, t, my_id) : 0.0f;
    // (accurate: the weights are made of it)
    auto score_of = [&](float v) { return p.softmax ? expf(v - xmax) * inv_total : 1.0f / (1.0f + expf(-v)); };
    if (!p.by_logit) {
        if (!open && n == p.k) behind_id = take(behind);
        const float bj = lane < n ? bias_at(p, my_id) : 0.0f, cj = unordered(my_key);
        const float xe = behind ? logit_at(p, t, behind_id) : 0.0f, be = behind ? bias_at(p, behind_id) : 0.0f;
        float xn = __shfl_down_sync(kAll, xj, 1), bn = __shfl_down_sync(kAll, bj, 1), cn = __shfl_down_sync(kAll, cj, 1);
        if (lane == n - 1) xn = xe, bn = be, cn = unordered(behind);
        const bool pair = lane < n - 1 || (lane == n - 1 && behind != 0);
        auto near = [&](float c1, float c2) { return c1 - c2 <= off + Margin::kSum * (fabsf(c1) + fabsf(c2)); };
        const bool tight = pair && !(xj == xn && bj == bn) && near(cj, cn);
        if (open) {
            my_id = choose64<VPL>(p, t, lane);
        } else if (__any_sync(kAll, tight)) {
            bool all = p.softmax || n >= 32;
            if (!all && behind) {         // is the one behind apart from the next?
                const int next_id = take(behind2);
                if (behind2) {
                    const float x2 = logit_at(p, t, next_id);
                    all = !(x2 == xe && bias_at(p, next_id) == be) && near(unordered(behind), unordered(behind2));
                }
            }
            if (all) my_id = choose64<VPL>(p, t, lane);
            else my_id = order64(p, t, lane == n && behind ? behind_id : my_id, behind ? n + 1 : n, n, lane);
        }
        xj = my_id >= 0 ? logit_at(p, t, my_id) : 0.0f;
    }
    float w = 0.0f;
    if (p.renorm) {
        if (p.softmax) {          // over the largest logit of the chosen: exact where the row's largest is far away
            float m = my_id >= 0 ? xj : -INFINITY;
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
            w = my_id >= 0 ? expf(xj - m) : 0.0f;
        } else {
            w = my_id >= 0 ? score_of(xj) : 0.0f;
        }
        float sum = w;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        w = w / fmaxf(sum, FLT_MIN);
    } else if (my_id >= 0) {
        w = score_of(xj);
    }
    if (lane < p.k) {
        const int64_t at = static_cast<int64_t>(t) * p.k + lane;
        p.ids[at] = my_id;
        p.weights[at] = my_id >= 0 ? w * p.scale : 0.0f;
        sid[lane] = my_id;
    }
}

constexpr int scored_threads(int vpl) { return vpl <= 8 ? 768 : 384; }

template <int VPL, bool BF16>
__global__ void __launch_bounds__(scored_threads(VPL), 2) route_select_scored(const __grid_constant__ ScoredParams p) {
    extern __shared__ __align__(16) unsigned long long mask[];            // [E]
    int* total = reinterpret_cast<int*>(mask + p.E);        // [E] (one chunk)
    int* sid = total + p.E;                                 // [CHUNK][k]
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int t0 = blockIdx.x * p.chunk, n = min(p.chunk, p.T - t0);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0;
    __syncthreads();
    for (int i = warp; i < n; i += warps) {
        route_scored_token<VPL, BF16>(p, t0 + i, lane, sid + i * p.k);
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
    return p.bf16 ? cudaLaunchKernelEx(&l.cfg, route_select_scored<VPL, true>, p)
                  : cudaLaunchKernelEx(&l.cfg, route_select_scored<VPL, false>, p);
}

}  // namespace
