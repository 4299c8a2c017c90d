// Routing by scores: softmax or sigmoid, a bias for the choice, groups of experts, top-k,
// renormalised and scaled weights.
//
//   s = softmax(l) or 1 / (1 + exp(-l));   c = s + bias;   a group's score: the sum of its
//   `top` largest c;   ids: the k largest c in the `kept` best groups;   w = s[id] (/ their sum) * scale
//
// One warp a token, lane l holding the logits l, l + 32, ...  The choice is that of exact
// arithmetic, ties to the lower index, so that it does not hang on how an exponential was
// rounded: without a bias (and with group scores of one expert) c grows with the logit
// and the logits themselves are compared; else c is computed in 32 bits with a bound on its
// error, and a token with two neighbours in the order closer than that is done again in 64
// bits (one in a thousand tokens of random logits), for the few experts that it is between.  A round of the
// choice is one warp reduction (redux) and a ballot: a lane keeps its keys sorted, so that the next one
// is in hand, and a key carries its place in the lane.
// Measured with 256 experts, 8 of them a token, sigmoid, bias, 4 of 8 groups: 1 token 3.1 us (in a graph), 5268
// 12 us, 21504 28 us.  What bounds it is instructions (about 1000 a token, issue slots 80% busy;
// the logits' 22 MB take 3.3 us): 19 us without groups, 15 without bias either.
#include <cfloat>

#include "qmm_internal.h"
#include "quant8.cuh"

namespace qmm {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxE = 512;
constexpr int kWarps = 4;   // of a CTA, where there are tokens enough

// Keys that order as the values do: larger value, larger key; 0 for an expert that is off.
// (-0 and +0 are one value.)
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k); }
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}
template <int LANES = 32>   // (of the first LANES, and the rest among themselves)
__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
template <int LANES = 32, class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float live_logit(float v) { return v == v ? v : -INFINITY; }   // (NaN: off, as -inf)
__device__ __forceinline__ float logit(const ScoredParams& p, long t, int e) {
    const long i = t * p.ldl + e;
    return live_logit(p.l_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[i]) : static_cast<const float*>(p.logits)[i]);
}

// exp(l) / (1 + exp(l)) from the side where nothing overflows, times exp(-shift) for l <= 0.
__device__ __forceinline__ float sigmoid(float l, float shift) {
    const float t = expf(-fabsf(l));
    return __fdividef(l > 0.0f ? 1.0f : shift == 0.0f ? t : expf(l - shift), 1.0f + t);
}
// The same for the choice.  2^(-|l| log2 e) by the exponential instruction is within 2 ulp and, for its
// rounded argument, 1.2 |l| ulp more, which exp(-|l|) / (1 + exp(-|l|))^2, the slope, brings below 7e-8
// for any l; the sum's rounding and the approximate reciprocal add 1.8e-7: within 2.5e-7 of the sigmoid.
__device__ __forceinline__ float fast_sigmoid(float l) {
    float t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fabsf(l) * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
    return l > 0.0f ? r : t * r;
}
constexpr float kSigmoidTol = 5e-7f;      // of the difference of two
constexpr float kSoftmaxTol = 3.9e-6f;    // the same, of the largest score: an exponential and a sum of 16 and then 32 terms
constexpr float kSumTol = 2.4e-7f;        // of a sum's size: the bias' addition, twice

// Where a row's expert e is kept in shared memory: groups of 32 start in different banks.
__device__ __forceinline__ int place(int e) { return e + (e >> 5) * 4; }

// The groups that stay, as the ballot of their lanes: the lanes share the groups, 2^p.per_shift
// each.  `c` holds the row's values (-inf: off); `tol` (32 bits): *close is set where the last
// group that stays and the first that goes are no further apart than their error.  *least: the smallest
// value in the lane's group's score.
template <class F>
__device__ __forceinline__ uint32_t groups_kept(const ScoredParams& p, const F* c, int lane, float tol, bool* close, F* least) {
    const int per = 1 << p.per_shift, g = lane >> p.per_shift, sub = lane & (per - 1);
    const bool live = g < p.groups;
    F a = -INFINITY, b = -INFINITY;   // the two largest
    if (live) {
        const int end = (g + 1) * p.group_size;
        for (int e = g * p.group_size + sub; e < end; e += 4 * per) {   // (four loads in flight)
            F v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = e + i * per < end ? c[place(e + i * per)] : (F)-INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                b = fmax(b, fmin(a, v[i]));
                a = fmax(a, v[i]);
            }
        }
    }
    for (int o = 1; o < per; o <<= 1) {
        const F a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
        b = fmax(fmin(a, a2), fmax(b, b2));
        a = fmax(a, a2);
    }
    const F score = p.group_top == 1 ? a : b > -INFINITY ? a + b : (F)-INFINITY;
    *least = p.group_top == 1 ? a : b;
    auto key = live && sub == 0 ? key_of(score) : 0;   // (a live group's is not 0)
    uint32_t kept = 0;
    F last = INFINITY;
    for (int i = 0; i < p.groups_kept; ++i) {
        const auto top = warp_max(key);
        const uint32_t who = __ballot_sync(kAll, key == top);
        const uint32_t first = who & -who;   // (the lowest group of equal ones)
        kept |= first;
        if (first >> lane & 1u) key = 0;
        if constexpr (sizeof(F) == 4) last = value_of(top);
    }
    if constexpr (sizeof(F) == 4) {
        const uint32_t next = warp_max(key);
        // (infinite biases add exactly; a finite sum past the largest number makes the size infinite: 64 bits decide)
        const float x = fabsf(a), y = p.group_top == 1 ? 0.0f : fabsf(b);
        const float parts = (x < INFINITY ? x : 0.0f) + (y < INFINITY ? y : 0.0f);
        const float size = __uint_as_float(__reduce_max_sync(kAll, live ? __float_as_uint(parts) : 0u));
        *close = size == INFINITY || (next > key_of(-INFINITY) && last - value_of(next) <= 2.0f * (tol + kSumTol * size));
    }
    return kept;
}

// Whether e's group stays (p.group_inv: 2^20 / group_size, rounded up).
__device__ __forceinline__ bool in_groups(const ScoredParams& p, uint32_t kept, int e) {
    return kept >> (((unsigned)e * p.group_inv >> 20) << p.per_shift & 31u) & 1u;
}

// A sigmoid's value for the choice in 64 bits (-inf for a bias that is NaN).
__device__ __forceinline__ double sigmoid64(const ScoredParams& p, long t, int e) {
    const double v = 1.0 / (1.0 + exp(-(double)logit(p, t, e))) + (p.bias ? (double)p.bias[e] : 0.0);
    return v == v ? v : -INFINITY;
}

// The groups that stay, from the 64-bit values of the n <= 32 experts in `list` that can be among the largest of
// their groups.
__device__ __noinline__ uint32_t groups64(const ScoredParams& p, long t, int lane, const int* list, int n) {
    const int e = lane < n ? list[lane] : 0;
    const double v = lane < n ? sigmoid64(p, t, e) : -INFINITY;
    const int of = (int)((unsigned)e * p.group_inv >> 20);
    double a = -INFINITY, b = -INFINITY;   // lane g: the two largest of group g
    for (int i = 0; i < n; ++i) {
        const double o = __shfl_sync(kAll, v, i);
        if (__shfl_sync(kAll, of, i) == lane) {
            b = fmax(b, fmin(a, o));
            a = fmax(a, o);
        }
    }
    const double score = p.group_top == 1 ? a : b > -INFINITY ? a + b : -INFINITY;
    int before = 0;
    for (int h = 0; h < p.groups; ++h) {
        const double o = __shfl_sync(kAll, score, h);
        before += o > score || (o == score && h < lane);
    }
    const uint32_t keep = __ballot_sync(kAll, lane < p.groups && before < p.groups_kept);
    uint32_t kept = 0;
    for (int h = 0; h < p.groups; ++h) kept |= (keep >> h & 1u) << (h << p.per_shift);
    return kept;
}

// The choice in 64 bits, from shared memory: lane j returns the j-th id.  `kept`: the groups that
// stay, or (again) not known yet; experts whose 32-bit value is below `least` (sigmoid) are not among the k.
template <bool SCORED, bool GROUPS>
__device__ __noinline__ int choose64(const ScoredParams& p, long t, int lane, double* c, bool again, uint32_t kept, float least) {
    double m = 0.0, z = 1.0;
    if (SCORED && !p.sigmoid) {
        float top = -INFINITY;
        for (int e = lane; e < p.E; e += 32) top = fmaxf(top, logit(p, t, e));
        m = warp_max_f(top);
        z = 0.0;
        for (int e = lane; e < p.E; e += 32) {
            const float l = logit(p, t, e);
            if (l > -INFINITY) z += exp((double)l - m);
        }
        z = warp_sum(z);
    }
    auto value = [&](float l, float b) {
        if (!SCORED) return (double)l;
        const double v = (p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - m) / z) + (double)b;
        return v == v ? v : -INFINITY;
    };
    if (SCORED && p.sigmoid && !again) {
        // The few that can be among the k, one to a lane: one exponential in 64 bits (1 us, and 8 for a lane's
        // eight one after the other: at the end of a launch nothing else runs beside it).  A value's
        // place is the number of those before it.
        int* list = reinterpret_cast<int*>(c);
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const float l = e < p.E ? logit(p, t, e) : -INFINITY, b = p.bias && e < p.E ? p.bias[e] : 0.0f;
            const bool in = l > -INFINITY && (!GROUPS || in_groups(p, kept, e)) && fast_sigmoid(l) + b >= least;
            const uint32_t who = __ballot_sync(kAll, in);
            const int at = n + __popc(who & ((1u << lane) - 1u));
            if (in && at < 32) list[at] = e;
            n += __popc(who);
        }
        __syncwarp();
        if (n <= 32) {
            const int e = lane < n ? list[lane] : kMaxE;
            const double v = lane < n ? sigmoid64(p, t, e) : -INFINITY;
            int before = 0;
            for (int i = 0; i < n; ++i) {
                const double o = __shfl_sync(kAll, v, i);
                before += o > v || (o == v && i < lane);   // (the list is in ascending order)
            }
            __syncwarp();
            if (lane < n && v > -INFINITY) list[before] = e;
            const int got = __popc(__ballot_sync(kAll, lane < n && v > -INFINITY));
            __syncwarp();
            return lane < p.k && lane < got ? list[lane] : -1;
        }
        __syncwarp();
    }
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) {
        const float l = logit(p, t, e);
        c[place(e)] = l > -INFINITY ? value(l, p.bias ? p.bias[e] : 0.0f) : -INFINITY;
    }
    __syncwarp();
    bool unused;
    double unused_too;
    if (GROUPS && again) kept = groups_kept<double>(p, c, lane, 0.0f, &unused, &unused_too);
    __syncwarp();
    uint64_t* keys = reinterpret_cast<uint64_t*>(c);
    for (int e = lane; e < p.E; e += 32) {
        const double v = c[place(e)];
        keys[place(e)] = v > -INFINITY && (!GROUPS || in_groups(p, kept, e)) ? key_of(v) : 0ull;
    }
    int mine = -1;
    for (int j = 0; j < p.k; ++j) {
        uint64_t best = 0;
        int at = kMaxE;
        for (int e = lane; e < p.E; e += 32) {
            if (keys[place(e)] > best) {
                best = keys[place(e)];
                at = e;
            }
        }
        const uint64_t top = warp_max(best);
        if (top == 0) break;
        const int e = (int)__reduce_min_sync(kAll, (unsigned)(best == top ? at : kMaxE));
        if (lane == j) mine = e;
        if ((e & 31) == lane) keys[place(e)] = 0;
    }
    return mine;
}

// Largest first (a bitonic network: two operations a comparator).
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&k)[N]) {
#pragma unroll
    for (int size = 2; size <= N; size *= 2) {
#pragma unroll
        for (int step = size / 2; step > 0; step /= 2) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int o = i ^ step;
                if (o > i) {
                    const bool down = (i & size) == 0;
                    const uint32_t hi = max(k[i], k[o]), lo = min(k[i], k[o]);
                    k[i] = down ? hi : lo;
                    k[o] = down ? lo : hi;
                }
            }
        }
    }
}

// SCORED: the choice needs the scores (a bias, or sums of a group); else the logits decide.
template <int EPL, bool SCORED, bool GROUPS>
__global__ void __launch_bounds__(32 * kWarps) route_scored_kernel(const __grid_constant__ ScoredParams p) {
    extern __shared__ double smem[];   // a row of place(E) a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    launch_dependents();
    wait_prerequisites();
    const long t = (long)blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= p.T) return;
    if (p.live && t >= *p.live) {
        if (lane < p.k) {
            p.ids[t * p.k + lane] = -1;
            p.w[t * p.k + lane] = 0.0f;
        }
        return;
    }
    float c[EPL], bias[EPL], m = -INFINITY, z = 0.0f;
    if (p.l_bf16) {
        const __nv_bfloat16* a = static_cast<const __nv_bfloat16*>(p.logits) + t * p.ldl + lane;
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = lane + 32 * i < p.E ? __bfloat162float(a[32 * i]) : -INFINITY;
    } else {
        const float* a = static_cast<const float*>(p.logits) + t * p.ldl + lane;
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = lane + 32 * i < p.E ? a[32 * i] : -INFINITY;
    }
    if (SCORED) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) bias[i] = p.bias && lane + 32 * i < p.E ? p.bias[lane + 32 * i] : 0.0f;
    }
    // (a NaN is not greater than -inf: off too)
    const bool need_z = !p.sigmoid && (SCORED || !p.renorm);
    float tol = 0.0f;   // bound on the difference of the errors of two scores
    if (need_z) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) m = fmaxf(m, c[i]);
        m = warp_max_f(m);
        float x[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            x[i] = c[i] > -INFINITY ? expf(c[i] - m) : 0.0f;
            z += x[i];
        }
        z = warp_sum(z);
        if (SCORED) {
            const float rz = 1.0f / z;
            tol = kSoftmaxTol * rz;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float v = x[i] * rz + bias[i];
                c[i] = c[i] > -INFINITY && v > -INFINITY ? v : -INFINITY;
            }
        }
    } else if (SCORED) {
        tol = kSigmoidTol;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float v = fast_sigmoid(c[i]) + bias[i];
            c[i] = c[i] > -INFINITY && v > -INFINITY ? v : -INFINITY;
        }
    }
    uint32_t kept = ~0u;
    bool again = false;   // groups too close to tell
    double* row = smem + warp * place(p.E + 31);
    if constexpr (GROUPS) {
        float* cf = reinterpret_cast<float*>(row);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane + 32 * i < p.E) cf[place(lane + 32 * i)] = c[i] > -INFINITY ? c[i] : -INFINITY;
        __syncwarp();
        float least;
        kept = groups_kept<float>(p, cf, lane, tol, &again, &least);
        again &= SCORED;
        __syncwarp();
        if (SCORED && again && p.sigmoid) {   // (the same in the whole warp)
            int* list = reinterpret_cast<int*>(row);
            int n = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const unsigned group = (unsigned)(lane + 32 * i) * p.group_inv >> 20;
                const float l = __shfl_sync(kAll, least, group << p.per_shift & 31u);
                const float margin = fabsf(l) < INFINITY ? 2.0f * (tol + kSumTol * fabsf(l)) : 0.0f;
                const bool in = c[i] > -INFINITY && c[i] >= l - margin;
                const uint32_t who = __ballot_sync(kAll, in);
                const int at = n + __popc(who & ((1u << lane) - 1u));
                if (in && at < 32) list[at] = lane + 32 * i;
                n += __popc(who);
            }
            __syncwarp();
            if (n <= 32) {
                kept = groups64(p, t, lane, list, n);
                again = false;
            }
            __syncwarp();
        }
    }
    // A lane's keys, sorted, largest first.  A key's low bits give way to the place i in the lane, from
    // which a lower index is larger; keys whose other bits differ order as the values do, and where two
    // neighbours' are equal the values may differ in what was cut off (bf16 logits lose nothing).
    constexpr uint32_t kPlace = EPL - 1;
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        key[i] = c[i] > -INFINITY && (!GROUPS || in_groups(p, kept, lane + 32 * i)) ? (key_of(c[i]) & ~kPlace) | (kPlace - i) : 0u;
    sort_down(key);
    // k rounds, and one more: the first that is not chosen must not be close to the last that is either.
    // Lane j keeps the key and the lane of the j-th (key 0: there is none).
    uint32_t my_key = 0, my_lane = 0;
    for (int j = 0; j <= p.k; ++j) {
        const uint32_t top = warp_max(key[0]);
        const uint32_t from = __ffs(__ballot_sync(kAll, key[0] == top)) - 1;   // (equal keys: of one place, the lowest lane first)
        if (lane == j) {
            my_key = top;
            my_lane = from;
        }
        if (lane == from) {
#pragma unroll
            for (int i = 0; i + 1 < EPL; ++i) key[i] = key[i + 1];
            key[EPL - 1] = 0;
        }
    }
    const bool got = my_key != 0 && lane <= p.k;
    int mine = got && lane < p.k ? (int)(my_lane + 32 * (kPlace - (my_key & kPlace))) : -1;
    // Lane j looks at the j-th and the next.
    const float cut = kPlace * 1.2e-7f + kSumTol;   // of a value's size: what was cut off, and kSumTol
    const uint32_t next_key = __shfl_down_sync(kAll, my_key, 1);
    const float v = value_of(my_key & ~kPlace), next = value_of(next_key & ~kPlace);
    bool close = lane < p.k && next_key != 0;
    close = close && (SCORED ? v - next <= tol + cut * fabsf(next) : !p.l_bf16 && v == next);
    if (again || __any_sync(kAll, close)) {
        const float last = __shfl_sync(kAll, v, p.k), size = __shfl_sync(kAll, fabsf(v), p.k);
        const bool all = __shfl_sync(kAll, my_key, p.k) == 0;   // (no more than k to choose from)
        mine = choose64<SCORED, GROUPS>(p, t, lane, row, again, kept, all ? -INFINITY : last - 2.0f * (tol + cut * size));
    }

    // The weights: lane j has id j.  Renormalised ones are ratios, from exponentials relative to the largest
    // chosen logit, so that scores which all underflow keep their ratio.
    const bool on = mine >= 0;
    const float lj = on ? logit(p, t, mine) : -INFINITY;
    float s = 0.0f;
    if (p.renorm) {
        const float top = warp_max_f<16>(lj);   // (k <= 16)
        if (on) s = p.sigmoid ? sigmoid(lj, fminf(top, 0.0f)) : expf(lj - top);
        const float sum = warp_sum<16>(s);
        s = sum == 0.0f ? 0.0f : __fdividef(s, sum);
    } else if (on) {
        s = p.sigmoid ? sigmoid(lj, 0.0f) : expf(lj - m) / z;
    }
    if (lane < p.k) {
        p.ids[t * p.k + lane] = mine;
        p.w[t * p.k + lane] = on ? s * p.scale : 0.0f;   // (0 whatever the scale)
    }
}

template <int EPL, bool SCORED, bool GROUPS>
cudaError_t launch(const ScoredParams& p, int warps, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {overlap_attribute()};
    cfg.gridDim = dim3((unsigned)((p.T + warps - 1) / warps), 1, 1);
    cfg.blockDim = dim3(32 * warps, 1, 1);
    cfg.dynamicSmemBytes = (size_t)warps * (p.E + 31 + ((p.E + 31) >> 5) * 4) * 8;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_scored_kernel<EPL, SCORED, GROUPS>, p);
}

template <int EPL>
cudaError_t launch_mode(const ScoredParams& p, int warps, cudaStream_t s) {
    const bool groups = p.groups > 1, scored = p.bias || (groups && p.group_top > 1);
    if (groups) return scored ? launch<EPL, true, true>(p, warps, s) : launch<EPL, false, true>(p, warps, s);
    return scored ? launch<EPL, true, false>(p, warps, s) : launch<EPL, false, false>(p, warps, s);
}

}  // namespace

cudaError_t launch_route_scored(ScoredParams p, int sms, cudaStream_t s) {
    p.group_size = p.E / p.groups;
    p.group_inv = ((1u << 20) + p.group_size - 1) / p.group_size;   // e / group_size = e * inv >> 20 for e < 512
    p.per_shift = 5;
    while ((32 >> p.per_shift) < p.groups) --p.per_shift;
    const int warps = p.T > sms ? kWarps : 1;   // (few tokens: each on an SM of its own)
    const int epl = (p.E + 31) / 32;
    if (epl <= 1) return launch_mode<1>(p, warps, s);
    if (epl <= 2) return launch_mode<2>(p, warps, s);
    if (epl <= 4) return launch_mode<4>(p, warps, s);
    if (epl <= 8) return launch_mode<8>(p, warps, s);
    return launch_mode<16>(p, warps, s);
}

}  // namespace qmm
