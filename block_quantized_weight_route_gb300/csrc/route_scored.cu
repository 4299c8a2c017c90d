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
// bits (one in some hundred tokens of random logits).  Each of the k rounds is two warp
// reductions (redux): the largest key, then the lowest index that has it.
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
__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float logit(const ScoredParams& p, long t, int e) {
    const long i = t * p.ldl + e;
    const float v = p.l_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[i]) : static_cast<const float*>(p.logits)[i];
    return v == v ? v : -INFINITY;   // (NaN: off, as -inf)
}

// exp(l) / (1 + exp(l)) from the side where nothing overflows, times exp(-shift) for l <= 0.
__device__ __forceinline__ float sigmoid(float l, float shift) {
    const float t = expf(-fabsf(l));
    return (l > 0.0f ? 1.0f : shift == 0.0f ? t : expf(l - shift)) / (1.0f + t);
}

// The groups that stay, as a mask; `c` holds the row's values (-inf: off).  Lanes share the groups
// evenly; `tol` (32 bits): *close is set where a group that stays and one that goes are no
// further apart than their error.
template <class F>
__device__ __forceinline__ uint32_t groups_kept(const ScoredParams& p, const F* c, int lane, float tol, bool* close) {
    const int p2 = p.groups <= 1 ? 1 : 1 << (32 - __clz(p.groups - 1)), per = 32 / p2;   // lanes a group
    const int g = lane / per, sub = lane % per;
    F a = -INFINITY, b = -INFINITY;   // the two largest
    if (g < p.groups) {
        const F* row = c + g * p.group_size;
        for (int i = sub; i < p.group_size; i += per) {
            const F v = row[i];
            b = fmax(b, fmin(a, v));
            a = fmax(a, v);
        }
    }
    for (int o = 1; o < per; o <<= 1) {
        const F a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
        b = fmax(fmin(a, a2), fmax(b, b2));
        a = fmax(a, a2);
    }
    const F score = p.group_top == 1 ? a : b > -INFINITY ? a + b : (F)-INFINITY;
    int before = 0;
    for (int h = 0; h < p.groups; ++h) {
        const F s = __shfl_sync(kAll, score, h * per);
        before += s > score || (s == score && h < g);
    }
    const bool live = g < p.groups, keep = live && before < p.groups_kept;
    if constexpr (sizeof(F) == 4) {
        const float low = -warp_max_f(keep ? -(float)score : -INFINITY);            // the worst that stays
        const float high = warp_max_f(live && !keep ? (float)score : -INFINITY);    // the best that goes
        const float size = warp_max_f(score > -INFINITY && score < INFINITY ? fabsf(a) + fabsf(b > -INFINITY ? b : a) : 0.0f);
        *close = high > -INFINITY && low - high <= 2.0f * (tol + 2.4e-7f * size);
    }
    const uint32_t lanes = __ballot_sync(kAll, keep && sub == 0);
    uint32_t mask = 0;
    for (int h = 0; h < p.groups; ++h) mask |= (lanes >> (h * per) & 1u) << h;
    return mask;
}

__device__ __forceinline__ bool in_groups(const ScoredParams& p, uint32_t mask, int e) {
    return p.groups == 1 || (mask >> ((unsigned)e * p.group_inv >> 20) & 1u);
}

// The choice in 64 bits, from shared memory: lane j returns the j-th id.
__device__ __noinline__ int choose64(const ScoredParams& p, long t, int lane, double* c) {
    double m = 0.0, z = 1.0;
    if (!p.sigmoid) {
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
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) {
        const float l = logit(p, t, e);
        double v = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - m) / z;
        if (p.bias) v += (double)p.bias[e];
        c[e] = l > -INFINITY && v == v ? v : -INFINITY;
    }
    __syncwarp();
    uint32_t mask = ~0u;
    bool unused;
    if (p.groups > 1) mask = groups_kept<double>(p, c, lane, 0.0f, &unused);
    __syncwarp();
    uint64_t* keys = reinterpret_cast<uint64_t*>(c);
    for (int e = lane; e < p.E; e += 32) {
        const double v = c[e];
        keys[e] = v > -INFINITY && in_groups(p, mask, e) ? key_of(v) : 0ull;
    }
    int mine = -1;
    for (int j = 0; j < p.k; ++j) {
        uint64_t best = 0;
        int at = kMaxE;
        for (int e = lane; e < p.E; e += 32) {
            if (keys[e] > best) {
                best = keys[e];
                at = e;
            }
        }
        const uint64_t top = warp_max(best);
        if (top == 0) break;
        const int e = (int)__reduce_min_sync(kAll, (unsigned)(best == top ? at : kMaxE));
        if (lane == j) mine = e;
        if ((e & 31) == lane) keys[e] = 0;
    }
    return mine;
}

template <int EPL>
__global__ void __launch_bounds__(32 * kWarps) route_scored_kernel(ScoredParams p) {
    extern __shared__ double smem[];   // [warps][E], where scores are needed
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
    float l[EPL], m = -INFINITY, z = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < p.E ? logit(p, t, e) : -INFINITY;
        m = fmaxf(m, l[i]);
    }
    const bool by_logit = !p.bias && (p.groups == 1 || p.group_top == 1);
    float x[EPL];   // softmax: exp(l - max)
    const bool need_z = !p.sigmoid && (!p.renorm || !by_logit);
    if (need_z) {
        m = warp_max_f(m);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            x[i] = l[i] > -INFINITY ? expf(l[i] - m) : 0.0f;
            z += x[i];
        }
        z = warp_sum(z);
    }
    float c[EPL];
    float tol = 0.0f;   // bound on the difference of the errors of two scores
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = l[i];
    } else {
        // A sigmoid is off by at most 7 roundings' halves (expf 2 ulp, sum, quotient), a softmax
        // by those of its exponential and of a sum of 16 and then 32 terms; both at most
        // their largest score.
        const float rz = 1.0f / z;
        tol = p.sigmoid ? 9.6e-7f : 3.9e-6f * rz;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 32 * i;
            float s = p.sigmoid ? sigmoid(l[i], 0.0f) : x[i] * rz;
            if (p.bias && e < p.E) s += __ldg(p.bias + e);
            c[i] = l[i] > -INFINITY && s == s ? s : -INFINITY;
        }
    }
    uint32_t mask = ~0u;
    bool close = false;
    double* row = smem + warp * p.E;
    if (p.groups > 1) {
        float* cf = reinterpret_cast<float*>(row);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane + 32 * i < p.E) cf[lane + 32 * i] = c[i];
        __syncwarp();
        mask = groups_kept<float>(p, cf, lane, tol, &close);
        close &= !by_logit;
        __syncwarp();
    }
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = c[i] > -INFINITY && in_groups(p, mask, lane + 32 * i) ? key_of(c[i]) : 0u;
    int mine = -1;
    float last = INFINITY;
    const int rounds = p.k + !by_logit;   // (one more: the first that is not chosen must not be close either)
    for (int j = 0; j < rounds; ++j) {
        uint32_t best = 0;
        int at = kMaxE;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
            }
        }
        const uint32_t top = warp_max(best);
        if (top == 0) break;
        const int e = (int)__reduce_min_sync(kAll, (unsigned)(best == top ? at : kMaxE));
        if (lane == j && j < p.k) mine = e;
        const float v = value_of(top);
        close |= !by_logit && last - v <= tol + 2.4e-7f * fabsf(v);
        last = v;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e == lane + 32 * i) key[i] = 0;
    }
    if (close) mine = choose64(p, t, lane, row);   // (the same in the whole warp)

    // The weights: lane j has id j.  Renormalised ones are ratios, from exponentials relative to the largest
    // chosen logit, so that scores which all underflow keep their ratio.
    const bool on = mine >= 0;
    const float lj = on ? logit(p, t, mine) : -INFINITY;
    float s = 0.0f;
    if (p.renorm) {
        const float top = warp_max_f(lj);
        if (on) s = p.sigmoid ? sigmoid(lj, fminf(top, 0.0f)) : expf(lj - top);
        const float sum = warp_sum(s);
        s = sum == 0.0f ? 0.0f : s / sum;
    } else if (on) {
        s = p.sigmoid ? sigmoid(lj, 0.0f) : expf(lj - m) / z;
    }
    if (lane < p.k) {
        p.ids[t * p.k + lane] = mine;
        p.w[t * p.k + lane] = s * p.scale;
    }
}

template <int EPL>
cudaError_t launch(const ScoredParams& p, int warps, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {overlap_attribute()};
    cfg.gridDim = dim3((unsigned)((p.T + warps - 1) / warps), 1, 1);
    cfg.blockDim = dim3(32 * warps, 1, 1);
    cfg.dynamicSmemBytes = p.bias || p.groups > 1 ? (size_t)warps * p.E * 8 : 0;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_scored_kernel<EPL>, p);
}

}  // namespace

cudaError_t launch_route_scored(ScoredParams p, int sms, cudaStream_t s) {
    p.group_size = p.E / p.groups;
    p.group_inv = ((1u << 20) + p.group_size - 1) / p.group_size;   // e / group_size = e * inv >> 20 for e < 512
    const int warps = p.T > sms ? kWarps : 1;   // (few tokens: each on an SM of its own)
    const int epl = (p.E + 31) / 32;
    if (epl <= 1) return launch<1>(p, warps, s);
    if (epl <= 2) return launch<2>(p, warps, s);
    if (epl <= 4) return launch<4>(p, warps, s);
    if (epl <= 8) return launch<8>(p, warps, s);
    return launch<16>(p, warps, s);
}

}  // namespace qmm
