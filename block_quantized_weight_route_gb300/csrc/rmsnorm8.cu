// Residual addition + RMS norm + output in 8 bits (qmm_add_rmsnorm_fp8,
// qmm_add_rmsnorm_q8_1).
//
//   v = x, or r' = x + r rounded to the residual's type and stored;
//   y = v / sqrt(mean(v^2) + eps) * g;  y in groups of 128 (E4M3) or 32 (q8_1).
// Everything between the loads and the stores is fp32.  One CTA per row; a
// thread holds NV vectors of 8 consecutive values in registers, so the row is
// read once; 16 (or 4) consecutive lanes hold one group, whose maximum is a few
// shuffles.
#include "qmm_internal.h"
#include "quant8.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const void* p, long i, bool bf16, float (&v)[8]) {
    if (bf16) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float a) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

template <bool Q81, int NV>
__global__ void __launch_bounds__(kThreads) rmsnorm8_kernel(NormParams p) {
    __shared__ float part[kThreads / 32];
    launch_dependents();
    wait_prerequisites();
    const long t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float v[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int i = (n * kThreads + threadIdx.x) * 8;
        if (i < p.D) {
            load8(p.X, t * p.ldx + i, p.x_bf16, v[n]);
            if (p.R) {
                float r[8];
                load8(p.R, t * p.ldr + i, p.r_bf16, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[n][j] += r[j];
                if (p.r_bf16) {
                    // the stored sum is what the next layer adds to, so the norm is of
                    // the stored (rounded) sum
                    const uint4 u = pack_bf16(v[n]);
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.Rout) + t * p.ldro + i) = u;
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[n][2 * j] = __uint_as_float(w[j] << 16);
                        v[n][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                    }
                } else {
                    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p.Rout) + t * p.ldro + i);
                    q[0] = make_float4(v[n][0], v[n][1], v[n][2], v[n][3]);
                    q[1] = make_float4(v[n][4], v[n][5], v[n][6], v[n][7]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[n][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[n][j], v[n][j], ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) ss += part[w];
    const float rstd = 1.0f / sqrtf(ss / (float)p.D + p.eps);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int i = (n * kThreads + threadIdx.x) * 8;
        const bool in = i < p.D;
        float g[8];
        if (in) load8(p.G, i, p.g_bf16, g);
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[n][j] = in ? v[n][j] * rstd * g[j] : 0.f;
            amax = max_nan(amax, fabsf(v[n][j]));
        }
        if (p.Y && in) *reinterpret_cast<uint4*>(p.Y + t * p.D + i) = pack_bf16(v[n]);
        if constexpr (!Q81) {
            amax = lanes_max<16>(amax);
            const float s = amax / 448.0f;
            const GroupScale gs = group_scale(s);
            if (in) {
                uint2 q;
                q.x = e4m3x4(gs(v[n][0]), gs(v[n][1]), gs(v[n][2]), gs(v[n][3]));
                q.y = e4m3x4(gs(v[n][4]), gs(v[n][5]), gs(v[n][6]), gs(v[n][7]));
                *reinterpret_cast<uint2*>(p.Q + t * p.D + i) = q;
                if ((lane & 15) == 0) p.S[t * ((p.D + 127) / 128) + i / 128] = s;
            }
        } else {
            amax = lanes_max<4>(amax);
            const float d = amax / 127.0f;
            const GroupScale gs = group_scale(d);
            int q[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q[j] = (int)fminf(fmaxf(roundf(gs(v[n][j])), -127.f), 127.f);
                sum += q[j];
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (in) {
                uint2 u;
                u.x = (q[0] & 255) | ((q[1] & 255) << 8) | ((q[2] & 255) << 16) | ((uint32_t)q[3] << 24);
                u.y = (q[4] & 255) | ((q[5] & 255) << 8) | ((q[6] & 255) << 16) | ((uint32_t)q[7] << 24);
                *reinterpret_cast<uint2*>(p.Q + t * p.D + i) = u;
                if ((lane & 3) == 0) {
                    const long b = t * (p.D / 32) + i / 32;
                    p.Yd[b] = __float2half_rn(d);
                    p.Ys[b] = __float2half_rn(d * (float)sum);
                }
            }
        }
    }
}

template <bool Q81>
cudaError_t launch(const NormParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {overlap_attribute()};
    cfg.gridDim = dim3(p.T, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int nv = (p.D + kThreads * 8 - 1) / (kThreads * 8);
    if (nv <= 1) return cudaLaunchKernelEx(&cfg, rmsnorm8_kernel<Q81, 1>, p);
    if (nv <= 2) return cudaLaunchKernelEx(&cfg, rmsnorm8_kernel<Q81, 2>, p);
    if (nv <= 4) return cudaLaunchKernelEx(&cfg, rmsnorm8_kernel<Q81, 4>, p);
    return cudaLaunchKernelEx(&cfg, rmsnorm8_kernel<Q81, 8>, p);
}

}  // namespace

int rmsnorm8_max_width() { return kThreads * 8 * 8; }

cudaError_t launch_rmsnorm8(const NormParams& p, bool q81, cudaStream_t s) {
    return q81 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace qmm
