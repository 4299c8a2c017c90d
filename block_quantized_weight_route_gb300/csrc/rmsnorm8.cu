// Residual addition + RMS norm + output in 8 bits (qmm_add_rmsnorm_fp8,
// qmm_add_rmsnorm_q8_1).
//
//   v = x, or r' = x + r rounded to the residual's type and stored;
//   y = v / sqrt(mean(v^2) + eps) * g;  y in groups of 128 (E4M3) or 32 (q8_1).
// Everything between the loads and the stores is fp32.  Bandwidth bounds it: a row is
// read once and held in registers, NV vectors of 8 consecutive values a thread, all of
// whose loads (x, the residual and g) are issued before anything waits on them.  A CTA
// takes one row, or, for rows of at most 1024 values, each warp one.  16 (or 4)
// consecutive lanes hold one group, whose maximum is a few shuffles.
// Measured: 21504 x 2560, fp32 rows and residual, bf16 rows out beside the codes (830 MB)
// 118 us = 7.0 TB/s; all bf16 56 us = 7.0 TB/s; 2048 x 5120 bf16 (74 MB) 13.7 us = 5.4 TB/s;
// 5268 x 2048, fp32 rows, bf16 residual, q8_1 (98 MB) 17.4 us = 5.7 TB/s; one row 2 us,
// the launch.  Not kept: a persistent grid that loads the next row ahead (slower).
#include "qmm_internal.h"
#include "quant8.cuh"

namespace qmm {
namespace {

constexpr int kWarpRows = 8;   // rows of a CTA that gives each to a warp

// Eight consecutive values as four packed pairs.
__device__ __forceinline__ void unpack_bf16(const uint4& u, uint64_t (&v)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pack2u(w[j] << 16, w[j] & 0xFFFF0000u);
}

// Eight consecutive values as they lie in memory.  Turned into fp32 only when all of a
// thread's loads are on their way: with the conversion in the same branch as the load,
// the next load waits for it.
struct Raw8 {
    uint4 lo, hi;   // (bf16: lo only)
};

__device__ __forceinline__ Raw8 load8(const void* p, long i, bool bf16) {
    Raw8 u;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (bf16 ? 2 : 4));
    u.lo = q[0];
    u.hi = bf16 ? make_uint4(0, 0, 0, 0) : q[1];
    return u;
}

__device__ __forceinline__ void widen8(const Raw8& u, bool bf16, uint64_t (&v)[4]) {
    if (bf16) {
        unpack_bf16(u.lo, v);
    } else {
        v[0] = pack2u(u.lo.x, u.lo.y), v[1] = pack2u(u.lo.z, u.lo.w);
        v[2] = pack2u(u.hi.x, u.hi.y), v[3] = pack2u(u.hi.z, u.hi.w);
    }
}

__device__ __forceinline__ uint4 pack_bf16(const uint64_t (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2(v[j]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
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

// HALF: x, the residual and g are all bf16
template <bool Q81, int NV, bool WARP, bool HALF>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : HALF && NV > 1 ? 512 : 1024, !WARP && NV == 4 ? 2 : 0) rmsnorm8_kernel(NormParams p) {
    __shared__ float part[32];
    launch_dependents();
    wait_prerequisites();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long t = WARP ? (long)blockIdx.x * kWarpRows + warp : (long)blockIdx.x;
    const int first = WARP ? lane : (int)threadIdx.x, step = WARP ? 32 : (int)blockDim.x;
    if (WARP && t >= p.T) return;
    const Raw8 none = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    Raw8 vr[NV], rr[NV], gr[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int i = (n * step + first) * 8;
        vr[n] = rr[n] = gr[n] = none;
        if (i < p.D) {
            vr[n] = load8(p.X, t * p.ldx + i, HALF || p.x_bf16);
            if (p.R) rr[n] = load8(p.R, t * p.ldr + i, HALF || p.r_bf16);
            gr[n] = load8(p.G, i, HALF || p.g_bf16);
        }
    }
    uint64_t v[NV][4];
#pragma unroll
    for (int n = 0; n < NV; ++n) widen8(vr[n], HALF || p.x_bf16, v[n]);
    if (p.R) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int i = (n * step + first) * 8;
            uint64_t r[4];
            widen8(rr[n], HALF || p.r_bf16, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[n][j] = add2(v[n][j], r[j]);
            if (HALF || p.r_bf16) {
                // the stored sum is what the next layer adds to, so the norm is of the
                // stored (rounded) sum
                const uint4 u = pack_bf16(v[n]);
                if (i < p.D) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.Rout) + t * p.ldro + i) = u;
                unpack_bf16(u, v[n]);
            } else if (i < p.D) {
                ulonglong2* q = reinterpret_cast<ulonglong2*>(static_cast<float*>(p.Rout) + t * p.ldro + i);
                q[0] = make_ulonglong2(v[n][0], v[n][1]);
                q[1] = make_ulonglong2(v[n][2], v[n][3]);
            }
        }
    }
    uint64_t sq = 0;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) sq = fma2(v[n][j], v[n][j], sq);
    const float2 sq2 = unpack2(sq);
    float ss = sq2.x + sq2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if constexpr (!WARP) {
        if (lane == 0) part[warp] = ss;
        __syncthreads();
        ss = lane < (step >> 5) ? part[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float rstd = 1.0f / sqrtf(ss / (float)p.D + p.eps);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int i = (n * step + first) * 8;
        const bool in = i < p.D;
        uint64_t y[4], g[4];
        widen8(gr[n], HALF || p.g_bf16, g);
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = mul2(mul2(v[n][j], pack2(rstd, rstd)), g[j]);   // (0 past the row's end)
            const float2 h = unpack2(y[j]);
            f[2 * j] = h.x, f[2 * j + 1] = h.y;
        }
        if (p.Y && in) *reinterpret_cast<uint4*>(p.Y + t * p.D + i) = pack_bf16(y);
        float top = max_nan_abs(max_nan_abs(f[0], f[1], f[2]), f[3], f[4]);
        top = max_nan_abs(max_nan_abs(top, f[5], f[6]), f[7], 0.0f);
        top = lanes_max<Q81 ? 4 : 16>(top);
        const GroupScale gs = group_scale<Q81 ? 127 : 448>(top);
        if (gs.tiny()) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], pack2(gs.up, gs.up));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 h = unpack2(mul2(y[j], pack2(gs.inv, gs.inv)));
            f[2 * j] = h.x, f[2 * j + 1] = h.y;
        }
        if constexpr (!Q81) {
            if (in) {
                *reinterpret_cast<uint2*>(p.Q + t * p.D + i) =
                    make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
                if ((lane & 15) == 0) p.S[t * ((p.D + 127) / 128) + i / 128] = gs.s;
            }
        } else {
            int q[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q[j] = (int)fminf(fmaxf(roundf(f[j]), -127.f), 127.f);
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
                    p.Yd[b] = __float2half_rn(gs.s);
                    p.Ys[b] = __float2half_rn(gs.s * (float)sum);
                }
            }
        }
    }
}

template <bool Q81>
cudaError_t launch(const NormParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {overlap_attribute()};
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int vecs = (p.D + 7) / 8;
    const bool half = p.x_bf16 && p.g_bf16 && (!p.R || p.r_bf16);
    if (vecs <= 128) {
        cfg.gridDim = dim3((p.T + kWarpRows - 1) / kWarpRows, 1, 1);
        cfg.blockDim = dim3(32 * kWarpRows, 1, 1);
        if (vecs <= 32) return cudaLaunchKernelEx(&cfg, half ? rmsnorm8_kernel<Q81, 1, true, true> : rmsnorm8_kernel<Q81, 1, true, false>, p);
        if (vecs <= 64) return cudaLaunchKernelEx(&cfg, half ? rmsnorm8_kernel<Q81, 2, true, true> : rmsnorm8_kernel<Q81, 2, true, false>, p);
        return cudaLaunchKernelEx(&cfg, half ? rmsnorm8_kernel<Q81, 4, true, true> : rmsnorm8_kernel<Q81, 4, true, false>, p);
    }
    // What is in flight on an SM sets the bandwidth: bf16 vectors are half as large and their
    // kernel needs fewer registers, so a thread takes two (21504 x 2560: 56 us against 63 with
    // one; one row 0.1 us more), above 8192 four (4096 x 16384: 73 us against 87 with two);
    // fp32 vectors one, above 8192 two
    const int nv = half ? (vecs <= 1024 ? 2 : 4) : vecs <= 1024 ? 1 : 2;
    cfg.gridDim = dim3(p.T, 1, 1);
    cfg.blockDim = dim3(((vecs + nv - 1) / nv + 31) / 32 * 32, 1, 1);
    if (half) return cudaLaunchKernelEx(&cfg, nv == 2 ? rmsnorm8_kernel<Q81, 2, false, true> : rmsnorm8_kernel<Q81, 4, false, true>, p);
    return cudaLaunchKernelEx(&cfg, nv == 1 ? rmsnorm8_kernel<Q81, 1, false, false> : rmsnorm8_kernel<Q81, 2, false, false>, p);
}

}  // namespace

int rmsnorm8_max_width() { return 16384; }

cudaError_t launch_rmsnorm8(const NormParams& p, bool q81, cudaStream_t s) {
    return q81 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace qmm
