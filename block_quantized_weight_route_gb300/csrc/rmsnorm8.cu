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

__device__ __forceinline__ void load8(const void* p, long i, bool bf16, uint64_t (&v)[4]) {
    if (bf16) {
        unpack_bf16(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), v);
    } else {
        const ulonglong2* q = reinterpret_cast<const ulonglong2*>(static_cast<const float*>(p) + i);
        const ulonglong2 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
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

template <bool Q81, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : 1024) rmsnorm8_kernel(NormParams p) {
    __shared__ float part[32];
    launch_dependents();
    wait_prerequisites();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long t = WARP ? (long)blockIdx.x * kWarpRows + warp : (long)blockIdx.x;
    const int first = WARP ? lane : (int)threadIdx.x, step = WARP ? 32 : (int)blockDim.x;
    if (WARP && t >= p.T) return;
    uint64_t v[NV][4], r[NV][4], g[NV][4];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int i = (n * step + first) * 8;
        if (i < p.D) {
            load8(p.X, t * p.ldx + i, p.x_bf16, v[n]);
            if (p.R) load8(p.R, t * p.ldr + i, p.r_bf16, r[n]);
            load8(p.G, i, p.g_bf16, g[n]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[n][j] = r[n][j] = g[n][j] = 0;
        }
    }
    if (p.R) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int i = (n * step + first) * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[n][j] = add2(v[n][j], r[n][j]);
            if (p.r_bf16) {
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
        uint64_t y[4];
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = mul2(mul2(v[n][j], pack2(rstd, rstd)), g[n][j]);   // (0 past the row's end)
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
    if (vecs <= 128) {
        cfg.gridDim = dim3((p.T + kWarpRows - 1) / kWarpRows, 1, 1);
        cfg.blockDim = dim3(32 * kWarpRows, 1, 1);
        if (vecs <= 32) return cudaLaunchKernelEx(&cfg, rmsnorm8_kernel<Q81, 1, true>, p);
        if (vecs <= 64) return cudaLaunchKernelEx(&cfg, rmsnorm8_kernel<Q81, 2, true>, p);
        return cudaLaunchKernelEx(&cfg, rmsnorm8_kernel<Q81, 4, true>, p);
    }
    // one vector a thread while a CTA has the threads (two: 24 us against 20 at 2048 x 5120
    // bf16 with residual, 3.1 against 2.6 for one row; four: 32 and 5.7)
    const int nv = vecs <= 1024 ? 1 : 2;
    cfg.gridDim = dim3(p.T, 1, 1);
    cfg.blockDim = dim3(((vecs + nv - 1) / nv + 31) / 32 * 32, 1, 1);
    if (nv == 1) return cudaLaunchKernelEx(&cfg, rmsnorm8_kernel<Q81, 1, false>, p);
    return cudaLaunchKernelEx(&cfg, rmsnorm8_kernel<Q81, 2, false>, p);
}

}  // namespace

int rmsnorm8_max_width() { return 16384; }

cudaError_t launch_rmsnorm8(const NormParams& p, bool q81, cudaStream_t s) {
    return q81 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace qmm
