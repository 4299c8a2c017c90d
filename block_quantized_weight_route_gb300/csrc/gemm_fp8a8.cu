// FP8 x FP8 products with block scales (qmm_fp8a8_blk128, qmm_fp8a8_swiglu_blk128).
//
//   y[m][n] = sum_kb Xs[m][kb] S[n/128][kb] sum_{k in kb} e4m3(Xq[m][k]) e4m3(W[n][k])
//   h = silu(y gate) * y up, rounded to E4M3 per 128 columns
// One thread per output column and 16 tokens per CTA: the block's activations
// are converted to fp32 in shared memory and read as broadcasts, each thread
// reads its own weight row 16 bytes at a time.  fp32 throughout.
#include "qmm_internal.h"
#include "quant8.cuh"

namespace qmm {
namespace {

constexpr int kTok = 16;

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&f)[4]) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
    f[0] = fa.x, f[1] = fa.y, f[2] = fb.x, f[3] = fb.y;
}

// GATED: 256 threads, columns n0 + 0..127 of the gate rows and of the up rows;
// else 128 threads, columns n0 + 0..127.
template <bool GATED>
__global__ void __launch_bounds__(GATED ? 256 : 128) fp8a8_simple_kernel(Fp8a8Params p) {
    __shared__ float xs[kTok][128];
    __shared__ float ux[GATED ? 128 : 1][kTok + 1];
    __shared__ float wmax[4][kTok];
    constexpr int kThreads = GATED ? 256 : 128;
    const int n0 = blockIdx.x * 128, half = threadIdx.x >> 7, c = threadIdx.x & 127;
    const long m0 = (long)blockIdx.y * kTok;
    const int kbs = (p.K + 127) / 128;
    const bool col_ok = n0 + c < p.N;
    const long wrow = (GATED ? (long)half * p.N : 0) + n0 + (col_ok ? c : 0);   // gated: p.N = F
    const int nblk = (int)((GATED ? (long)half * p.N + n0 : (long)n0) / 128);
    float acc[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) acc[i] = 0.f;
    for (int kb = 0; kb < kbs; ++kb) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTok * 8; i += kThreads) {
            const int r = i >> 3, k = kb * 128 + (i & 7) * 16;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (m0 + r < p.M && k < p.K) v = *reinterpret_cast<const uint4*>(p.Xq + (m0 + r) * p.K + k);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[4];
                e4m3x4_to_f32(w[j], f);
                *reinterpret_cast<float4*>(&xs[r][(i & 7) * 16 + j * 4]) = make_float4(f[0], f[1], f[2], f[3]);
            }
        }
        __syncthreads();
        float part[kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) part[i] = 0.f;
        for (int k = 0; k < 128 && kb * 128 + k < p.K; k += 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(p.W + wrow * p.K + kb * 128 + k);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[4];
                e4m3x4_to_f32(w[j], f);
#pragma unroll
                for (int i = 0; i < kTok; ++i) {
                    const float4 x = *reinterpret_cast<const float4*>(&xs[i][k + j * 4]);
                    part[i] = fmaf(f[3], x.w, fmaf(f[2], x.z, fmaf(f[1], x.y, fmaf(f[0], x.x, part[i]))));
                }
            }
        }
        const float sw = p.S[(long)nblk * kbs + kb];
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (m0 + i < p.M) acc[i] = fmaf(part[i], p.Xs[(m0 + i) * kbs + kb] * sw, acc[i]);
    }
    if constexpr (!GATED) {
        if (col_ok) {
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                if (m0 + i >= p.M) break;
                const long o = (m0 + i) * p.N + n0 + c;
                if (p.y_bf16) static_cast<__nv_bfloat16*>(p.Y)[o] = __float2bfloat16_rn(acc[i]);
                else static_cast<float*>(p.Y)[o] = acc[i];
            }
        }
    } else {
        if (half == 1) {
#pragma unroll
            for (int i = 0; i < kTok; ++i) ux[c][i] = acc[i];
        }
        __syncthreads();
        if (half == 0) {
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                acc[i] = acc[i] / (1.0f + expf(-acc[i])) * ux[c][i];
                float a = fabsf(acc[i]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
                if ((c & 31) == 0) wmax[c >> 5][i] = a;
            }
        }
        __syncthreads();
        if (half == 0) {
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                if (m0 + i >= p.M) break;
                const float a = max_nan(max_nan(wmax[0][i], wmax[1][i]), max_nan(wmax[2][i], wmax[3][i]));
                const float s = a / 448.0f;
                const GroupScale gs = group_scale(s);
                p.Hq[(m0 + i) * p.N + n0 + c] = (uint8_t)__nv_cvt_float_to_fp8(gs(acc[i]), __NV_SATFINITE, __NV_E4M3);
                if (c == 0) p.Hs[(m0 + i) * (p.N / 128) + n0 / 128] = s;
            }
        }
    }
}

}  // namespace

// Columns of a prompt tile: the width whose waves of pairs take least, counting a
// wave as its width plus a fixed part for filling and draining the pipeline.
Fp8a8Plan fp8a8_plan(int M, int K, int N, bool gated, int sms) {
    (void)K;
    Fp8a8Plan pl{};
    if (M <= 64) return pl;
    pl.pair = true;
    pl.x_rows = 128;
    pl.bn = 256;
    if (!gated) {
        const long pairs = sms / 2, mt = (M + 255) / 256;
        double best = 1e30;
        for (int bn : {256, 192, 128}) {
            const long tiles = mt * ((N + bn - 1) / bn);
            const double cost = (double)((tiles + pairs - 1) / pairs) * (bn + 16);
            if (cost < best) {
                best = cost;
                pl.bn = bn;
            }
        }
    }
    pl.w_rows = pl.bn / 2;
    return pl;
}

cudaError_t launch_fp8a8(const Fp8a8Params& p, bool gated, cudaStream_t s) {
    const dim3 grid((p.N + 127) / 128, (p.M + kTok - 1) / kTok);
    if (gated) fp8a8_simple_kernel<true><<<grid, 256, 0, s>>>(p);
    else fp8a8_simple_kernel<false><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace qmm
