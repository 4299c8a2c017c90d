// Pieces shared by the FP8 x FP8 kernels: the E4M3 MMA, pair copies, packed fp32
// arithmetic, output stores and the SwiGLU.
#pragma once
#include "ptx.cuh"
#include "qmm_internal.h"
#include "quant8.cuh"

namespace qmm {

// Instruction descriptor, kind::f8f6f4: D f32, A and B E4M3, both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// As tc_mma_f16_pair, kind::f8f6f4 (K = 32 per instruction).
__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// As tma_load_2d into this CTA's shared memory, completing on the mbarrier at
// `bar`'s offset in the even CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
    asm volatile(
        "{\n\t.reg .b32 ra;\n\t"
        "mapa.shared::cluster.u32 ra, %4, 0;\n\t"
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [ra];"
        "\n\t}" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// Two fp32 values in one 64-bit register, and their packed multiply-add.
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) { return pack2u(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Wait (bounded) for the completion of the `issued` most recent fills of a ring.
__device__ __forceinline__ void drain_ring(uint64_t* full, long issued, int stages, uint32_t* err) {
    const long pending = issued < stages ? issued : stages;
    for (long i = 0; i < pending; ++i) {
        const long idx = issued - 1 - i;
        const int s = (int)(idx % stages);
        const uint32_t par = (uint32_t)((idx / stages) & 1);
        if (mbar_try_wait(&full[s], par)) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&full[s], par)) {
            if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
                atomicCAS(err, 0u, DEV_TIMEOUT_DRAIN);
                break;
            }
        }
    }
}

// silu(g) * u = g / (1 + exp(-g)) * u, from t = exp(-|g|) <= 1 so that neither the
// exponential nor the fast division (a few ulp) leaves its range: g / (1 + t), or
// g t / (1 + t) for negative g.  NaN and the formula's NaN at -inf pass.
__device__ __forceinline__ float swiglu(float g, float u) {
    const float t = __expf(-fabsf(g));
    return __fdividef(g < 0.0f ? g * t : g, 1.0f + t) * u;
}

// First column, inside the tile, of 32-column chunk c of a fold thread of half hf:
// consecutive columns, or (gated) chunks 0, 1 gate and 2, 3 the same columns of up.
template <class C>
__device__ __forceinline__ int chunk_col(int hf, int c) {
    if constexpr (C::GATED) return (c < 2 ? 0 : 128) + hf * 64 + (c & 1) * 32;
    else return hf * (C::BN / 2) + c * 32;
}

// 32 consecutive outputs of one row, as 16-byte vectors where the row pitch
// allows, masked at the last column.
__device__ __forceinline__ void store_chunk(const Fp8a8Params& p, long grow, int col, const uint64_t (&v)[16]) {
    const long o = grow * p.N + col;
    const bool whole = col + 32 <= p.N;
    if (p.y_bf16) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.Y) + o;
        if (whole && (p.N & 7) == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2(v[4 * j + i]);
                    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
                    w[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
                reinterpret_cast<uint4*>(dst)[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float2 f = unpack2(v[j]);
                if (col + 2 * j < p.N) dst[2 * j] = __float2bfloat16_rn(f.x);
                if (col + 2 * j + 1 < p.N) dst[2 * j + 1] = __float2bfloat16_rn(f.y);
            }
        }
    } else {
        float* dst = static_cast<float*>(p.Y) + o;
        if (whole && (p.N & 3) == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 a = unpack2(v[2 * j]), b = unpack2(v[2 * j + 1]);
                reinterpret_cast<float4*>(dst)[j] = make_float4(a.x, a.y, b.x, b.y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float2 f = unpack2(v[j]);
                if (col + 2 * j < p.N) dst[2 * j] = f.x;
                if (col + 2 * j + 1 < p.N) dst[2 * j + 1] = f.y;
            }
        }
    }
}

}  // namespace qmm
