// Pieces shared by the FP8 x FP8 kernels: the E4M3 MMA, pair copies, TMEM loads, the
// SwiGLU and the output stores.  (Packed fp32 arithmetic: quant8.cuh.)
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

// Arrive once on the mbarrier at `bar`'s offset in the even CTA of the pair, after
// this thread's TMEM reads (complete at tcgen05.wait::ld, ordered by
// tcgen05.fence::before_thread_sync).  No shared or global memory is handed over,
// so the release is at CTA scope: a cluster-scope release took about 1200 cycles
// per hand-over (it made the kernel 1.8 times as slow at 2048 x 5120 x 5120).
// crank: this CTA's rank; the even CTA arrives without the detour over the cluster.
__device__ __forceinline__ void mbar_arrive_even(uint64_t* bar, int crank) {
    asm volatile(
        "{\n\t.reg .b32 ra;\n\t.reg .pred p;\n\t"
        "setp.eq.s32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t"
        "@!p mapa.shared::cluster.u32 ra, %0, 0;\n\t"
        "@!p mbarrier.arrive.shared::cluster.b64 _, [ra];\n\t}" ::"r"(smem_u32(bar)),
        "r"(crank)
        : "memory");
}

// As tc_mma_f16, kind::f8f6f4.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
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

// 32 lanes x 64, 32, 16 or 8 consecutive 32-bit TMEM columns.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Prefetch of a box into L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

// Four rows of 128 bytes, each a row of its own (the map's box is one row high), to four consecutive rows.
__device__ __forceinline__ void tma_gather4(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, const int (&y)[4]) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
            smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(smem_u32(bar))
        : "memory");
}

// A box of shared memory to global memory, in this thread's bulk group; and the wait until its
// groups have been read from shared memory, or are complete.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* smem_src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(smem_src)), "r"(x), "r"(y)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

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

// Two at once: the two quotients share one reciprocal, 1 / (d0 d1) with d = 1 + t in [1, 2] (the
// reciprocals and exponentials are what bounds a tile's SwiGLU: 8 cycles each a warp).
__device__ __forceinline__ uint64_t swiglu2(uint64_t g2, uint64_t u2) {
    const float2 g = unpack2(g2);
    const float t0 = __expf(-fabsf(g.x)), t1 = __expf(-fabsf(g.y));
    const float d0 = 1.0f + t0, d1 = 1.0f + t1;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d0 * d1));
    // (u last: g u may be past the largest number where h is not)
    const uint64_t n = mul2(g2, pack2(g.x < 0.0f ? t0 : 1.0f, g.y < 0.0f ? t1 : 1.0f));
    return mul2(mul2(n, mul2(pack2(r, r), pack2(d1, d0))), u2);
}

// The activations of the product's epilogue (qmm_act's order).  silu and tanh's gelu are v times
// the logistic function of z: with t = exp(-|z|) <= 1, v / (1 + t), or v t / (1 + t) for negative
// z: nothing overflows or cancels.  erf's gelu is v times the normal distribution, whose tail is
// Phi(-x) = q(r) exp(-x^2 / 2), r = 1 / (1 + 5/16 x): q is r times a polynomial of degree 7 fitted to
// Phi(-x) exp(x^2 / 2) so that its largest relative error on 0 <= x <= 14.4 (where v Phi(v) leaves 32 bits) is
// least, 2.3e-7 with the coefficients in fp32 (found by linear programming at 1200 Chebyshev points).  So
// a small negative result keeps its bits too; a formula within an absolute bound on erf would not do (one
// of degree 5 within 1.5e-7 was 1e-2 off at v = -8).
// Errors relative to the result, in units of 2^-24, for exact v: silu 16 + 3 |v|, gelu_tanh 16 + 9 |z| with
// z = 2 sqrt(2 / pi) (v + 0.044715 v^3), gelu 32 + 2 v^2.  The first part is the reciprocals and products, the other
// the exponential's argument: __expf is within 2 + 1.173 |argument| units of 2^-23, its rounded argument adds
// the rest.  (An error of half a unit in v itself changes the results by as much.)
// Columns n and n + 1 (n even) share a reciprocal, that of both denominators' product.
// v or v t, and the denominator (finite also for a NaN or an infinity, which stay in their column)
__device__ __forceinline__ float act_parts(float v, int act, float* d) {
    if (act == 3) {
        *d = fminf(fmaf(0.3125f, fabsf(v), 1.0f), 1e18f);
        return v;
    }
    const float z = act == 2 ? v : 1.5957691216f * v * fmaf(0.044715f * v, v, 1.0f);   // 2 sqrt(2 / pi) (v + 0.044715 v^3)
    const float t = fminf(__expf(-fabsf(z)), 1.0f);
    *d = 1.0f + t;
    return z < 0.0f ? v * t : v;
}
// The activation from these and the denominator's reciprocal.
__device__ __forceinline__ float act_finish(float x, float r, int act) {
    if (act != 3) return x * r;
    float q = fmaf(r, 0.0353278928f, -0.135801405f);
    q = fmaf(r, q, 0.140355065f);
    q = fmaf(r, q, -0.00452047074f);
    q = fmaf(r, q, 0.10540054f);
    q = fmaf(r, q, 0.109672867f);
    q = fmaf(r, q, 0.124903277f);
    q = r * fmaf(r, q, 0.124662347f);
    const float h = fminf(x, 1e18f) * (q * __expf(-0.5f * x * x));   // x Phi(-|x|)
    return x < 0.0f ? h : x - h;
}
__device__ __forceinline__ float reciprocal(float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}
template <int ACT>
__device__ __forceinline__ float4 activate4(float4 v) {
    float d[4];
    const float4 x = make_float4(act_parts(v.x, ACT, d), act_parts(v.y, ACT, d + 1), act_parts(v.z, ACT, d + 2), act_parts(v.w, ACT, d + 3));
    const float r = reciprocal(d[0] * d[1]), s = reciprocal(d[2] * d[3]);
    return make_float4(act_finish(x.x, r * d[1], ACT), act_finish(x.y, r * d[0], ACT), act_finish(x.z, s * d[3], ACT),
                       act_finish(x.w, s * d[2], ACT));
}
__device__ __forceinline__ float4 relu4(float4 v) {
    return make_float4(max_nan(v.x, 0.0f), max_nan(v.y, 0.0f), max_nan(v.z, 0.0f), max_nan(v.w, 0.0f));
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
// f(a function of four values) for the activation `act`
template <class F>
__device__ __forceinline__ void with_activation(int act, F f) {
    if (act == 0) f([](float4 v) { return v; });
    else if (act == 1) f([](float4 v) { return relu4(v); });
    else if (act == 2) f([](float4 v) { return activate4<2>(v); });
    else if (act == 3) f([](float4 v) { return activate4<3>(v); });
    else f([](float4 v) { return activate4<4>(v); });
}
// The same with a column a lane.
__device__ __forceinline__ float activate_lanes(float v, int act) {
    if (act == 0) return v;
    if (act == 1) return max_nan(v, 0.0f);
    float d;
    const float x = act_parts(v, act, &d), d2 = __shfl_xor_sync(0xffffffffu, d, 1);
    return act_finish(x, reciprocal(d * d2) * d2, act);
}

// The bias of columns n .. n + 3 and the residual of row m there (past the end zeros), and
// act(y + bias) + R.
__device__ __forceinline__ float4 epilogue_bias(const Fp8a8EpilogueParams& p, int n) {
    float b[4] = {};
    if (p.bias && p.vec4 && n < p.N) return load4(p.bias, p.bias_bf16, n);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (p.bias && n + j < p.N) b[j] = load1(p.bias, p.bias_bf16, n + j);
    return make_float4(b[0], b[1], b[2], b[3]);
}
__device__ __forceinline__ float4 epilogue_residual(const Fp8a8EpilogueParams& p, long m, int n) {
    float r[4] = {};
    if (p.R && p.vec4 && n < p.N) return load4(p.R, p.r_bf16, m * p.ldr + n);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (p.R && n + j < p.N) r[j] = load1(p.R, p.r_bf16, m * p.ldr + n + j);
    return make_float4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ float4 epilogue4(const Fp8a8EpilogueParams& p, float4 y, float4 b, float4 r) {
    y = add4(y, b);
    if (p.act) with_activation(p.act, [&](auto act) { y = act(y); });
    return add4(y, r);
}

// The column, inside the tile, of a fold thread's column i, for column group cq:
// consecutive columns, or (gated) half of them gate, then the same columns of up.
template <class C>
__device__ __forceinline__ int fold_col(int cq, int i) {
    if constexpr (C::GATED) return (i / (C::CW / 2)) * 128 + cq * (C::CW / 2) + i % (C::CW / 2);
    else return cq * C::CW + i;
}

// 4-byte asynchronous copy to shared memory, or a zero.
__device__ __forceinline__ void cp_async4(void* smem_dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(smem_dst)), "l"(src), "r"(in ? 4 : 0)
                 : "memory");
}
// One of the arrivals `bar` was initialised with, when this thread's copies so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Eight outputs as bf16.
__device__ __forceinline__ uint4 bf16x8(const uint64_t* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(v[i]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's staging for outputs: 32 rows x 128 bytes, 16-byte chunk c of row r at c ^ (r % 8) (no bank
// conflicts on either side).  Copied to Y at (row0, col): eight lanes to a row.
__device__ __forceinline__ void flush_aligned(const Fp8a8Base& p, const uint8_t* stg, int lane, long row0, int col, int esz) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + lane / 8, c = lane % 8;
        const uint4 d = *reinterpret_cast<const uint4*>(stg + (r * 8 + (c ^ (r & 7))) * 16);
        const int cc = col + c * (16 / esz);
        if (row0 + r < p.M && cc < p.N)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.Y) + ((row0 + r) * p.N + cc) * esz) = d;
    }
}

// A lane's 16 consecutive outputs (two per element of `v`) to its row of the staging, chunk c0 and on.
template <bool BF16>
__device__ __forceinline__ void stage16(uint8_t* stg, int lane, int c0, const uint64_t* v) {
#pragma unroll
    for (int c = 0; c < (BF16 ? 2 : 4); ++c) {
        uint4 d;
        if constexpr (BF16) {
            d = bf16x8(v + 4 * c);
        } else {
            const float2 a = unpack2(v[2 * c]), b = unpack2(v[2 * c + 1]);
            d = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
        }
        *reinterpret_cast<uint4*>(stg + (lane * 8 + ((c0 + c) ^ (lane & 7))) * 16) = d;
    }
}

// The same to rows of Y whose pitch is no multiple of 16 bytes: a row at a time, 4 bytes a lane.
// A row of bf16 that starts at an
// odd element (4-byte stores are aligned) is shifted by one; the first and the last
// element of such rows follow, a row per lane.
template <bool BF16, int UNROLL>
__device__ __forceinline__ void flush_ragged(const Fp8a8Base& p, const uint8_t* stg, int lane, long row0, int col) {
    const int rows = p.M - (int)row0 < 32 ? p.M - (int)row0 : 32, cols = p.N - col;
    auto word = [&](int r, int i) { return reinterpret_cast<const uint32_t*>(stg + (r * 8 + ((i / 4) ^ (r & 7))) * 16)[i % 4]; };
    if constexpr (!BF16) {
        if (lane >= cols) return;
        uint32_t* dst = static_cast<uint32_t*>(p.Y) + row0 * p.N + col + lane;
#pragma unroll UNROLL
        for (int r = 0; r < rows; ++r) dst[(long)r * p.N] = word(r, lane);
    } else {
        uint16_t* dst = static_cast<uint16_t*>(p.Y) + row0 * p.N + col;
#pragma unroll UNROLL
        for (int r = 0; r < rows; ++r) {
            const int odd = ((int)row0 + r) & p.N & 1, e = 2 * lane - odd;   // the lane's elements: e, e + 1
            uint32_t d = word(r, lane);
            if (odd) d = (d << 16) | (word(r, (lane + 31) & 31) >> 16);
            uint16_t* at = dst + (long)r * p.N + e;
            if (e >= 0 && e + 1 < cols) *reinterpret_cast<uint32_t*>(at) = d;
            else if (e >= 0 && e < cols) at[0] = (uint16_t)d;
        }
        if (lane < rows && (((int)row0 + lane) & p.N & 1)) {
            if (cols > 0) dst[(long)lane * p.N] = (uint16_t)word(lane, 0);
            if (cols > 63) dst[(long)lane * p.N + 63] = (uint16_t)(word(lane, 31) >> 16);
        }
    }
}

// A warp's 32 rows x 64 columns (lane = row, `v` its 64 consecutive outputs, two per element) to Y
// at (row0, col), through the warp's staging, so that a store instruction writes runs of 128
// bytes.  Runs of 32 (with 2 KB of staging) took 46 us instead of 34 at 5268 x 1024 x 5120,
// single elements in ragged rows 262 instead of 49 at 5268 x 1024 x 5119 (there a run's two
// ends are sectors written in part).  Ragged rows are copied UNROLL at a time, what the
// kernel's registers allow.
template <bool BF16, bool RAGGED, int UNROLL>
__device__ __forceinline__ void store_columns(const Fp8a8Base& p, uint8_t* stg, int lane, long row0, int col,
                                              const uint64_t* v) {
    constexpr int STEP = BF16 ? 64 : 32;
#pragma unroll
    for (int c = 0; c < 64; c += STEP) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < STEP; k += 16) stage16<BF16>(stg, lane, k * 8 / STEP, v + (c + k) / 2);
        __syncwarp();
        if constexpr (RAGGED) flush_ragged<BF16, UNROLL>(p, stg, lane, row0, col + c);
        else flush_aligned(p, stg, lane, row0, col + c, BF16 ? 2 : 4);
    }
}

// The epilogue's bias for a tile's BN columns, on its way to shared memory (in its type, past the end
// zeros), and the residual's rows of the tile on theirs to L2: by threads 0 .. THREADS - 1, while the tile's
// K blocks are folded.
template <int BN, int ROWS, int THREADS>
__device__ __forceinline__ void prefetch_epilogue(const Fp8a8EpilogueParams& p, float* bias, int thread, long row0, int col0) {
    if (p.bias) {
        const int esz = p.bias_bf16 ? 2 : 4;
        for (int x = thread * 16; x < BN * esz; x += THREADS * 16) {
            const int n = col0 + x / esz, left = (p.N - n) * esz, bytes = left < 0 ? 0 : left < 16 ? left : 16;
            const uint8_t* src = static_cast<const uint8_t*>(p.bias) + (bytes ? (long)n * esz : 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(reinterpret_cast<uint8_t*>(bias) + x)), "l"(src), "r"(bytes)
                         : "memory");
        }
    }
    if (p.R) {
        const int esz = p.r_bf16 ? 2 : 4, cols = p.N - col0 < BN ? p.N - col0 : BN;
        for (int r = thread; r < ROWS && row0 + r < p.M; r += THREADS) {
            const uint8_t* a = static_cast<const uint8_t*>(p.R) + ((row0 + r) * p.ldr + col0) * esz;
#pragma unroll 1
            for (int x = 0; x < cols * esz; x += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(a + x) : "memory");
        }
    }
}

// A lane's share of a part of 32 rows x 32 columns: four columns of eight rows, through `at(i)`, plus the bias
// and the residual, to Y.  RT: the residual's raw four elements (float4: fp32, uint2: bf16), or void.
// All eight residual loads and sums are in registers before the first store: R may be Y, and a store
// through a plain pointer could be to shared memory, so the compiler would not move them past it.
__device__ __forceinline__ float4 widen4(float4 v) { return v; }
__device__ __forceinline__ float4 widen4(uint2 w) {
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
template <bool BF16, class RT, class AT>
__device__ __forceinline__ void finish_part(const Fp8a8EpilogueParams& p, int lane, long row0, int n, float4 b, AT at) {
    const bool in = n < p.N;
    RT r[8];
    const int nn = in ? n : 0;   // (what is past the end reads an element that exists)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long m = row0 + i * 4 + lane / 8;
        r[i] = *reinterpret_cast<const RT*>(static_cast<const uint8_t*>(p.R) + ((m < p.M ? m : p.M - 1) * p.ldr + nn) * (sizeof(RT) / 4));
    }
    if (p.act) {
        with_activation(p.act, [&](auto act) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) *at(i) = act(add4(*at(i), b));
        });
        b = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float4 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = add4(add4(*at(i), b), widen4(r[i]));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long m = row0 + i * 4 + lane / 8;
        if (in && m < p.M) store4(p.Y, BF16, m * p.N + n, y[i]);
    }
}

// store_columns with the epilogue: CH columns at a time as fp32 through the staging (CH / 32 parts of 32 rows x
// 128 bytes), then, coalesced, the bias (`bias`, bias0 the warp's first column of it), the activation and the
// residual's rows, and the rounding.  VEC: eight lanes a row, four columns each; else a column a lane.
// The loops over the parts are not unrolled, nor the activation's (but for two at once with nothing behind it):
// the code, many times over, does not fit the instruction cache.
template <bool BF16, bool VEC, int COLS, int CH>
__device__ __forceinline__ void store_epilogue(const Fp8a8EpilogueParams& p, uint8_t* stg, const float* bias, int bias0, int lane, long row0, int col0,
                                               const uint64_t* v) {
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += CH) {
        __syncwarp();
#pragma unroll
        for (int h = 0; h < CH / 32; ++h) {
            stage16<false>(stg + h * 4096, lane, 0, v + (c0 + h * 32) / 2);
            stage16<false>(stg + h * 4096, lane, 4, v + (c0 + h * 32) / 2 + 8);
        }
        __syncwarp();
#pragma unroll 1
        for (int h = 0; h < CH / 32; ++h) {
            uint8_t* part = stg + h * 4096;
            if constexpr (VEC) {
                const int c = lane % 8, n = col0 + c0 + 32 * h + 4 * c;
                const float4 b = p.bias ? load4(bias, p.bias_bf16, bias0 + c0 + 32 * h + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
                auto at = [&](int i) {   // (this lane's alone)
                    const int q = i * 4 + lane / 8;
                    return reinterpret_cast<float4*>(part + (q * 8 + (c ^ (q & 7))) * 16);
                };
                if (!p.R) {
                    with_activation(p.act, [&](auto act) {
#pragma unroll 2
                        for (int i = 0; i < 8; ++i) {
                            const long m = row0 + i * 4 + lane / 8;
                            const float4 y = act(add4(*at(i), b));
                            if (n < p.N && m < p.M) store4(p.Y, BF16, m * p.N + n, y);
                        }
                    });
                } else if (p.r_bf16) {
                    finish_part<BF16, uint2>(p, lane, row0, n, b, at);
                } else {
                    finish_part<BF16, float4>(p, lane, row0, n, b, at);
                }
            } else {
                const int n = col0 + c0 + 32 * h + lane, rows = p.M - row0 < 32 ? (int)(p.M - row0) : 32;
                const bool in = n < p.N;
                const float b = p.bias ? load1(bias, p.bias_bf16, bias0 + c0 + 32 * h + lane) : 0.0f;
#pragma unroll 1
                for (int q0 = 0; q0 < rows; q0 += 8) {
                    float r[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = p.R && in && q0 + i < rows ? load1(p.R, p.r_bf16, (row0 + q0 + i) * p.ldr + n) : 0.0f;
#pragma unroll 4
                    for (int i = 0; p.act && i < 8; ++i) {   // (of 32 rows staged)
                        const int q = q0 + i;
                        float* at = reinterpret_cast<float*>(part + (q * 8 + ((lane / 4) ^ (q & 7))) * 16) + lane % 4;
                        *at = activate_lanes(*at + b, p.act);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int q = q0 + i;
                        r[i] += reinterpret_cast<const float*>(part + (q * 8 + ((lane / 4) ^ (q & 7))) * 16)[lane % 4] + (p.act ? 0.0f : b);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const long at = (row0 + q0 + i) * p.N + n;
                        if (in && q0 + i < rows) {
                            if constexpr (BF16) static_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(r[i]);
                            else static_cast<float*>(p.Y)[at] = r[i];
                        }
                    }
                }
            }
        }
    }
}

}  // namespace qmm
