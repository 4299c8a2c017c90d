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
__device__ __forceinline__ void flush_aligned(const Fp8a8Params& p, const uint8_t* stg, int lane, long row0, int col, int esz) {
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
__device__ __forceinline__ void flush_ragged(const Fp8a8Params& p, const uint8_t* stg, int lane, long row0, int col) {
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
__device__ __forceinline__ void store_columns(const Fp8a8Params& p, uint8_t* stg, int lane, long row0, int col,
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

}  // namespace qmm
