// Data movement of the FP8 expert stage: grouping of (token, expert) pairs by expert, the
// gather of the tokens' rows, and the weighted combine.
//
// Grouping: pair q = t * k + j with expert ids[q] takes row offsets[e] + its rank among the
// expert's pairs, in ascending q; pairs without an expert (ids[q] outside [0, E)) take none.
// The combine reads each expert's row once: 5268 tokens of 2048 columns and 8 experts 38 us (216 MB, 5.7 TB/s), 21504
// of 2560 188 us (5.9 TB/s), with the rows as fp16 in units (as fp32 they are twice the bytes: 55 us).
// Ranks come from counts of fixed pieces (a warp's 32 pairs, then chunks of 2048), never from
// atomic slot claims: the same rows every call, also where a token names an expert twice.
// (What an earlier kernel of the stage wrote is read by plain loads: launches overlap, and the
// non-coherent path could hold a line from before the wait.)
#include "ptx.cuh"
#include "qmm_internal.h"
#include "quant8.cuh"

#include <type_traits>

namespace qmm {
namespace {

constexpr int kThreads = 1024, kPieces = kMoeChunk / 32;   // pieces of 32 pairs in a chunk

// Pairs of each expert in each chunk.
__global__ void __launch_bounds__(kThreads) moe_count_kernel(const int32_t* ids, int P, int E, int32_t* chunk_counts) {
    __shared__ int32_t count[kMoeMaxExperts];
    launch_dependents();
    wait_prerequisites();
    for (int e = threadIdx.x; e < E; e += kThreads) count[e] = 0;
    __syncthreads();
    const long q0 = (long)blockIdx.x * kMoeChunk;
    for (int i = threadIdx.x; i < kMoeChunk; i += kThreads) {
        const int e = q0 + i < P ? ids[q0 + i] : -1;
        if ((unsigned)e < (unsigned)E) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) chunk_counts[(long)blockIdx.x * E + e] = count[e];
}

// Exclusive scan of one int a thread over the block.
__device__ int block_scan(int v, int* total) {
    __shared__ int warp_sums[kThreads / 32];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[wid] = x;
    __syncthreads();
    if (wid == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    *total = warp_sums[kThreads / 32 - 1];
    return (wid ? warp_sums[wid - 1] : 0) + x - v;
}

// One CTA a chunk: the rows of its pairs.  The first CTA writes what belongs to all of them:
// counts, offsets and the tiles of `tile_rows` rows.
__global__ void __launch_bounds__(kThreads) moe_rows_kernel(const int32_t* ids, int P, int E, int k, MoeGroups g) {
    extern __shared__ uint16_t piece[];   // [kPieces][E]: pairs of the expert in a piece, then in the pieces before it
    __shared__ int32_t first[kMoeMaxExperts];   // the chunk's first row of an expert
    __shared__ int32_t all_pairs[kMoeMaxExperts], earlier_pairs[kMoeMaxExperts];
    launch_dependents();
    wait_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long q0 = (long)blockIdx.x * kMoeChunk;
    const int n = (int)(P - q0 < kMoeChunk ? P - q0 : kMoeChunk), pieces = (n + 31) / 32;
    for (int i = threadIdx.x; i < (pieces * E + 1) / 2; i += kThreads) reinterpret_cast<uint32_t*>(piece)[i] = 0;
    __syncthreads();
    if (gridDim.x > 1 && !g.chunk_counts) {   // few chunks: each CTA counts them all
        for (int e = threadIdx.x; e < E; e += kThreads) all_pairs[e] = earlier_pairs[e] = 0;
        __syncthreads();
        for (long q = threadIdx.x; q < P; q += kThreads) {
            const int e = ids[q];
            if ((unsigned)e < (unsigned)E) {
                atomicAdd(&all_pairs[e], 1);
                if (q < q0) atomicAdd(&earlier_pairs[e], 1);
            }
        }
    }
    int mine[kMoeChunk / kThreads], rank[kMoeChunk / kThreads];
#pragma unroll
    for (int r = 0; r < kMoeChunk / kThreads; ++r) {
        const int i = r * kThreads + threadIdx.x;
        int e = i < n ? ids[q0 + i] : -1;
        if ((unsigned)e >= (unsigned)E) e = -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        mine[r] = e;
        rank[r] = __popc(same & ((1u << lane) - 1u));
        if (e >= 0 && rank[r] == 0) piece[(r * (kThreads / 32) + warp) * E + e] = (uint16_t)__popc(same);
    }
    __syncthreads();
    int total = 0, before = 0;   // the expert's pairs: all, and in earlier chunks
    const int e = threadIdx.x;
    if (e < E) {
        int run = 0;
        for (int i = 0; i < pieces; ++i) {
            const int v = piece[i * E + e];
            piece[i * E + e] = (uint16_t)run;
            run += v;
        }
        total = run;
        if (gridDim.x > 1 && !g.chunk_counts) {
            total = all_pairs[e];
            before = earlier_pairs[e];
        } else if (gridDim.x > 1) {
            total = 0;
#pragma unroll 8
            for (int c = 0; c < (int)gridDim.x; ++c) {
                const int v = g.chunk_counts[(long)c * E + e];
                before += c < (int)blockIdx.x ? v : 0;
                total += v;
            }
        }
    }
    int all;
    const int offset = block_scan(total, &all);
    if (e < E) first[e] = offset + before;
    if (blockIdx.x == 0) {
        const int tiles = (total + g.tile_rows - 1) / g.tile_rows;
        int num;
        const int t0 = block_scan(tiles, &num);
        if (e < E) {
            g.counts[e] = total;
            g.offsets[e] = offset;
            for (int i = 0; i < tiles; ++i)
                if (t0 + i < g.max_tiles)
                    g.tiles[t0 + i] = make_int4(e, offset + i * g.tile_rows, min(g.tile_rows, total - i * g.tile_rows), 0);
        }
        if (e == 0) {
            g.offsets[E] = all;
            *g.num_tiles = min(num, g.max_tiles);
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kMoeChunk / kThreads; ++r) {
        const int i = r * kThreads + threadIdx.x;
        if (i < n) {
            int at = -1;
            if (mine[r] >= 0) {
                at = first[mine[r]] + piece[(r * (kThreads / 32) + warp) * E + mine[r]] + rank[r];
                g.src[at] = (int32_t)((q0 + i) / k);
            }
            g.row[q0 + i] = at;
        }
    }
}

// Xp[r] = Xq[src[r]] and its scales: a warp a row.  For the kernel of many rows only, which takes its
// rows by one TMA copy: gathered there by TMA (32 copies of four rows a K block) they took the stage of
// 5268 tokens from 323 to 491 us.
__global__ void __launch_bounds__(256) moe_gather_kernel(const uint4* Xq, const float* Xs, const int32_t* src, const int32_t* rows,
                                                         int vecs, int kbs, uint4* Xp, float* Xps) {
    launch_dependents();
    wait_prerequisites();
    const int lane = threadIdx.x & 31, n = *rows;
    for (long r = (blockIdx.x * (long)blockDim.x + threadIdx.x) >> 5; r < n; r += (long)gridDim.x * blockDim.x >> 5) {
        const long t = src[r];
        const uint4* in = Xq + t * vecs;
        uint4* out = Xp + r * vecs;
        int i = lane;
        for (; i + 96 < vecs; i += 128) {   // four loads in flight a lane
            const uint4 a = in[i], b = in[i + 32], c = in[i + 64], d = in[i + 96];
            out[i] = a;
            out[i + 32] = b;
            out[i + 64] = c;
            out[i + 96] = d;
        }
        for (; i < vecs; i += 32) out[i] = in[i];
        for (int j = lane; j < kbs; j += 32) Xps[r * kbs + j] = Xs[t * kbs + j];
    }
}

// Y[t] = R[t] + sum_j w[t][j] y[row[t][j]], j ascending, in fp32; four columns a thread.
// HALF: y is fp16 in units of y_unit, one per 64 columns.  SPLIT: a block takes 256 threads' columns,
// and the grid's second dimension counts them; else a block takes its token's columns in turn.
template <int K, bool HALF, bool SPLIT>
__global__ void __launch_bounds__(256) moe_combine_kernel(const void* y, const float* y_unit, const int32_t* row, const float* w, int k,
                                                          int vecs, const void* R, int r_bf16, long ldr, void* Y, int y_bf16) {
    launch_dependents();
    wait_prerequisites();
    const long t = blockIdx.x;
    int rr[K];
    float ww[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        rr[j] = j < k ? row[t * k + j] : -1;
        ww[j] = j < k ? w[t * k + j] : 0.0f;
    }
    for (int i = SPLIT ? blockIdx.y * 256 + threadIdx.x : threadIdx.x; i < vecs; i += SPLIT ? vecs : 256) {
        using V = std::conditional_t<HALF, uint2, float4>;
        V v[K];
        float u[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (rr[j] >= 0) {
                v[j] = __ldcs(static_cast<const V*>(y) + (long)rr[j] * vecs + i);
                if constexpr (HALF) u[j] = y_unit[(long)rr[j] * ((vecs + 15) / 16) + i / 16];
            }
        }
        float4 a = R ? load4(R, r_bf16, t * ldr + i * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (rr[j] >= 0) {
                float4 f;
                float wj = ww[j];
                if constexpr (HALF) {
                    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&v[j].x)), hi = __half22float2(*reinterpret_cast<const __half2*>(&v[j].y));
                    f = make_float4(lo.x * u[j], lo.y * u[j], hi.x * u[j], hi.y * u[j]);   // (exact)
                } else {
                    f = v[j];
                }
                a.x = fmaf(wj, f.x, a.x);
                a.y = fmaf(wj, f.y, a.y);
                a.z = fmaf(wj, f.z, a.z);
                a.w = fmaf(wj, f.w, a.w);
            }
        }
        store4(Y, y_bf16, (t * vecs + i) * 4, a);
    }
}

template <class A>
struct Same {   // (an argument converts to the kernel's type)
    using type = A;
};
template <class... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, typename Same<A>::type... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {overlap_attribute()};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_moe_group(const int32_t* ids, int P, int E, int k, const MoeGroups& g, int dev, cudaStream_t s) {
    static PerDevice ready;
    if (!ready.get(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(moe_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kPieces * kMoeMaxExperts * 2);
        if (e != cudaSuccess) return e;
        ready.set(dev, 1);
    }
    const int chunks = (P + kMoeChunk - 1) / kMoeChunk;
    // (up to eight chunks a launch that counts them costs more than each CTA counting all)
    MoeGroups groups = g;
    if (chunks <= 8) groups.chunk_counts = nullptr;
    if (chunks > 8) {
        const cudaError_t e = launch(moe_count_kernel, chunks, kThreads, 0, s, ids, P, E, g.chunk_counts);
        if (e != cudaSuccess) return e;
    }
    const int pieces = P < kMoeChunk ? (P + 31) / 32 : kPieces;
    return launch(moe_rows_kernel, chunks, kThreads, ((size_t)pieces * E * 2 + 3) / 4 * 4, s, ids, P, E, k, groups);
}

cudaError_t launch_moe_gather(const uint8_t* Xq, const float* Xs, int P, int D, const MoeGroups& g, int E, uint8_t* Xp, float* Xps,
                              int sms, cudaStream_t s) {
    const long ctas = ((long)P + 7) / 8, most = (long)sms * 8;
    return launch(moe_gather_kernel, (unsigned)(ctas < most ? ctas : most), 256, 0, s, reinterpret_cast<const uint4*>(Xq), Xs, g.src,
                  g.offsets + E, D / 16, (D + 127) / 128, reinterpret_cast<uint4*>(Xp), Xps);
}

template <bool HALF, bool SPLIT>
static cudaError_t combine(const void* y, const float* y_unit, const int32_t* row, const float* w, int T, int k, int D, const void* R,
                           int r_bf16, long ldr, void* Y, int y_bf16, cudaStream_t s) {
    const auto kernel = k <= 2   ? moe_combine_kernel<2, HALF, SPLIT>
                        : k <= 4 ? moe_combine_kernel<4, HALF, SPLIT>
                        : k <= 8 ? moe_combine_kernel<8, HALF, SPLIT>
                                 : moe_combine_kernel<16, HALF, SPLIT>;
    return launch(kernel, dim3(T, SPLIT ? (D / 4 + 255) / 256 : 1, 1), 256, 0, s, y, y_unit, row, w, k, D / 4, R, r_bf16, ldr, Y, y_bf16);
}

cudaError_t launch_moe_combine(const void* y, const float* y_unit, const int32_t* row, const float* w, int T, int k, int D, const void* R,
                               int r_bf16, long ldr, void* Y, int y_bf16, int sms, cudaStream_t s) {
    // Where a block to a token would not fill the device (eight to an SM), its columns go to more
    // blocks: one after another their loads would be waited for in turn (a stage of 32 tokens 107.2 ->
    // 104.5 us, 301 tokens 130.3 -> 127.6).  With more tokens a block reads its rows' numbers once
    // (21504 tokens 1671 us, 1684 split).
    if (moe_combine_splits(T, sms))
        return y_unit ? combine<true, true>(y, y_unit, row, w, T, k, D, R, r_bf16, ldr, Y, y_bf16, s)
                      : combine<false, true>(y, nullptr, row, w, T, k, D, R, r_bf16, ldr, Y, y_bf16, s);
    return y_unit ? combine<true, false>(y, y_unit, row, w, T, k, D, R, r_bf16, ldr, Y, y_bf16, s)
                  : combine<false, false>(y, nullptr, row, w, T, k, D, R, r_bf16, ldr, Y, y_bf16, s);
}

}  // namespace qmm
