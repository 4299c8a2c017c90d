// FP8 x FP8 products with block scales, few tokens (decoding, short prompts).
//
//   y[m][n] = sum_kb Xs[m][kb] S[n/128][kb] P_kb[m][n],   P_kb = sum_{k in kb} Xq[m][k] W[n][k]
//   GATED: h = silu(y gate) * y up, rounded to E4M3 per 128 columns of a token
//
// With few tokens the weights' bytes are the work, so the operands are swapped: a CTA
// streams 128 weight rows (GATED: 128 gate and 128 up rows) through the M side of
// M = 128, N = TN MMAs, and TN tokens are the N side.  The K blocks are split over the
// CTAs of a cluster; each folds its blocks' P into fp32 sums in registers (lane = weight
// row, one register per token), writes them to its shared memory, and the cluster
// adds them up in rank order from each other's shared memory: one launch, no scratch,
// the same result every call.
//   warp 0: TMA producer   warp 1: MMA issuer   warp 2: scales (asynchronous copies)
//   warps 4..: fold, four warps for each 128 weight rows and 32 tokens
// With 128 tokens a tile (TOKENS_M) the tokens are the M side and the weights the N side:
// swapped, every fold thread reads every token's scale from shared memory, 512 cycles a
// K block for 128 tokens; with a token per lane it reads one.
// What bounds it: with a few tokens the weights' way from HBM once it flows (gate/up of one
// token, 178 MB: 28.4 us, 6.3 TB/s = 0.93 of a plain copy; of 64 33.4 us, of 100 34.4) and, for a
// single small matrix, the launch and the cluster's sum (5120 x 5120, 26 MB: 7.2 us,
// 3.6 TB/s; 6.0 where the weights are in L2); at 128 tokens a tile shared memory (32 KB
// written and read a K block, 0.27 of the 0.30 us it takes; 300 x 5120 x 5120: 16.7 us).
#include "fp8a8.cuh"

namespace qmm {
namespace {

template <int TN_, bool GATED_>
struct NarrowCfg {
    static constexpr int TN = TN_, MATS = GATED_ ? 2 : 1;
    static constexpr bool GATED = GATED_, TOKENS_M = TN == 128;
    static constexpr int W_BYTES = MATS * 128 * 128, X_BYTES = TN * 128, STAGE_BYTES = W_BYTES + X_BYTES;
    // Two CTAs on an SM where a stage (and a fold thread) is small: one's start and end run beside the other's
    // stream, and a product of few tiles is split over more CTAs (one token, 5120 x 5120:
    // 7.2 us over 240 CTAs, 8.0 over 120; one CTA with twice the stages 5% slower still)
    static constexpr int PER_SM = TN * MATS <= 32 ? 2 : 1;
    static constexpr int STAGES = (PER_SM == 2 ? 106496 : 196608) / STAGE_BYTES;
    static constexpr int ACC_COLS = TN * MATS;
    static constexpr int TMEM_COLS = ACC_COLS <= 32 ? 128 : ACC_COLS <= 64 ? 256 : 512;
    static constexpr int NBUF_RAW = TMEM_COLS / ACC_COLS, NBUF = NBUF_RAW < STAGES ? NBUF_RAW : (STAGES & ~1);
    static constexpr int SC_SLOTS = 4, SC_KB = 4, SC_PITCH = TN + 4, SC_FLOATS = SC_SLOTS * SC_KB * SC_PITCH;
    // fold warps: four (the lanes) x the matrices x token groups of at most 32
    static constexpr int CW = TN < 32 ? TN : 32, TG = TN / CW;
    static constexpr int FOLD_WARPS = TOKENS_M ? 16 : 4 * MATS * TG, THREADS = 128 + 32 * FOLD_WARPS;
    // 64 sums a thread (tokens on the M side, gate and up): more registers for the fold warps
    static constexpr bool REG_SPLIT = TOKENS_M && GATED;
    static constexpr int REGS_EVEN = 65536 / (THREADS * PER_SM) / 8 * 8, REGS = REGS_EVEN < 255 ? REGS_EVEN : 255;
    static constexpr int REGS_FOLD = 104, REGS_OTHER = 64;
    static_assert(!REG_SPLIT || REGS_FOLD * 32 * FOLD_WARPS + REGS_OTHER * 128 == REGS * THREADS, "register shares = launch registers");
    static constexpr int COPIES = MATS + 1;
    static_assert(COPIES * STAGES <= 32, "a lane per copy");
    static constexpr int BARS = 2 * STAGES + NBUF + 2 * SC_SLOTS + 1;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + SC_FLOATS * 4 + BARS * 8 + 64;
    static_assert(PER_SM * (SMEM + 1024) <= 233472 && PER_SM * TMEM_COLS <= 512, "shared memory and TMEM");
    static_assert(TN * 128 * 4 * MATS <= STAGES * STAGE_BYTES, "the sums fit the stages");
    static_assert(!TOKENS_M || SC_KB % NBUF == 0, "buffer = K block's place in its slot");
    static_assert(NBUF >= 1 && NBUF <= STAGES, "a stage's MMA barrier completes again only after its accumulator was read");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t local, int rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 ra;\n\t"
        "mapa.shared::cluster.u32 ra, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [ra];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(local), "r"(rank)
        : "memory");
    return v;
}

// Sum over the cluster's CTAs, in rank order, of four consecutive floats at `local`.
__device__ __forceinline__ float4 cluster_sum(uint32_t local, int cs) {
    float4 v = ld_cluster_f4(local, 0);
    for (int r = 1; r < cs; ++r) {
        const float4 x = ld_cluster_f4(local, r);
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
    }
    return v;
}

// The fold of a warp, weights on the M side: lane = weight row, `acc` the tokens.
template <class C>
__device__ __forceinline__ void fold_weights_m(const Fp8a8Params& p, int warp, int lane, int kb0, int kb1, uint32_t tmem_base,
                                               const float* sc, float* sums, uint64_t* done, uint64_t* acc_empty,
                                               uint64_t* sc_full, uint64_t* sc_empty, volatile int* abort_flag) {
    constexpr int LD = 16;   // columns of a TMEM load
    const int set = (warp - 4) >> 2, q = warp & 3, row = q * 32 + lane;
    const int mat = set % C::MATS, tg = set / C::MATS;
    const uint32_t lane_addr = tmem_base + ((uint32_t)(q * 32) << 16) + mat * C::TN + tg * C::CW;
    int st = 0, slot = 0, buf = 0;
    uint32_t ph = 0, sph = 0;
    bool ok = true;
    uint64_t acc[C::CW / 2];
#pragma unroll
    for (int j = 0; j < C::CW / 2; ++j) acc[j] = 0;
    for (int kb = kb0; kb < kb1 && ok; kb += C::SC_KB) {
        if (!mbar_wait(&sc_full[slot], sph, abort_flag, p.err, DEV_TIMEOUT_CONV)) break;
#pragma unroll
        for (int k = 0; k < C::SC_KB; ++k) {
            if (kb + k >= kb1) break;
            const float* scr = sc + (slot * C::SC_KB + k) * C::SC_PITCH;
            const float sw = scr[C::TN + mat];
            const uint64_t sw2 = pack2(sw, sw);
            const ulonglong2* sx = reinterpret_cast<const ulonglong2*>(scr + tg * C::CW);
            if (!mbar_wait(&done[st], ph, abort_flag, p.err, DEV_TIMEOUT_ACC)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t a0 = lane_addr + (uint32_t)(buf * C::ACC_COLS);
#pragma unroll
            for (int x = 0; x < C::CW; x += LD) {
                uint32_t r[LD];
                tmem_ld(a0 + x, r);
                tmem_ld_wait();
                if (x + LD == C::CW) {
                    // every column is in registers: the MMA may write the buffer again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[buf]);
                }
#pragma unroll
                for (int j = 0; j < LD / 4; ++j) {
                    const ulonglong2 s = sx[x / 4 + j];   // four tokens' scales
                    uint64_t& y0 = acc[x / 2 + 2 * j];
                    uint64_t& y1 = acc[x / 2 + 2 * j + 1];
                    y0 = fma2(pack2u(r[4 * j], r[4 * j + 1]), mul2(s.x, sw2), y0);
                    y1 = fma2(pack2u(r[4 * j + 2], r[4 * j + 3]), mul2(s.y, sw2), y1);
                }
            }
            if (++buf == C::NBUF) buf = 0;
            if (++st == C::STAGES) {
                st = 0;
                ph ^= 1u;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_empty[slot]);
        if (++slot == C::SC_SLOTS) {
            slot = 0;
            sph ^= 1u;
        }
    }
    // This warp saw the last K block's barrier: every MMA is complete, so every copy has
    // landed and been read, and the stages become the sums' buffer.  (After a time-out
    // the sums mean nothing.)
#pragma unroll
    for (int j = 0; j < C::CW / 2; ++j) {
        const float2 f = unpack2(acc[j]);
        float* dst = sums + (mat * C::TN + tg * C::CW + 2 * j) * 128 + row;
        dst[0] = f.x;
        dst[128] = f.y;
    }
}

// Tokens on the M side: lane = token, `acc` 32 weight rows (GATED: 32 gate, then 32 up).
template <class C>
__device__ __forceinline__ void fold_tokens_m(const Fp8a8Params& p, int warp, int lane, int kb0, int kb1, uint32_t tmem_base,
                                              const float* sc, float* sums, uint64_t* done, uint64_t* acc_empty,
                                              uint64_t* sc_full, uint64_t* sc_empty, volatile int* abort_flag) {
    constexpr int COLS = 32 * C::MATS, LD = C::GATED ? 16 : 32;   // sums of a thread; columns of a TMEM load
    const int q = warp & 3, cg = (warp - 4) >> 2, row = q * 32 + lane;
    const uint32_t lane_addr = tmem_base + ((uint32_t)(q * 32) << 16) + cg * 32;
    int st = 0, slot = 0;
    uint32_t ph = 0, sph = 0;
    bool ok = true;
    uint64_t acc[COLS / 2];
#pragma unroll
    for (int j = 0; j < COLS / 2; ++j) acc[j] = 0;
    for (int kb = kb0; kb < kb1 && ok; kb += C::SC_KB) {
        if (!mbar_wait(&sc_full[slot], sph, abort_flag, p.err, DEV_TIMEOUT_CONV)) break;
        const float* scr = sc + slot * C::SC_KB * C::SC_PITCH;
#pragma unroll
        for (int k = 0; k < C::SC_KB; ++k) {
            if (kb + k >= kb1) break;
            const float sx = scr[k * C::SC_PITCH + row], s0 = sx * scr[k * C::SC_PITCH + C::TN];
            const float s1 = C::GATED ? sx * scr[k * C::SC_PITCH + C::TN + 1] : s0;
            if (!mbar_wait(&done[st], ph, abort_flag, p.err, DEV_TIMEOUT_ACC)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int buf = k % C::NBUF;   // (SC_KB is a multiple of NBUF)
            const uint32_t a0 = lane_addr + (uint32_t)(buf * C::ACC_COLS);
#pragma unroll
            for (int x = 0; x < COLS; x += LD) {
                uint32_t r[LD];
                tmem_ld(a0 + (x / 32) * 128 + x % 32, r);
                tmem_ld_wait();
                if (x + LD == COLS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[buf]);
                }
                const float sf = x < 32 ? s0 : s1;
                const uint64_t s2 = pack2(sf, sf);
#pragma unroll
                for (int j = 0; j < LD / 2; ++j) acc[x / 2 + j] = fma2(pack2u(r[2 * j], r[2 * j + 1]), s2, acc[x / 2 + j]);
            }
            if (++st == C::STAGES) {
                st = 0;
                ph ^= 1u;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_empty[slot]);
        if (++slot == C::SC_SLOTS) {
            slot = 0;
            sph ^= 1u;
        }
    }
    // (the stages are free, as above)  16-byte chunk c of a token's row at c ^ (token % 32)
#pragma unroll
    for (int j = 0; j < COLS / 4; ++j) {
        const float2 a = unpack2(acc[2 * j]), b = unpack2(acc[2 * j + 1]);
        *reinterpret_cast<float4*>(sums + ((j / 8) * C::TN + row) * 128 + (((cg * 8 + j % 8) ^ lane) << 2)) = make_float4(a.x, a.y, b.x, b.y);
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS) __maxnreg__(C::REGS)
    fp8a8_narrow_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, Fp8a8Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stage = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* sums = reinterpret_cast<float*>(stage);               // afterwards: [mat][token][128 rows]
    float* sc = reinterpret_cast<float*>(stage + C::STAGES * C::STAGE_BYTES);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sc + C::SC_FLOATS);
    uint64_t* full = bars;
    uint64_t* done = full + C::STAGES;        // a stage's MMAs are complete: its operands are free, its P is in TMEM
    uint64_t* acc_empty = done + C::STAGES;
    uint64_t* sc_full = acc_empty + C::NBUF;
    uint64_t* sc_empty = sc_full + C::SC_SLOTS;
    uint64_t* drain = sc_empty + C::SC_SLOTS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&done[i], 1);
        }
        for (int i = 0; i < C::NBUF; ++i) mbar_init(&acc_empty[i], C::FOLD_WARPS);
        for (int i = 0; i < C::SC_SLOTS; ++i) {
            mbar_init(&sc_full[i], 32);
            mbar_init(&sc_empty[i], C::FOLD_WARPS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    const int cs = (int)gridDim.x, rank = (int)blockIdx.x;   // one cluster per row of the grid
    const int n0 = p.n_first + (int)blockIdx.y * 128, m0 = (int)blockIdx.z * C::TN;
    const int kbs = (p.K + 127) / 128;
    const int kb0 = (int)((long)rank * kbs / cs), kb1 = (int)((long)(rank + 1) * kbs / cs);
    if (warp == 0) {
        // The first stages' weights on their way to L2 while the kernel before may still run
        // (only a hint: whatever that kernel writes, the copies below read after it)
        const int kb = kb0 + lane / C::MATS, m = lane % C::MATS;
        if (lane < C::STAGES * C::MATS && kb < kb1) tma_prefetch_2d(&tmW, kb * 128, m * p.N + n0);
    }
    if (warp == 1) tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_prerequisites();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    if (warp >= 4) {
        if constexpr (C::REG_SPLIT) setmaxnreg_inc<C::REGS_FOLD>();
        if constexpr (C::TOKENS_M) fold_tokens_m<C>(p, warp, lane, kb0, kb1, tmem_base, sc, sums, done, acc_empty, sc_full, sc_empty, abort_flag);
        else fold_weights_m<C>(p, warp, lane, kb0, kb1, tmem_base, sc, sums, done, acc_empty, sc_full, sc_empty, abort_flag);
    } else {
        if constexpr (C::REG_SPLIT) setmaxnreg_dec<C::REGS_OTHER>();
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            int s = 0;
            uint32_t ph = 0;
            long issued = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                const bool got = mbar_wait(&done[s], ph ^ 1u, abort_flag, p.err, DEV_TIMEOUT_TMA_EMPTY);
                if (__any_sync(0xffffffffu, !got)) break;
                // one copy at a time executes per thread: each copy of a stage on its own lane
                const int c = lane - s * C::COPIES;
                if (c == 0) mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
                __syncwarp();
                uint8_t* dst = stage + s * C::STAGE_BYTES + c * 128 * 128;
                if (c >= 0 && c < C::MATS) tma_load_2d(dst, &tmW, &full[s], kb * 128, c * p.N + n0);
                else if (c == C::MATS) tma_load_2d(dst, &tmX, &full[s], kb * 128, m0);
                __syncwarp();
                ++issued;
                if (++s == C::STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (lane == 0) drain_ring(full, issued, C::STAGES, p.err);
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            // (In order: the fold's waits rely on a K block's MMAs completing after those of
            // the blocks before it.)
            const uint32_t st0 = smem_u32(stage);
            int s = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                const bool got = mbar_wait(&full[s], ph, abort_flag, p.err, DEV_TIMEOUT_TMA_FULL) &&
                                 mbar_wait(&acc_empty[buf], bph ^ 1u, abort_flag, p.err, DEV_TIMEOUT_ACC_EMPTY);
                if (__any_sync(0xffffffffu, !got)) break;
                tc_fence_after();
                const uint32_t sa = st0 + (uint32_t)(s * C::STAGE_BYTES);
                const uint64_t xd = smem_desc_sw128(sa + C::W_BYTES);
                const uint32_t d = tmem_base + (uint32_t)(buf * C::ACC_COLS);
                if (elect_one_sync()) {
                    if constexpr (C::TOKENS_M) {
                        const uint64_t wd = smem_desc_sw128(sa);
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 codes (32 bytes) per MMA
                            tc_mma_f8(d, xd + (uint64_t)(k * 2), wd + (uint64_t)(k * 2), idesc_e4m3(128, C::ACC_COLS), k > 0);
                    } else {
#pragma unroll
                        for (int m = 0; m < C::MATS; ++m) {
                            const uint64_t wd = smem_desc_sw128(sa + m * 128 * 128);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc_mma_f8(d + m * C::TN, wd + (uint64_t)(k * 2), xd + (uint64_t)(k * 2), idesc_e4m3(128, C::TN), k > 0);
                        }
                    }
                    tc_commit(&done[s]);
                }
                __syncwarp();
                if (++buf == C::NBUF) {
                    buf = 0;
                    bph ^= 1u;
                }
                if (++s == C::STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (elect_one_sync()) tc_commit(drain);
            __syncwarp();
            if (lane == 0) drain_ring(drain, 1, 1, p.err);
            __syncwarp();
        } else if (warp == 2) {
            // ------------------------------------------------------------ scales
            int slot = 0;
            uint32_t sph = 0;
            const long b0 = n0 / 128, b1 = (p.N + n0) / 128;   // weight blocks (gated: gate, up)
            for (int kb = kb0; kb < kb1; kb += C::SC_KB) {
                if (!mbar_wait(&sc_empty[slot], sph ^ 1u, abort_flag, p.err, DEV_TIMEOUT_CONV_EMPTY)) break;
                float* dst = sc + slot * C::SC_KB * C::SC_PITCH;
                for (int i = lane; i < C::SC_KB * C::TN; i += 32) {
                    const int k = i / C::TN, r = i % C::TN;
                    const bool in = kb + k < kb1 && m0 + r < p.M;
                    cp_async4(dst + k * C::SC_PITCH + r, in ? p.Xs + (long)(m0 + r) * kbs + kb + k : p.Xs, in);
                }
                if (lane < C::MATS * C::SC_KB) {
                    const int k = lane / C::MATS, m = lane % C::MATS;
                    const bool in = kb + k < kb1;
                    cp_async4(dst + k * C::SC_PITCH + C::TN + m, in ? p.S + (m ? b1 : b0) * kbs + kb + k : p.S, in);
                }
                cp_async_arrive(&sc_full[slot]);
                if (++slot == C::SC_SLOTS) {
                    slot = 0;
                    sph ^= 1u;
                }
            }
            cp_async_wait_all();
        }
    }

    __syncthreads();
    cluster_sync();   // every CTA's sums are in its shared memory
    for (int t = rank + cs * warp; t < C::TN && m0 + t < p.M; t += cs * (C::THREADS / 32)) {
        const long m = (long)m0 + t;
        const uint32_t a = smem_u32(sums + t * 128 + (C::TOKENS_M ? lane ^ (t & 31) : lane) * 4);
        const float4 y = cluster_sum(a, cs);
        const int n = n0 + lane * 4;
        if constexpr (!C::GATED) {
            const float v[4] = {y.x, y.y, y.z, y.w};
            if (p.y_bf16) {
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.Y) + m * p.N + n;
                if ((p.N & 3) == 0) {
                    if (n < p.N) {
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
                        *reinterpret_cast<uint2*>(dst) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + j < p.N) dst[j] = __float2bfloat16_rn(v[j]);
                }
            } else {
                float* dst = static_cast<float*>(p.Y) + m * p.N + n;
                if ((p.N & 3) == 0) {
                    if (n < p.N) *reinterpret_cast<float4*>(dst) = y;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + j < p.N) dst[j] = v[j];
                }
            }
        } else {
            const float4 u = cluster_sum(a + C::TN * 512, cs);
            const float h[4] = {swiglu(y.x, u.x), swiglu(y.y, u.y), swiglu(y.z, u.z), swiglu(y.w, u.w)};
            float top = max_nan_abs(max_nan_abs(h[0], h[1], h[2]), h[3], 0.0f);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            const GroupScale gs = group_scale<448>(top);
            *reinterpret_cast<uint32_t*>(p.Hq + m * p.N + n) = e4m3x4(gs(h[0]), gs(h[1]), gs(h[2]), gs(h[3]));
            if (lane == 0) p.Hs[m * (p.N / 128) + n0 / 128] = gs.s;
        }
    }
    cluster_sync();   // no CTA leaves while another may read its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// One-time set-up on device `dev` (the current one).
template <class C>
cudaError_t prepare(int dev) {
    static PerDevice ready;
    if (!ready.get(dev)) {
        cudaError_t e = cudaFuncSetAttribute(fp8a8_narrow_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if constexpr (C::REG_SPLIT) {
            // the warpgroups' shares add up to the launch's registers: launch only if the
            // kernel is allocated exactly that many (a setmaxnreg.inc past the pool waits)
            cudaFuncAttributes fa{};
            e = cudaFuncGetAttributes(&fa, fp8a8_narrow_kernel<C>);
            if (e != cudaSuccess) return e;
            if (fa.numRegs != C::REGS) return cudaErrorInvalidConfiguration;
        }
        ready.set(dev, 1);
    }
    return cudaSuccess;
}

template <class C>
cudaError_t launch(const CUtensorMap& tx, const CUtensorMap& tw, const Fp8a8Params& p, int cs, int dev, cudaStream_t s) {
    const cudaError_t e = prepare<C>(dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1] = overlap_attribute();
    cfg.gridDim = dim3(cs, (p.n_end - p.n_first + 127) / 128, (p.M + C::TN - 1) / C::TN);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fp8a8_narrow_kernel<C>, tx, tw, p);
}

}  // namespace

namespace {

template <class C>
cudaError_t clusters_at_once(int cs, int dev, int* clusters) {
    static PerDevice at_once[9];   // by cs
    if (at_once[cs].get(dev) == 0) {
        cudaError_t e = prepare<C>(dev);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cs;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(cs, 64, 1);
        cfg.blockDim = dim3(C::THREADS, 1, 1);
        cfg.dynamicSmemBytes = C::SMEM;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, fp8a8_narrow_kernel<C>, &cfg);
        if (e != cudaSuccess) return e;
        // (the query counts one CTA per SM for a kernel that allocates TMEM; two whose shared
        // memory, registers and TMEM fit do run side by side: one token, 5120 x 5120, takes 7.2 us
        // over 240 CTAs, and 12.9 over 280, where a second wave begins)
        at_once[cs].set(dev, n * C::PER_SM);
    }
    *clusters = at_once[cs].get(dev);
    return cudaSuccess;
}

// f(configuration) for the kernel of tn tokens a tile
template <class F>
auto with_config(bool gated, int tn, F f) {
    if (gated) {
        if (tn == 16) return f(NarrowCfg<16, true>{});
        if (tn == 32) return f(NarrowCfg<32, true>{});
        if (tn == 64) return f(NarrowCfg<64, true>{});
        return f(NarrowCfg<128, true>{});
    }
    if (tn == 16) return f(NarrowCfg<16, false>{});
    if (tn == 32) return f(NarrowCfg<32, false>{});
    if (tn == 64) return f(NarrowCfg<64, false>{});
    return f(NarrowCfg<128, false>{});
}

}  // namespace

// (A cluster's CTAs are on SMs of one group of SMs, so fewer fit than slots / cs.)
cudaError_t fp8a8_narrow_at_once(bool gated, int tn, int cs, int dev, int* clusters) {
    return with_config(gated, tn, [&](auto c) { return clusters_at_once<decltype(c)>(cs, dev, clusters); });
}

cudaError_t launch_fp8a8_narrow(const CUtensorMap& tx, const CUtensorMap& tw, const Fp8a8Params& p, bool gated, int tn,
                                int cs, int dev, cudaStream_t s) {
    return with_config(gated, tn, [&](auto c) { return launch<decltype(c)>(tx, tw, p, cs, dev, s); });
}

}  // namespace qmm
