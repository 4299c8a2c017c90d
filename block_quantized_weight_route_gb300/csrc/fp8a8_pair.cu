// FP8 x FP8 products with block scales, prompt form (many tokens).
//
//   y[m][n] = sum_kb Xs[m][kb] S[n/128][kb] P_kb[m][n],   P_kb = sum_{k in kb} Xq[m][k] W[n][k]
//   GATED: h = silu(y gate) * y up, rounded to E4M3 per 128 columns of a token
//
// Persistent CTA pairs (cta_group::2), each on one 256 x BN tile: the even CTA
// issues M = 256, N = BN, K = 32 MMAs over both CTAs' shared memory, each CTA's
// TMEM holds its 128 rows x BN columns of P_kb.  A block's sum cannot stay in the
// tensor core (its scale differs by row and by block), so the fold warps take each
// P_kb out of TMEM into fp32 running sums in registers, two or four TMEM buffers
// apart from the MMA.
//   warp 0: TMA producer   warp 1: MMA issuer (even CTA)
//   warps 2, 3: the scales of four or eight K blocks at a time, by asynchronous copies into a ring
//   warps 4..: fold, four warps for each 64 columns (16, 12 or 8 in all); warp w reads
//              TMEM lanes 32 (w % 4) .. +31 (a row per lane), columns 64 ((w - 4) / 4) .. +63
// What bounds it: a TMEM buffer's way from the MMA's end through the fold and back to
// the even CTA takes about 1000 cycles, even with nothing folded (MMA latency, the commit's
// and the release's way across the pair): with two buffers that is more than the other
// buffer's MMA (512 cycles at BN = 256), so the length of the fold's path counts, not its
// throughput.  BN = 128 has four buffers and is bound by shared memory (48 KB written and
// read a K block, 470 cycles).  Per K block: 0.42 us at BN = 256, 0.375 at 192, 0.245 at 128.
// Measured: 2048 x 5120 x 5120 49 us (2.19 PFLOP/s; the last 256 columns in the narrow
// kernel), 5268 x 17408 x 5120 354 us (2.65 PFLOP/s; 390 us in a row of calls that meets the
// power limit), gate/up 2048 x 5120 x 2 x 17408 290 us (2.52 PFLOP/s; 310 in a row).
// Next to that way the fold's instructions count: 112 a K block and fold warp (gate/up 137),
// 32 of them the packed FMAs; a spill in the K loop costs 20 to 40%.
// Not kept: three buffers of 160 columns with 20 fold warps, halves of the tile with MMAs
// and warps of their own, two MMA issuers, a producer warp per operand (all within 5%),
// polling instead of sleeping waits (5% slower), sleeping without a look first (10%), 8 fold
// warps of 128 columns at BN = 256 (as fast for the product, 9% slower for gate/up), a fold
// loop of one or two K blocks (8 to 25%), unpacked FMAs (12%), gate/up with gate and up columns
// in different warps that exchange halves at the end (18%).  At 2.7 PFLOP/s the power limit
// is near: without any fold the same loop reaches 3.0 PFLOP/s at clocks down to 1.6 GHz.
#include "fp8a8.cuh"

#include <type_traits>

namespace qmm {
namespace {

// RAGGED: Y's row pitch is no multiple of 16 bytes.  BF16: Y is bf16, not fp32.  (One kernel with
// all four ways to store makes the fold spill.)
// EPI: y = act(y + bias) + R before the rounding (2048 x 5120 x 17408 with bias and tanh's gelu 188 us, 5268 x 17408 x
// 5120 onto an fp32 residual 405 us: the K loop as without it, and 4 to 6 us at a tile's end, when every CTA's
// fold warps stop at about the same time); RAGGED is then Y's or R's pitch no multiple of 4 elements.
template <int BN_, bool GATED_, bool BF16_ = true, bool RAGGED_ = false, bool EPI_ = false>
struct PairCfg {
    static constexpr int BN = BN_;
    static constexpr bool GATED = GATED_, RAGGED = RAGGED_, BF16 = BF16_, EPI = EPI_;
    using Params = std::conditional_t<EPI, Fp8a8EpilogueParams, Fp8a8Base>;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BN / 2 * 128, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGING = EPI ? 8192 : 4096;   // of a fold warp, for its outputs
    // 160 KB of operands (256 columns to a product: 128 KB beside the 64 KB of staging, as fast)
    static constexpr int STAGES = (!GATED && (BN == 256 || EPI) ? 131072 : 163840) / STAGE_BYTES;
    static constexpr int NBUF = BN <= 128 ? 4 : 2, BUF_COLS = 512 / NBUF;
    // Ring of scales: slots of SC_KB K blocks, which is also how many the fold loop unrolls: the
    // loop's end moves sums between registers (131 instructions a K block unrolled by four,
    // 112 by eight; 4% slower at 5268 x 17408 x 5120).  Gate/up unrolled by eight spills.
    static constexpr int SC_KB = GATED ? 4 : 8, SC_SLOTS = 16 / SC_KB;
    static constexpr int SC_PITCH = 128 + 4;                      // per K block: the rows' scales, the two blocks'
    static constexpr int SC_FLOATS = SC_SLOTS * SC_KB * SC_PITCH;
    // Fold threads: a row and CW columns, LW of them a TMEM load.  Few large loads are best
    // where the registers hold them (8 fold warps: all 64 columns at once, 37 us against 45
    // with loads of 32 at 256 x 17408 x 5120; 12 warps: 32); 16 warps need more than an even
    // share of the registers for their sums (a register split) and loads of 8 (gate/up with
    // loads of 16: 15% slower at 2048 x 5120 x 2 x 17408).
    // With the epilogue: 8 warps of 128 columns at BN = 256, which leaves registers for it (16 warps
    // spill in the K loop: 292 us in place of 188 at 2048 x 5120 x 17408 with bias and GELU).
    static constexpr bool WIDE = EPI && BN == 256;
    static constexpr int CW = WIDE ? 128 : 64, GROUPS = BN / CW, FOLD_WARPS = 4 * GROUPS, LW = WIDE ? 64 : BN == 256 ? 8 : BN == 192 ? (EPI ? 8 : 32) : 64;
    static constexpr int OUT_BYTES = GATED ? 2 * GROUPS * 128 * 4 : FOLD_WARPS * STAGING;   // row maxima, or output staging
    static constexpr bool REG_SPLIT = BN == 256;
    static constexpr int THREADS = 128 + 32 * FOLD_WARPS, REGS = 65536 / THREADS / 8 * 8, REGS_FOLD = WIDE ? 224 : 104, REGS_OTHER = WIDE ? 56 : 64;
    static_assert(!REG_SPLIT || REGS_FOLD * 32 * FOLD_WARPS + REGS_OTHER * 128 == REGS * THREADS, "register shares = launch registers");
    static constexpr int BARS = 2 * STAGES + NBUF + 2 * SC_SLOTS + 3;
    // The bias of four tiles: the scales' warps, which copy it, are at most SC_SLOTS = 2 tiles ahead of the tile
    // whose K blocks are folded, and the epilogue of the tile before that one may still be reading its own.
    static constexpr int BIAS_FLOATS = EPI ? 4 * BN : 0;
    static_assert(!EPI || SC_SLOTS <= 2, "the scales' warps are too far ahead");
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + OUT_BYTES + (SC_FLOATS + BIAS_FLOATS) * 4 + BARS * 8 + 64;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(!GATED || BN == 256, "gate/up: 128 + 128 columns");
    static_assert(NBUF <= STAGES, "a stage's MMA barrier completes again only after its accumulator was read");
};

struct PairTile {
    int m0, n0;   // first row of this CTA, first column (gated: first h column)
};

template <class C>
__device__ __forceinline__ PairTile pair_tile(const Fp8a8Base& p, int t, int crank) {
    const int mt = t % p.m_tiles, nt = t / p.m_tiles;
    PairTile r;
    r.m0 = mt * 256 + crank * 128;
    r.n0 = p.n_first + nt * (C::GATED ? 128 : C::BN);
    return r;
}

// E4M3 codes of four values scaled by gs
__device__ __forceinline__ uint32_t codes4(const GroupScale& gs, uint64_t a, uint64_t b) {
    const float2 x = unpack2(a), y = unpack2(b);
    return e4m3x4(gs(x.x), gs(x.y), gs(y.x), gs(y.y));
}

template <class C>
__global__ void __launch_bounds__(C::THREADS) __maxnreg__(C::REGS)
    fp8a8_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, typename C::Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stage = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* outs = stage + C::STAGES * C::STAGE_BYTES;         // output staging of the fold warps
    float* rowmax = reinterpret_cast<float*>(outs);              // gated: [tile parity][quarter][128]
    float* sc = reinterpret_cast<float*>(outs + C::OUT_BYTES);   // [slot][kb][128 rows, 2 weight blocks]
    uint64_t* bars = reinterpret_cast<uint64_t*>(sc + C::SC_FLOATS + C::BIAS_FLOATS);
    uint64_t* full = bars;                    // even CTA's: both CTAs' operands of a stage have landed
    uint64_t* done = full + C::STAGES;        // a stage's MMAs are complete: its operands are free, its P is in TMEM
    uint64_t* acc_empty = done + C::STAGES;   // even CTA's: both CTAs' fold warps have read the buffer
    uint64_t* sc_full = acc_empty + C::NBUF;
    uint64_t* sc_empty = sc_full + C::SC_SLOTS;
    uint64_t* drain = sc_empty + C::SC_SLOTS;
    uint64_t* rm_full = drain + 1;            // gated: every fold warp's row maxima are in shared memory
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rm_full + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    // (read through a shuffle, so that the compiler knows it and the TMEM addresses made
    // from it to be the same in the whole warp)
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&done[i], 1);
        }
        for (int i = 0; i < C::NBUF; ++i) mbar_init(&acc_empty[i], 2 * C::FOLD_WARPS);
        for (int i = 0; i < C::SC_SLOTS; ++i) {
            mbar_init(&sc_full[i], 64);
            mbar_init(&sc_empty[i], C::FOLD_WARPS);
        }
        mbar_init(drain, 1);
        mbar_init(&rm_full[0], C::FOLD_WARPS);
        mbar_init(&rm_full[1], C::FOLD_WARPS);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    wait_prerequisites();
    cluster_sync();   // the peer's barriers are initialised before any copy or commit signals them
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const int crank = __shfl_sync(0xffffffffu, (int)cluster_ctarank(), 0);
    const int cid = __shfl_sync(0xffffffffu, (int)cluster_id_x(), 0), ncl = (int)(gridDim.x >> 1);
    const int tiles = p.m_tiles * p.n_tiles, kbs = (p.K + 127) / 128;

    if (warp >= 4) {
        if constexpr (C::REG_SPLIT) setmaxnreg_inc<C::REGS_FOLD>();
        // ------------------------------------------------------------ fold
        const int q = warp & 3, cq = (warp - 4) >> 2, row = q * 32 + lane;
        const uint32_t lane_addr = tmem_base + ((uint32_t)(q * 32) << 16);
        int st = 0, slot = 0, round = 0;
        uint32_t ph = 0, sph = 0, rph = 0;
        bool ok = true;
        for (int t = cid; t < tiles && ok; t += ncl, ++round) {
            // which of the tile's two weight blocks the thread's 64 columns are in (gated: the
            // first half in one, the second in the other)
            const int blk = !C::GATED && cq * C::CW >= 128 - (pair_tile<C>(p, t, crank).n0 & 127);
            uint64_t acc[C::CW / 2];
#pragma unroll
            for (int j = 0; j < C::CW / 2; ++j) acc[j] = 0;
            for (int kb0 = 0; kb0 < kbs && ok; kb0 += C::SC_KB) {
                ok &= mbar_wait(&sc_full[slot], sph, abort_flag, p.err, DEV_TIMEOUT_CONV);
                const float* scr = sc + slot * C::SC_KB * C::SC_PITCH;
#pragma unroll
                for (int k = 0; k < C::SC_KB; ++k) {
                    if (kb0 + k >= kbs) break;
                    const float sx = scr[k * C::SC_PITCH + row];
                    const float s0 = sx * scr[k * C::SC_PITCH + 128 + blk];
                    const float s1 = C::GATED ? sx * scr[k * C::SC_PITCH + 129] : s0;
                    // (after a time-out the sums mean nothing; the loop ends with this group)
                    ok &= mbar_wait(&done[st], ph, abort_flag, p.err, DEV_TIMEOUT_ACC);
                    tc_fence_after();
                    const int buf = k & (C::NBUF - 1);
                    const uint32_t a0 = lane_addr + (uint32_t)(buf * C::BUF_COLS);
#pragma unroll
                    for (int x = 0; x < C::CW; x += C::LW) {
                        uint32_t r[C::LW];
                        tmem_ld(a0 + fold_col<C>(cq, x), r);
                        tmem_ld_wait();
                        if (x == C::CW - C::LW) {
                            // every column is in registers: the MMA may write the buffer again
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_even(&acc_empty[buf], crank);
                        }
                        const float sf = x < C::CW / 2 ? s0 : s1;
                        const uint64_t s2 = pack2(sf, sf);
#pragma unroll
                        for (int j = 0; j < C::LW / 2; ++j) {
                            acc[x / 2 + j] = fma2(pack2u(r[2 * j], r[2 * j + 1]), s2, acc[x / 2 + j]);
                        }
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
            if (!ok) break;
            int te = t;   // (the tile's place is worked out again, not kept in registers through its K blocks)
            asm volatile("" : "+r"(te));
            const PairTile ti = pair_tile<C>(p, te, crank);
            if constexpr (!C::GATED) {
                uint8_t* stg = outs + (warp - 4) * C::STAGING;
                if constexpr (C::EPI) store_epilogue<C::BF16, !C::RAGGED, C::CW, C::STAGING / 128>(p, stg, sc + C::SC_FLOATS + (round & 3) * C::BN, fold_col<C>(cq, 0), lane, (long)ti.m0 + q * 32, ti.n0 + fold_col<C>(cq, 0), acc);
                else store_columns<C::BF16, C::RAGGED, C::BN == 256 ? 4 : 8>(p, stg, lane, (long)ti.m0 + q * 32, ti.n0 + fold_col<C>(cq, 0), acc);
            } else {
                // the first half of acc: gate columns; the second half: the same columns of up
                constexpr int HP = C::CW / 4;   // pairs
                const long grow = (long)ti.m0 + row;
                float a = 0.f;
#pragma unroll
                for (int j = 0; j < HP; ++j) {
                    const float2 g = unpack2(acc[j]), u = unpack2(acc[HP + j]);
                    const float h0 = swiglu(g.x, u.x), h1 = swiglu(g.y, u.y);
                    a = max_nan_abs(a, h0, h1);
                    acc[j] = pack2(h0, h1);
                }
                const int parity = round & 1;
                float* rm = rowmax + parity * 512 + row;
                rm[cq * 128] = a;
                __syncwarp();
                if (lane == 0) mbar_arrive(&rm_full[parity]);
                if (!mbar_wait(&rm_full[parity], rph, abort_flag, p.err, DEV_TIMEOUT_ACC)) break;
                rph ^= (uint32_t)parity;
#pragma unroll
                for (int i = 0; i < C::GROUPS; ++i) a = max_nan(a, rm[i * 128]);
                const GroupScale gs = group_scale<448>(a);
                if (grow < p.M) {
                    uint4* dst = reinterpret_cast<uint4*>(p.Hq + grow * p.N + ti.n0 + cq * (C::CW / 2));
#pragma unroll
                    for (int j = 0; j < HP / 8; ++j) {
                        const uint64_t* v = acc + 8 * j;
                        dst[j] = make_uint4(codes4(gs, v[0], v[1]), codes4(gs, v[2], v[3]), codes4(gs, v[4], v[5]), codes4(gs, v[6], v[7]));
                    }
                    if (cq == 0) p.Hs[grow * (p.N / 128) + ti.n0 / 128] = gs.s;
                }
            }
        }
    } else {
        if constexpr (C::REG_SPLIT) setmaxnreg_dec<C::REGS_OTHER>();
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            // Both CTAs' copies complete on the even CTA's barrier, which expects all of
            // them; a stage is free again when its MMAs' one commit arrives in both CTAs.
            int s = 0;
            uint32_t ph = 0;
            long issued = 0;
            bool ok = true;
            for (int t = cid; t < tiles && ok; t += ncl) {
                const PairTile ti = pair_tile<C>(p, t, crank);
                // this CTA's BN/2 weight rows (gated: the even CTA gate, the odd CTA up rows)
                const int w0 = C::GATED ? ti.n0 + crank * p.N : ti.n0 + crank * (C::BN / 2);
                for (int kb = 0; kb < kbs; ++kb) {
                    const bool got = mbar_wait(&done[s], ph ^ 1u, abort_flag, p.err, DEV_TIMEOUT_TMA_EMPTY);
                    if (__any_sync(0xffffffffu, !got)) {
                        ok = false;
                        break;
                    }
                    // one copy at a time executes per thread: each copy of a stage on its own lane
                    const int l0 = (s * 2) & 31;
                    if (crank == 0 && lane == l0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE_BYTES);
                    __syncwarp();
                    uint8_t* st = stage + s * C::STAGE_BYTES;
                    if (lane == l0) tma_load_2d_pair(st, &tmX, &full[s], kb * 128, ti.m0);
                    else if (lane == l0 + 1) tma_load_2d_pair(st + C::A_BYTES, &tmW, &full[s], kb * 128, w0);
                    __syncwarp();
                    ++issued;
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // Every copy must have landed before the CTAs leave: the even CTA's barriers
            // count both CTAs' bytes.  After a time-out the odd CTA may have copies in
            // flight that the even CTA never expected: they land within microseconds.
            if (lane == 0 && crank == 0) drain_ring(full, issued, C::STAGES, p.err);
            if (!ok && crank != 0) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 5000000ull) {
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            // The whole warp runs the loop, so that descriptors and addresses are
            // warp-uniform, and one elected lane issues; from one lane's own branch each
            // MMA took about 80 cycles to issue.  One commit per K block (65 cycles to
            // issue) frees the stage and publishes the accumulator.
            if (crank == 0) {
                const uint32_t st0 = smem_u32(stage);
                int s = 0;
                uint32_t ph = 0, bph = 0;   // bph: a phase bit per buffer
                bool ok = true;
                for (int t = cid; t < tiles && ok; t += ncl) {
                    for (int kb = 0; kb < kbs; ++kb) {
                        // (every tile starts with buffer 0, so that the fold's is a constant)
                        const int buf = kb & (C::NBUF - 1);
                        const bool got = mbar_wait(&full[s], ph, abort_flag, p.err, DEV_TIMEOUT_TMA_FULL) &&
                                         mbar_wait(&acc_empty[buf], ((bph >> buf) & 1u) ^ 1u, abort_flag, p.err, DEV_TIMEOUT_ACC_EMPTY);
                        if (__any_sync(0xffffffffu, !got)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = st0 + (uint32_t)(s * C::STAGE_BYTES);
                        const uint64_t ad = smem_desc_sw128(sa), bd = smem_desc_sw128(sa + C::A_BYTES);
                        const uint32_t d = tmem_base + (uint32_t)(buf * C::BUF_COLS);
                        if (elect_one_sync()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)   // 32 codes (32 bytes) per MMA
                                tc_mma_f8_pair(d, ad + (uint64_t)(k * 2), bd + (uint64_t)(k * 2), idesc_e4m3(256, C::BN), k > 0);
                            tc_commit_pair(&done[s], 3);
                        }
                        __syncwarp();
                        bph ^= 1u << buf;
                        if (++s == C::STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
                if (elect_one_sync()) tc_commit_pair(drain, 1);
                __syncwarp();
                if (lane == 0) drain_ring(drain, 1, 1, p.err);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ scales
            // Copied 4 bytes at a time (any alignment and pitch; rows, K blocks and weight
            // blocks past the end are filled with zeros); a slot's barrier counts the
            // copies of all 64 lanes.
            const int l = threadIdx.x - 64;
            int slot = 0, round = 0;
            uint32_t sph = 0;
            bool ok = true;
            for (int t = cid; t < tiles && ok; t += ncl, ++round) {
                const PairTile ti = pair_tile<C>(p, t, crank);
                const long b0 = ti.n0 / 128, b1 = C::GATED ? (p.N + ti.n0) / 128 : b0 + 1;
                const long nblk = C::GATED ? p.N / 64 : (p.N + 127) / 128;
                for (int kb = 0; kb < kbs; kb += C::SC_KB) {
                    if (!mbar_wait(&sc_empty[slot], sph ^ 1u, abort_flag, p.err, DEV_TIMEOUT_CONV_EMPTY)) {
                        ok = false;
                        break;
                    }
                    // (the slot's barrier completes with the bias too)
                    if constexpr (C::EPI)
                        if (kb == 0) prefetch_epilogue<C::BN, 128, 64>(p, sc + C::SC_FLOATS + (round & 3) * C::BN, l, ti.m0, ti.n0);
                    float* dst = sc + slot * C::SC_KB * C::SC_PITCH;
#pragma unroll
                    for (int i = 0; i < 2 * C::SC_KB; ++i) {
                        const int k = i >> 1, r = (i & 1) * 64 + l;
                        const bool in = kb + k < kbs && ti.m0 + r < p.M;
                        cp_async4(dst + k * C::SC_PITCH + r, in ? p.Xs + ((long)ti.m0 + r) * kbs + kb + k : p.Xs, in);
                    }
                    if (l < 2 * C::SC_KB) {
                        const int k = l >> 1;
                        const long b = (l & 1) ? b1 : b0;
                        const bool in = kb + k < kbs && b < nblk;
                        cp_async4(dst + k * C::SC_PITCH + 128 + (l & 1), in ? p.S + b * kbs + kb + k : p.S, in);
                    }
                    cp_async_arrive(&sc_full[slot]);
                    if (++slot == C::SC_SLOTS) {
                        slot = 0;
                        sph ^= 1u;
                    }
                }
            }
            cp_async_wait_all();
        }
    }

    __syncthreads();
    cluster_sync();   // neither CTA leaves while the other's MMAs, copies or arrivals may reach it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

template <class C>
cudaError_t launch(const CUtensorMap& tx, const CUtensorMap& tw, const typename C::Params& p, int sms, int dev, cudaStream_t s) {
    static PerDevice most;   // pairs that fit the device at once
    cudaError_t e;
    int at_once = most.get(dev);
    if (at_once == 0) {
        e = cudaFuncSetAttribute(fp8a8_pair_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if constexpr (C::REG_SPLIT) {
            // the warpgroups' register shares add up to the launch's: launch only if the kernel
            // is allocated exactly that many (a setmaxnreg.inc past the pool waits)
            cudaFuncAttributes fa{};
            e = cudaFuncGetAttributes(&fa, fp8a8_pair_kernel<C>);
            if (e != cudaSuccess) return e;
            if (fa.numRegs != C::REGS) return cudaErrorInvalidConfiguration;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1] = overlap_attribute();
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (at_once == 0) {
        cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
        e = cudaOccupancyMaxActiveClusters(&at_once, fp8a8_pair_kernel<C>, &cfg);
        if (e != cudaSuccess) return e;
        if (at_once < 1) return cudaErrorInvalidConfiguration;
        most.set(dev, at_once);
    }
    const long tiles = (long)p.m_tiles * p.n_tiles;
    cfg.gridDim = dim3(2 * (unsigned)(tiles < at_once ? tiles : at_once), 1, 1);
    return cudaLaunchKernelEx(&cfg, fp8a8_pair_kernel<C>, tx, tw, p);
}

template <int BN>
cudaError_t launch_product(const CUtensorMap& tx, const CUtensorMap& tw, const Fp8a8Params& p, int sms, int dev, cudaStream_t s) {
    if (p.epilogue) {
        if (p.y_bf16)
            return p.vec4 ? launch<PairCfg<BN, false, true, false, true>>(tx, tw, p, sms, dev, s)
                          : launch<PairCfg<BN, false, true, true, true>>(tx, tw, p, sms, dev, s);
        return p.vec4 ? launch<PairCfg<BN, false, false, false, true>>(tx, tw, p, sms, dev, s)
                      : launch<PairCfg<BN, false, false, true, true>>(tx, tw, p, sms, dev, s);
    }
    const bool ragged = (long)p.N * (p.y_bf16 ? 2 : 4) % 16 != 0;
    if (p.y_bf16)
        return ragged ? launch<PairCfg<BN, false, true, true>>(tx, tw, p, sms, dev, s)
                      : launch<PairCfg<BN, false, true, false>>(tx, tw, p, sms, dev, s);
    return ragged ? launch<PairCfg<BN, false, false, true>>(tx, tw, p, sms, dev, s)
                  : launch<PairCfg<BN, false, false, false>>(tx, tw, p, sms, dev, s);
}

}  // namespace

cudaError_t launch_fp8a8_pair(const CUtensorMap& tx, const CUtensorMap& tw, Fp8a8Params p, bool gated, int bn, int sms,
                              int dev, cudaStream_t s) {
    p.m_tiles = (p.M + 255) / 256;
    p.n_tiles = (p.n_end - p.n_first + (gated ? 127 : bn - 1)) / (gated ? 128 : bn);
    if (gated) return launch<PairCfg<256, true>>(tx, tw, p, sms, dev, s);
    if (bn == 256) return launch_product<256>(tx, tw, p, sms, dev, s);
    if (bn == 192) return launch_product<192>(tx, tw, p, sms, dev, s);
    return launch_product<128>(tx, tw, p, sms, dev, s);
}

}  // namespace qmm
