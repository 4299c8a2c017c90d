// The FP8 expert stage's products, many rows an expert: rows grouped by expert against that
// expert's weights, tile by tile of a list that the grouping wrote on the device.
//
//   y[m][n] = sum_kb Xs[m][kb] S[e][n/128][kb] P_kb[m][n],   P_kb = sum_{k in kb} Xq[m][k] W[e][n][k]
//   GATED: h = silu(y gate) * y up, rounded to E4M3 per 128 columns of a row
//   else: the rows y, as fp32 or (HALF) as fp16 with a power of two per 64 columns
//
// Persistent CTAs, each on one tile of 128 rows x 256 weight rows (GATED: 128 gate, 128 up) at a
// time: M = 128, N = 256 MMAs of one CTA.  A block's scale differs by row, so each P_kb goes from
// TMEM to fp32 sums in registers, two TMEM buffers apart from the MMA, as in the pair kernel.
//   warp 0: TMA producer   warps 1, 2: MMA issuers, one for each half of the columns
//   warp 3: the scales of several K blocks at a time, by asynchronous copies into a ring
//   warps 4..11: fold, four for each half; warp w reads TMEM lanes 32 (w % 4) .. +31 (a row per lane)
// Tiles of 128 rows rather than a CTA pair's 256, because an expert's last tile is half empty in the
// mean: 42144 rows of 128 experts fill 84% of such tiles and 64% of the pair's.
// What bounds it: shared memory.  A K block takes about 900 cycles, of which its 48 KB in and 64 KB to the MMAs (each
// issuer reads the 16 KB of rows) at 128 bytes a cycle are 896; the MMAs take 656 (82 each at N = 128) and each
// fold warp about 700 (two TMEM loads of 64 columns and their latency, 64 packed FMAs), which one issuer's 768 cycles
// of shared memory do not hide either (N = 256 MMAs, 1% slower); a tile's end takes 2300 cycles (down) to 3500 (gate/up) more,
// hidden in part because the halves of the columns drift apart.  With few rows an expert the weights' bytes bound it.
// Measured (5268 tokens, D = 2048, F = 768, 128 experts, 8 a token): gate/up 151 us (1.76 PFLOP/s, tensor pipe 48%
// active), down 95 us (1.39 PFLOP/s); 64 tokens: gate/up 65 us (6.0 TB/s), down 39 us (5.0 TB/s).
// Not kept: CTA pairs for an expert's whole 256 rows and this form for the rest (414 us for the stage in place of
// 327: the fold's two warps of a scheduler are then in step, 1040 cycles a K block); 16 fold warps
// with loads of 8 or 16 columns (4 and 3% slower); one issuer of N = 256 MMAs (1%); K blocks in a rolled loop (8%),
// by eights (1%); unpacked FMAs (8%); fold warps without a live row skipping their loads (3%).
#include "fp8a8.cuh"

namespace qmm {
namespace {

template <bool GATED_, bool HALF_ = false>
struct ExpertsCfg {
    static constexpr bool GATED = GATED_, HALF = HALF_;
    static constexpr int BN = 256, A_BYTES = 128 * 128, B_BYTES = BN * 128, STAGE_BYTES = A_BYTES + B_BYTES;
    // Fold threads: a row and 128 columns, 64 of them a TMEM load.  (16 warps of 64 columns, whose
    // registers hold loads of 8 or 16: 4 and 3% slower at 5268 tokens of 2048 columns.)
    static constexpr int CW = 128, GROUPS = BN / CW, FOLD_WARPS = 4 * GROUPS, LW = 64;
    static constexpr int STAGING = CW * 64;   // of a fold warp, for its outputs
    static constexpr int OUT_BYTES = GATED ? 2 * GROUPS * 128 * 4 : FOLD_WARPS * STAGING;   // row maxima, or output staging
    static constexpr int STAGES = GATED ? 4 : 3, NBUF = 2, BUF_COLS = 256;   // a buffer holds both halves
    // Ring of scales: slots of SC_KB K blocks, which is also how many the fold loop unrolls
    // (eight: 1% slower); a slot holds the tile's first row and its rows too.
    static constexpr int SC_KB = 4, SC_SLOTS = 16 / SC_KB, SC_PITCH = 128 + 4, SC_FLOATS = SC_SLOTS * SC_KB * SC_PITCH;
    static constexpr int THREADS = 128 + 32 * FOLD_WARPS, REGS = 65536 / THREADS / 8 * 8, REGS_FOLD = 216, REGS_OTHER = 72;
    static_assert(REGS_FOLD * 32 * FOLD_WARPS + REGS_OTHER * 128 == REGS * THREADS, "register shares = launch registers");
    static_assert(GROUPS == 2, "a fold group for each half of the columns");
    static constexpr int W_ROWS = GATED ? 64 : 128, COPIES = 1 + BN / W_ROWS;   // rows of a weight copy; copies of a stage
    static_assert(COPIES * STAGES <= 32, "a lane per copy");
    static constexpr int BARS = STAGES + 2 * (STAGES + NBUF) + 2 * SC_SLOTS + 4;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + OUT_BYTES + SC_FLOATS * 4 + BARS * 8 + 64;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(NBUF <= STAGES, "a stage's MMA barrier completes again only after its accumulator was read");
};

// Tile t of the launch: rows [m0, m0 + rows) of expert e, columns from n0.
struct ExpertTile {
    int e, m0, rows, n0;
};
template <class C>
__device__ __forceinline__ ExpertTile expert_tile(const Fp8a8Params& p, int t) {
    const int entry = t / p.n_tiles;
    const int4 v = p.tiles[entry];
    return ExpertTile{v.x, v.y, v.z, (t - entry * p.n_tiles) * (C::GATED ? 128 : C::BN)};
}

__device__ __forceinline__ uint32_t codes4(const GroupScale& gs, uint64_t a, uint64_t b) {
    const float2 x = unpack2(gs.two(a)), y = unpack2(gs.two(b));
    return e4m3x4(x.x, x.y, y.x, y.y);
}

// A lane's 64 sums as fp16 in units of a power of two, which it returns: the largest finite
// one comes to 2^14 .. 2^15, so that 11 bits are kept of all within 2^28 of it; NaN and infinities stay.
__device__ __forceinline__ float halves(const uint64_t* v, uint32_t (&h)[32]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float2 f = unpack2(v[i]);
        top = max_nan_abs(top, f.x, f.y);
    }
    if (!(top < INFINITY)) {
        top = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float2 f = unpack2(v[i]);
            const float a = fabsf(f.x), b = fabsf(f.y);
            top = fmaxf(top, fmaxf(a < INFINITY ? a : 0.0f, b < INFINITY ? b : 0.0f));
        }
    }
    // 2^(14 - e) for a top of 2^e .. 2^(e + 1), at most 2^126
    const int e = (int)(__float_as_uint(top) >> 23);   // biased
    const int up = min(127 + 14 + 127 - e, 253);
    const float f = __uint_as_float((uint32_t)up << 23);
    const uint64_t f2 = pack2(f, f);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float2 x = unpack2(mul2(v[i], f2));
        const __half2 y = __floats2half2_rn(x.x, x.y);
        h[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    return __uint_as_float((uint32_t)(254 - up) << 23);
}

// A warp's 32 rows x 128 bytes of staging to Y: eight lanes a row.
__device__ __forceinline__ void flush_rows(const Fp8a8Params& p, const uint8_t* stg, int lane, long row0, int rows, int col, int esz) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + lane / 8, c = lane % 8, n = col + c * (16 / esz);
        const uint4 d = *reinterpret_cast<const uint4*>(stg + (r * 8 + (c ^ (r & 7))) * 16);
        if (r < rows && n < p.N) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.Y) + ((row0 + r) * p.N + n) * esz) = d;
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS) __maxnreg__(C::REGS)
    fp8a8_experts_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmY, Fp8a8Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stage = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* outs = stage + C::STAGES * C::STAGE_BYTES;
    float* rowmax = reinterpret_cast<float*>(outs);              // gated: [tile parity][column group][128]
    float* sc = reinterpret_cast<float*>(outs + C::OUT_BYTES);   // [slot][kb][128 rows, 2 weight blocks]
    uint64_t* bars = reinterpret_cast<uint64_t*>(sc + C::SC_FLOATS);
    uint64_t* full = bars;
    uint64_t* done = full + C::STAGES;        // [half][stage]: the half's MMAs of a stage are complete, its P is in TMEM
    uint64_t* acc_empty = done + 2 * C::STAGES;   // [half][buffer]
    uint64_t* sc_full = acc_empty + 2 * C::NBUF;
    uint64_t* sc_empty = sc_full + C::SC_SLOTS;
    uint64_t* drain = sc_empty + C::SC_SLOTS;     // [half]
    uint64_t* rm_full = drain + 2;            // gated: every fold warp's row maxima are in shared memory
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rm_full + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&done[i], 1);
            mbar_init(&done[C::STAGES + i], 1);
        }
        for (int i = 0; i < 2 * C::NBUF; ++i) mbar_init(&acc_empty[i], C::FOLD_WARPS / 2);
        for (int i = 0; i < C::SC_SLOTS; ++i) {
            mbar_init(&sc_full[i], 32);
            mbar_init(&sc_empty[i], C::FOLD_WARPS);
        }
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        mbar_init(&rm_full[0], C::FOLD_WARPS);
        mbar_init(&rm_full[1], C::FOLD_WARPS);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_prerequisites();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const int tiles = *p.num_tiles * p.n_tiles, kbs = (p.K + 127) / 128, step = (int)gridDim.x;

    if (warp >= 4) {
        setmaxnreg_inc<C::REGS_FOLD>();
        // ------------------------------------------------------------ fold
        const int q = warp & 3, cq = (warp - 4) >> 2, row = q * 32 + lane;
        const uint32_t lane_addr = tmem_base + ((uint32_t)(q * 32) << 16);
        int st = 0, slot = 0, parity = 0;
        uint32_t ph = 0, sph = 0, rph = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += step, parity ^= 1) {
            const int blk = !C::GATED && cq * C::CW >= 128;   // which of the tile's two weight blocks
            uint64_t acc[C::CW / 2];
#pragma unroll
            for (int j = 0; j < C::CW / 2; ++j) acc[j] = 0;
            int m0 = 0, tile_rows = 0;
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
                    ok &= mbar_wait(&done[cq * C::STAGES + st], ph, abort_flag, p.err, DEV_TIMEOUT_ACC);
                    tc_fence_after();
                    // (the buffer of the tile's K block kb: every tile starts with buffer 0)
                    const int buf = k & (C::NBUF - 1);
                    const uint32_t a0 = lane_addr + (uint32_t)(buf * C::BUF_COLS);
#pragma unroll
                    for (int x = 0; x < C::CW; x += C::LW) {
                        uint32_t r[C::LW];
                        tmem_ld(a0 + cq * C::CW + x, r);
                        tmem_ld_wait();
                        if (x == C::CW - C::LW) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&acc_empty[cq * C::NBUF + buf]);
                        }
                        const float sf = x < C::CW / 2 ? s0 : s1;
                        const uint64_t s2 = pack2(sf, sf);
#pragma unroll
                        for (int j = 0; j < C::LW / 2; ++j)
                            acc[x / 2 + j] = fma2(pack2u(r[2 * j], r[2 * j + 1]), s2, acc[x / 2 + j]);
                    }
                    if (++st == C::STAGES) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (kb0 + C::SC_KB >= kbs) {
                    m0 = __float_as_int(scr[130]);
                    tile_rows = __float_as_int(scr[131]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_empty[slot]);
                if (++slot == C::SC_SLOTS) {
                    slot = 0;
                    sph ^= 1u;
                }
            }
            if (!ok) break;
            int te = t;   // (the tile's column is worked out here, not kept in a register through its K blocks)
            asm volatile("" : "+r"(te));
            const int n0 = te % p.n_tiles * (C::GATED ? 128 : C::BN);
            if constexpr (!C::GATED) {
                uint8_t* stg = outs + (warp - 4) * C::STAGING;
                const int rows = tile_rows - q * 32, col = n0 + cq * C::CW;
                const long row0 = (long)m0 + q * 32;
                if constexpr (C::HALF) {
                    if (col + C::CW > p.N) {   // (the columns past the end, another expert's, have no say in the unit)
#pragma unroll
                        for (int j = 0; j < C::CW / 2; ++j)
                            if (col + 2 * j >= p.N) acc[j] = 0;
                    }
                    tma_store_wait_read();   // (the tile before)
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < C::CW; x += 64) {
                        uint32_t h[32];
                        const float unit = halves(acc + x / 2, h);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<uint4*>(stg + x * 64 + (lane * 8 + (c ^ (lane & 7))) * 16) =
                                make_uint4(h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]);
                        if (lane < rows && col + x < p.N) p.y_unit[(row0 + lane) * ((p.N + 63) / 64) + (col + x) / 64] = unit;
                    }
                    if (rows >= 32) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane < C::CW / 64 && col + lane * 64 < p.N) tma_store_2d(&tmY, stg + lane * 4096, col + lane * 64, (int)row0);
                    } else {   // (the rows behind the last one are another expert's)
                        __syncwarp();
#pragma unroll
                        for (int x = 0; x < C::CW; x += 64) flush_rows(p, stg + x * 64, lane, row0, rows, col + x, 2);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < C::CW; c += 32) {
                        __syncwarp();
                        stage16<false>(stg, lane, 0, acc + c / 2);
                        stage16<false>(stg, lane, 4, acc + c / 2 + 8);
                        __syncwarp();
                        flush_rows(p, stg, lane, row0, rows, col + c, 4);
                    }
                }
            } else {
                // the first half of acc: gate columns; the second half: the same columns of up
                constexpr int HP = C::CW / 4;   // pairs
                float a = 0.f;
#pragma unroll
                for (int j = 0; j < HP; ++j) {
                    acc[j] = swiglu2(acc[j], acc[HP + j]);
                    const float2 h = unpack2(acc[j]);
                    a = max_nan_abs(a, h.x, h.y);
                }
                float* rm = rowmax + parity * (C::GROUPS * 128) + row;
                rm[cq * 128] = a;
                __syncwarp();
                if (lane == 0) mbar_arrive(&rm_full[parity]);
                if (!mbar_wait(&rm_full[parity], rph, abort_flag, p.err, DEV_TIMEOUT_ACC)) break;
                rph ^= (uint32_t)parity;
#pragma unroll
                for (int i = 0; i < C::GROUPS; ++i) a = max_nan(a, rm[i * 128]);
                const GroupScale gs = group_scale<448>(a);
                if (row < tile_rows) {
                    const long grow = (long)m0 + row;
                    uint4* dst = reinterpret_cast<uint4*>(p.Hq + grow * p.N + n0 + cq * (C::CW / 2));
#pragma unroll
                    for (int j = 0; j < HP / 8; ++j) {
                        const uint64_t* v = acc + 8 * j;
                        dst[j] = make_uint4(codes4(gs, v[0], v[1]), codes4(gs, v[2], v[3]), codes4(gs, v[4], v[5]), codes4(gs, v[6], v[7]));
                    }
                    if (cq == 0) p.Hs[grow * (p.N / 128) + n0 / 128] = gs.s;
                }
            }
        }
        if (C::HALF) tma_store_wait();
    } else {
        setmaxnreg_dec<C::REGS_OTHER>();
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            int s = 0;
            uint32_t ph = 0;
            long issued = 0;
            bool ok = true;
            ExpertTile ti{};
            if ((int)blockIdx.x < tiles) ti = expert_tile<C>(p, blockIdx.x);
            for (int t = blockIdx.x; t < tiles && ok; t += step) {
                // this lane's copy: rows of X, or of the weights (gated: 64 gate and 64 up rows of each half)
                const int c = lane % C::COPIES, w = c - 1;
                const int y = c == 0 ? ti.m0
                                     : ti.e * p.N * (C::GATED ? 2 : 1) + ti.n0 + (C::GATED ? (w & 1) * p.N + (w >> 1) * 64 : w * 128);
                if (t + step < tiles) ti = expert_tile<C>(p, t + step);   // (read a tile ahead)
                for (int kb = 0; kb < kbs; ++kb) {
                    const bool got = mbar_wait(&done[s], ph ^ 1u, abort_flag, p.err, DEV_TIMEOUT_TMA_EMPTY) &&
                                     mbar_wait(&done[C::STAGES + s], ph ^ 1u, abort_flag, p.err, DEV_TIMEOUT_TMA_EMPTY);
                    if (__any_sync(0xffffffffu, !got)) {
                        ok = false;
                        break;
                    }
                    // one copy at a time executes per thread: each copy of a stage on its own lane
                    const bool mine = lane / C::COPIES == s;
                    if (mine && c == 0) mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
                    __syncwarp();
                    if (mine) tma_load_2d(stage + s * C::STAGE_BYTES + (c == 0 ? 0 : C::A_BYTES + w * C::W_ROWS * 128), c == 0 ? &tmX : &tmW, &full[s], kb * 128, y);
                    __syncwarp();
                    ++issued;
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (lane == 0) drain_ring(full, issued, C::STAGES, p.err);
        } else if (warp <= 2) {
            // ------------------------------------------------------------ MMA issuers, one for each half
            const int half = warp - 1;
            const uint32_t st0 = smem_u32(stage);
            int s = 0;
            uint32_t ph = 0, bph = 0;   // bph: a phase bit per buffer
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += step) {
                for (int kb = 0; kb < kbs; ++kb) {
                    const int buf = kb & (C::NBUF - 1);
                    const bool got = mbar_wait(&full[s], ph, abort_flag, p.err, DEV_TIMEOUT_TMA_FULL) &&
                                     mbar_wait(&acc_empty[half * C::NBUF + buf], ((bph >> buf) & 1u) ^ 1u, abort_flag, p.err, DEV_TIMEOUT_ACC_EMPTY);
                    if (__any_sync(0xffffffffu, !got)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = st0 + (uint32_t)(s * C::STAGE_BYTES);
                    const uint64_t ad = smem_desc_sw128(sa), bd = smem_desc_sw128(sa + C::A_BYTES + half * (C::B_BYTES / 2));
                    const uint32_t d = tmem_base + (uint32_t)(buf * C::BUF_COLS + half * 128);
                    if (elect_one_sync()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 codes (32 bytes) per MMA
                            tc_mma_f8(d, ad + (uint64_t)(k * 2), bd + (uint64_t)(k * 2), idesc_e4m3(128, 128), k > 0);
                        tc_commit(&done[half * C::STAGES + s]);
                    }
                    __syncwarp();
                    bph ^= 1u << buf;
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (elect_one_sync()) tc_commit(&drain[half]);
            __syncwarp();
            if (lane == 0) drain_ring(&drain[half], 1, 1, p.err);
            __syncwarp();
        } else {
            // ------------------------------------------------------------ scales
            int slot = 0;
            uint32_t sph = 0;
            bool ok = true;
            const int nblk = (p.N + 127) / 128;   // weight blocks of an expert (gated: of each half)
            ExpertTile ti{};
            if ((int)blockIdx.x < tiles) ti = expert_tile<C>(p, blockIdx.x);
            for (int t = blockIdx.x; t < tiles && ok; t += step) {
                const ExpertTile now = ti;
                if (t + step < tiles) ti = expert_tile<C>(p, t + step);
                // (a second block past the expert's last is not used: its columns are past N)
                const int c0 = now.n0 / 128, c1 = C::GATED ? nblk + c0 : min(c0 + 1, nblk - 1);
                const long b0 = (long)now.e * nblk * (C::GATED ? 2 : 1);
                for (int kb = 0; kb < kbs; kb += C::SC_KB) {
                    if (!mbar_wait(&sc_empty[slot], sph ^ 1u, abort_flag, p.err, DEV_TIMEOUT_CONV_EMPTY)) {
                        ok = false;
                        break;
                    }
                    float* dst = sc + slot * C::SC_KB * C::SC_PITCH;
#pragma unroll
                    for (int i = 0; i < 4 * C::SC_KB; ++i) {
                        const int k = i >> 2, r = (i & 3) * 32 + lane;
                        const bool in = kb + k < kbs && r < now.rows;
                        cp_async4(dst + k * C::SC_PITCH + r, in ? p.Xs + ((long)now.m0 + r) * kbs + kb + k : p.Xs, in);
                    }
                    if (lane < 2 * C::SC_KB) {
                        const int k = lane >> 1;
                        const bool in = kb + k < kbs;
                        cp_async4(dst + k * C::SC_PITCH + 128 + (lane & 1), in ? p.S + (b0 + ((lane & 1) ? c1 : c0)) * kbs + kb + k : p.S, in);
                    }
                    if (lane >= 30) {   // the tile's first row and its rows
                        const int entry = t / p.n_tiles;
                        cp_async4(dst + 130 + (lane & 1), reinterpret_cast<const int*>(p.tiles + entry) + 1 + (lane & 1), true);
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

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

template <class C>
cudaError_t launch(const CUtensorMap& tx, const CUtensorMap& tw, const CUtensorMap& ty, const Fp8a8Params& p, int sms, int dev,
                   cudaStream_t s) {
    static PerDevice ready;
    if (!ready.get(dev)) {
        cudaError_t e = cudaFuncSetAttribute(fp8a8_experts_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        // the warpgroups' register shares add up to the launch's: launch only if the kernel
        // is allocated exactly that many (a setmaxnreg.inc past the pool waits)
        cudaFuncAttributes fa{};
        e = cudaFuncGetAttributes(&fa, fp8a8_experts_kernel<C>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != C::REGS) return cudaErrorInvalidConfiguration;
        ready.set(dev, 1);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {overlap_attribute()};
    const long tiles = (long)p.max_tiles * p.n_tiles;
    cfg.gridDim = dim3((unsigned)(tiles < sms ? tiles : sms), 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp8a8_experts_kernel<C>, tx, tw, ty, p);
}

}  // namespace

cudaError_t launch_fp8a8_experts(const CUtensorMap& tx, const CUtensorMap& tw, const CUtensorMap& ty, Fp8a8Params p, bool gated, int sms,
                                 int dev, cudaStream_t s) {
    p.n_tiles = gated ? p.N / 128 : (p.N + 255) / 256;
    if (gated) return launch<ExpertsCfg<true>>(tx, tw, ty, p, sms, dev, s);
    if (p.y_unit) return launch<ExpertsCfg<false, true>>(tx, tw, ty, p, sms, dev, s);
    return launch<ExpertsCfg<false, false>>(tx, tw, ty, p, sms, dev, s);
}

}  // namespace qmm
