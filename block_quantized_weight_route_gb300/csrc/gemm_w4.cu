// W4 (e2m1 codes, E4M3 per-16 scales, fp32 scale2) GEMMs: the dense prefill
// projection and the routed-MoE gate/up product with its fused SwiGLU + q8_1
// epilogue.  Kernel body: qgemm.cuh.
#include "qgemm.cuh"

namespace qmm {

#ifndef QMM_GU_TSTAGES
#define QMM_GU_TSTAGES 4
#endif
#ifndef QMM_GU_CSTAGES
#define QMM_GU_CSTAGES 3
#endif

// Dense: 256 token rows per tile (two 128-row sub-tiles share each converted
// weight tile), 4 epilogue warps.  Wide: 256 weight rows per tile, which halves
// the conversion per FLOP again; the two 128 x 256 accumulators fill TMEM, so the
// epilogue of one tile is not overlapped with the next tile's MMAs; 16 converter
// warps, two threads per weight row (28 warps under a 120 / 64 register split:
// 0.267 ms at M=2048, K=5120, N=17408 against 0.279 with 8, one thread per row).
// Narrow: 128 weight rows, 8 converter warps, double-buffered accumulators, twice
// the tiles (for problems too small to fill the SMs with wide tiles).
#ifndef QMM_W4W_CONV
#define QMM_W4W_CONV 16
#endif
using CfgW4DenseWide = GemmCfg<BMode::W4, Epi::STORE, 256, QMM_W4W_CONV, 4, 3, 2, false, 2>;
using CfgW4Dense = GemmCfg<BMode::W4, Epi::STORE, 128, 8, 4, 4, 3, false, 2>;
// Gate/up: 256 token rows x (64 gate + 64 up) weight rows per tile.
// Operands swapped: the converted 128 weight rows as the MMA's A (M = 128), the
// 256 token rows as its B (N = 256, or a short tile's live rows rounded up to 16).
#ifndef QMM_GU_SWAP
#define QMM_GU_SWAP 1
#endif
// 16 converter warps, four threads per weight row (a quarter row each; 28 warps
// under a 120 / 64 register split): 0.3486 against 0.3499 ms with 8 at T=5268.
#ifndef QMM_GU_CONV
#define QMM_GU_CONV 16
#endif
using CfgW4GateUp = GemmCfg<BMode::W4, Epi::SWIGLU_Q81, 128, QMM_GU_CONV, 4, QMM_GU_TSTAGES, QMM_GU_CSTAGES, true, 2,
                            false, QMM_GU_SWAP != 0>;
// CTA-pair forms (clusters of 2): 256 token rows x 256 weight rows per pair,
// each CTA 128 token rows and 128 weight rows (gate/up: 64 gate + 64 up).
#ifndef QMM_PAIR_TSTAGES
#define QMM_PAIR_TSTAGES 6
#endif
#ifndef QMM_PAIR_CSTAGES
#define QMM_PAIR_CSTAGES 4
#endif
using CfgW4DensePair = GemmCfg<BMode::W4, Epi::STORE, 128, 8, 4, QMM_PAIR_TSTAGES, QMM_PAIR_CSTAGES, false, 1, true>;
using CfgW4GateUpPair = GemmCfg<BMode::W4, Epi::SWIGLU_Q81, 128, 8, 4, QMM_PAIR_TSTAGES, QMM_PAIR_CSTAGES, true, 1, true>;
static_assert(CfgW4GateUp::TILE_M == CfgW4GateUpPair::TILE_M, "one routing of rows for both forms");

// Wide tiles do a tile's work in about 1.75x the time of a narrow one (measured:
// 0.305 against 0.349 ms at M=2048, K=5120, N=17408), so they win unless their
// coarser waves leave more SMs idle.
TileShape w4_dense_shape(int M, int N, int sms) {
    // CTA pairs: narrow per-CTA tiles (the pair's tile is 256 x 256)
    if (QMM_PAIR && ((N + 127) / 128) % 2 == 0) return TileShape{256, 128};
    const long wide = (long)((M + 255) / 256) * ((N + 255) / 256);
    const long narrow = (long)((M + 255) / 256) * ((N + 127) / 128);
    const long wide_waves = (wide + sms - 1) / sms, narrow_waves = (narrow + sms - 1) / sms;
    return (wide_waves * 7 < narrow_waves * 4) ? TileShape{256, 256} : TileShape{256, 128};
}
TileShape w4_gate_up_shape() { return TileShape{CfgW4GateUp::BM, CfgW4GateUp::BN}; }

int pair_ctas(int n_tiles) { return QMM_PAIR && n_tiles % 2 == 0 ? 2 : 1; }

cudaError_t launch_w4a16_dense(const CUtensorMap& tmA, const CUtensorMap& tmB, const GemmParams& p, int cn,
                               cudaStream_t s) {
    const int items = p.m_tiles * (p.n_tiles / cn);
    if (p.n_step == 256) return launch_qgemm<CfgW4DenseWide>(tmA, tmB, p, items, s);
    if (QMM_PAIR && cn == 2) return launch_qgemm<CfgW4DensePair>(tmA, tmB, p, items, s);
    return launch_qgemm<CfgW4Dense>(tmA, tmB, p, items, s);
}

cudaError_t launch_w4_gate_up_swiglu(const CUtensorMap& tmA, const CUtensorMap& tmB, const GemmParams& p, int cn,
                                     cudaStream_t s) {
    if (QMM_PAIR && cn == 2) return launch_qgemm<CfgW4GateUpPair>(tmA, tmB, p, 0, s);
    return launch_qgemm<CfgW4GateUp>(tmA, tmB, p, 0, s);
}

}  // namespace qmm
