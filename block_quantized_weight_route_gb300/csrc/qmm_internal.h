// Internal declarations shared by the library's translation units (not installed).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device_cache.h"

namespace qmm {

// Parameters of one launch of the block-quantised GEMM kernel family.
struct GemmParams {
    int M, N, K;            // dense: output rows, columns; all: reduction length
    int F;                  // gate/up: rows of each half (gate, up) per expert
    int m_tiles, n_tiles;   // dense: tile grid; grouped: n_tiles per row-tile entry
    int n_step;             // output columns advanced per column tile
    const int4* tiles;      // grouped: {expert, first row, rows, 0} per 128-row entry
    const int* num_entries; // grouped: device count of valid entries
    int max_entries;        // grouped: capacity of `tiles`
    const uint8_t* w_scale; // W4: E4M3 scale bytes, one per 16 K per weight row
    const float* scale2;    // gate/up: fp32 scale2 per expert
    float scale2_dense;     // dense W4: fp32 scale2
    const float* blk_scale; // FP8: [N/128][K/128] block scales
    const float* dH32;      // down: fp32 d of H per 128-row tile entry, [entry][K/32][128]
    const __half* dW;       // down: IQ4_NL block scales, [E][N][K/32]
    // per-expert weights (pointer-table form of the expert stage; null: the
    // contiguous [E][...] arrays through tmB / tmA, w_scale and dW above)
    const CUtensorMap* wmaps;          // [E] tensor maps of each expert's weight codes
    const uint8_t* const* wscale_tab;  // gate/up: [E] E4M3 scale matrices [2F][D/16]
    const __half* const* dW_tab;       // down: [E] IQ4_NL scale matrices [D][F/32]
    const int32_t* src;     // down with the combine fused: token of each routed row [P]
    const float* wrow;      // down with the combine fused: routing weight of each routed row [P]
    void* Y;                // output (fp32 or bf16)
    int ydt;                // 0: fp32, 1: bf16
    long ldy;               // output row pitch in elements
    __half* Hq;             // gate/up: q8_1 codes of H [rows][F], exact f16 integers
    __half* Hd;             // gate/up: q8_1 d per 32-block [rows][F/32]
    __half* Hs;             // gate/up: q8_1 s per 32-block [rows][F/32]
    float* Hd32;            // gate/up: fp32 value of the fp16 d, [entry][F/32][128 rows]
    uint32_t* err;          // device error word
    // dense only: K splits of the last, partly filled wave of tiles.  Work items
    // [split_from, ...) are split_S consecutive K ranges of the tiles (items)
    // split_from, split_from + 1, ...; each split writes its fp32 partial tile
    // to split_part, and a reduction kernel launched after the GEMM adds them in
    // split order and writes the output.  split_S == 1: no splits.
    int split_from;
    int split_S;
    float* split_part;      // [split tile][cluster rank][split][BM][BN] fp32 (null: never split)
    long split_part_cap;    // floats available at split_part
};

// Launchers (return a cudaError_t from the launch).  Each takes two encoded
// tensor maps: tmA for the activation operand (box rows: the tile's / cn), tmB for
// the raw weight codes; cn, the CTAs that compute a tile (pair_ctas), must divide
// p.n_tiles.
int pair_ctas(int n_tiles);   // 2 in the CTA-pair build where the column tiles pair up, else 1
cudaError_t launch_w4a16_dense(const CUtensorMap& tmA, const CUtensorMap& tmB, const GemmParams& p, int cn,
                               cudaStream_t s);
cudaError_t launch_w4_gate_up_swiglu(const CUtensorMap& tmA, const CUtensorMap& tmB, const GemmParams& p, int cn,
                                     cudaStream_t s);
// token rows and weight rows (gate + up for the gate/up product) of one W4 tile
struct TileShape {
    int rows, bn;
};
TileShape w4_dense_shape(int M, int N, int sms);   // the launch picks the kernel by n_step (128 or 256)
TileShape w4_gate_up_shape();
// token rows of one FP8 tile (the activation box height before a pair's split)
int fp8_tile_rows();
cudaError_t launch_fp8_blk128(const CUtensorMap& tmA, const CUtensorMap& tmB, const GemmParams& p, int cn,
                              cudaStream_t s);
// combine = false: per-slot rows p.Y [P][N] fp32; true: Y[src[r]] += wrow[r] * y_r
// accumulated into p.Y [T][N] fp32 (which must start at zero).
cudaError_t launch_iq4_down(const CUtensorMap& tmA, const CUtensorMap& tmB, const GemmParams& p, int grid, bool combine,
                            cudaStream_t s);

int smem_iq4_down();

// Dense Q8_0 x q8_1 projection re-quantised to q8_1 (gemm_q8.cu): tmA Q8_0 codes
// [N][K] int8 (or, when q8_weights_f16(), the same codes as f16, 128-byte swizzle),
// tmB activation codes [M][K] f16, tmW weight scales [N][K/32] fp16;
// p.tiles / num_entries: 128-row tiles of M (launch_dense_tiles), p.dH32: the
// activations' d per tile [entry][K/32][128] fp32.
bool q8_weights_f16();
cudaError_t launch_dense_tiles(int M, int4* tiles, int32_t* num_entries, cudaStream_t s);
cudaError_t launch_q8_dense(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmW, const GemmParams& p,
                            int8_t* Yq, __half* Yd, __half* Ys, float* Y, int M, int grid, cudaStream_t s);

// Routing and data-movement kernels (route.cu).
struct RouteBufs {
    int32_t* ids;         // [T][k]
    float* w;             // [T][k]
    int32_t* counts;      // [E]
    int32_t* offsets;     // [E+1]
    int32_t* src;         // [T*k]
    int32_t* row;         // [T][k]
    int32_t* chunk_hist;  // [chunks][E]  (scratch)
    int4* tiles;          // [max_entries] 128-row entries (optional)
    int32_t* num_entries; // [1]            (optional)
    int max_entries;
    int4* tiles2;         // [max_entries2] 256-row entries (optional, needs tiles)
    int32_t* num_entries2;
    int max_entries2;
    float* wrow = nullptr;    // [T*k] weight of the pair at each routed row (optional)
    float* yzero = nullptr;   // [T][yzero_D] fp32 rows set to zero by the top-k kernel (optional)
    int yzero_D = 0;
};
constexpr int kRouteChunk = 256;   // tokens per grouping chunk
cudaError_t launch_route(const float* logits, int T, int E, int k, const RouteBufs& b, cudaStream_t s);
cudaError_t launch_gather_rows(const uint16_t* X, const int32_t* src, int rows, int D, uint16_t* Xp, cudaStream_t s);
cudaError_t launch_tiles_from_offsets(const int32_t* offsets, int E, int P, uint32_t* err, const RouteBufs& b,
                                      cudaStream_t s);
cudaError_t launch_codes_f16_to_i8(const __half* src, int8_t* dst, long n, cudaStream_t s);
cudaError_t launch_codes_i8_to_f16(const int8_t* src, __half* dst, long n, cudaStream_t s);
cudaError_t launch_hd_to_entries(const __half* Hd, const int4* tiles, const int32_t* num_entries, int max_entries,
                                 int groups, float* Hd32, cudaStream_t s);
cudaError_t launch_wait_timeout_probe(uint32_t* err, uint64_t limit_ns, cudaStream_t s);
cudaError_t launch_combine(const float* Yslot, int P, const int32_t* row, const float* w, int T, int k, int D,
                           float* Y, uint32_t* err, cudaStream_t s);

// Residual addition + RMS norm + 8-bit output (rmsnorm8.cu).
struct NormParams {
    const void* X;       // [T][ldx] f32 or bf16
    const void* R;       // [T][ldr] residual, or null
    void* Rout;          // [T][ldro] the sum in the residual's type
    const void* G;       // [D]
    long ldx, ldr, ldro; // row pitches in elements
    int x_bf16, r_bf16, g_bf16;
    float eps;
    int T, D;
    uint8_t* Q;          // [T][D] codes: E4M3, or q8_1's int8
    float* S;            // [T][ceil(D/128)] E4M3 scales
    __half *Yd, *Ys;     // [T][D/32] q8_1's d and d * sum
    uint16_t* Y;         // [T][D] bf16 rows, or null
};
int rmsnorm8_max_width();
cudaError_t launch_rmsnorm8(const NormParams& p, bool q81, cudaStream_t s);

// Grouping of the FP8 expert stage (moe_fp8.cu).
constexpr int kMoeChunk = 2048, kMoeMaxExperts = 512;   // pairs of a grouping chunk
constexpr int kMoeSmall = 32;                           // pairs that one warp groups
struct MoeGroups {
    int32_t* counts;        // [E]
    int32_t* offsets;       // [E + 1]
    int32_t* src;           // [P] token of each row
    int32_t* row;           // [P] row of each pair, -1 for one without an expert
    int32_t* chunk_counts;  // [chunks][E] (scratch)
    int4* tiles;            // {expert, first row, rows, 0}
    int* num_tiles;
    int tile_rows, max_tiles;
};

// FP8 x FP8 products with block scales (gemm_fp8a8.cu).  A kernel takes the fields that its form has and no more:
// with those of the other forms beside them, which none of its code reads, two of the plain products' 256-column pair
// kernels spill in their K loops (44 and 96 bytes stored; 5268 x 17408 x 5120 with fp32 output 487 us in place of
// 355, 2048 x 5120 x 17407 285 in place of 165), and the others are 5% slower (364 us in place of 348 with bf16 output).
struct Fp8a8Base {
    const uint8_t* Xq;   // [M][K] E4M3
    const float* Xs;     // [M][ceil(K/128)]
    const uint8_t* W;    // [N][K] E4M3; gated: [2N][K], gate rows first
    const float* S;      // [ceil(rows/128)][ceil(K/128)]
    int M, K, N;         // gated: N = F
    void* Y;             // [M][N]
    int y_bf16;
    uint8_t* Hq;         // gated: [M][F] E4M3
    float* Hs;           // gated: [M][F/128]
    uint32_t* err;       // device error word
    int n_first, n_end;  // the launch's columns (n_first a multiple of 128)
    int m_tiles, n_tiles;
};
// y = act(y + bias[n]) + R[m][n]
struct Fp8a8EpilogueParams : Fp8a8Base {
    bool epilogue;
    int act;             // a qmm_act
    const void* bias;    // [N], or null
    const void* R;       // [M][ldr], or null; may be Y
    long ldr;
    int bias_bf16, r_bf16;
    bool vec4;           // N and ldr are multiples of 4
};
// rows grouped by expert: W [E][N or 2N][K], S alike, M all rows
struct Fp8a8Params : Fp8a8EpilogueParams {
    const int4* tiles;   // {expert, first row, rows, 0}; null: not grouped
    const int* num_tiles;   // on the device
    int max_tiles;       // room in `tiles`
    const int32_t* src;  // narrow kernel, gated: a row's token (Xq and Xs are the tokens', gathered by the kernel)
    const int32_t* ids;  // narrow kernel, gated: not null: it groups the pairs by itself (M <= kMoeSmall of them) and
    int E, k;            // writes the grouping that the tiles come from
    MoeGroups groups;
    float* y_unit;       // [M][ceil(N/64)]: Y is fp16 in these units (null: fp32)
};
// Which kernel takes a product: the pair kernel (many tokens) with its tile's columns,
// or the narrow kernel (few) with its tile's tokens and the CTAs that share its K blocks.
struct Fp8a8Plan {
    bool pair;
    int bn;      // pair: columns of a tile
    int tn, cs;  // narrow
};
// The columns [0, split) go to one launch, [split, N) to a second one (none if split = N).
struct Fp8a8Plans {
    Fp8a8Plan first, second;
    int split;
};
cudaError_t fp8a8_plan(int M, int K, int N, bool gated, int sms, int dev, Fp8a8Plans* plans);
// The expert stage's tiles: tokens of a tile, and the CTAs that share the K blocks of one in
// the gate/up and in the down product.
struct MoePlan {
    bool many;           // the kernel for many rows an expert (tiles of 128), else the narrow one
    int tn, cs_gate_up, cs_down;
};
bool moe_plan_fits(const MoePlan& pl, int T, int D, int F, int E, int k);   // whether the kernels can run a given tiling
cudaError_t moe_plan(int T, int D, int F, int E, int k, int sms, int dev, MoePlan* plan);
bool fp8a8_plans_fit(const Fp8a8Plans& r, int M, int K, int N, bool gated);   // whether the kernels can run a given tiling
// clusters of cs CTAs that the device holds at once (0: none)
cudaError_t fp8a8_narrow_at_once(bool gated, int tn, int cs, int dev, int* clusters);
cudaError_t launch_fp8a8_narrow(const CUtensorMap& tx, const CUtensorMap& tw, const Fp8a8Params& p, bool gated, int tn,
                                int cs, int dev, cudaStream_t s);
// (ty: the fp16 rows, boxes of 32 rows x 64 columns; not read where they are fp32)
cudaError_t launch_fp8a8_experts(const CUtensorMap& tx, const CUtensorMap& tw, const CUtensorMap& ty, Fp8a8Params p, bool gated, int sms,
                                 int dev, cudaStream_t s);
cudaError_t launch_fp8a8_pair(const CUtensorMap& tx, const CUtensorMap& tw, Fp8a8Params p, bool gated, int bn, int sms,
                              int dev, cudaStream_t s);

cudaError_t launch_moe_group(const int32_t* ids, int P, int E, int k, const MoeGroups& g, int dev, cudaStream_t s);
cudaError_t launch_moe_gather(const uint8_t* Xq, const float* Xs, int P, int D, const MoeGroups& g, int E, uint8_t* Xp, float* Xps,
                              int sms, cudaStream_t s);
// Whether the combine's tokens are too few to fill the device with a block each (eight to an SM).
inline bool moe_combine_splits(int T, int sms) { return T <= 8 * sms; }
// (y_unit: y is fp16 in units of it, as launch_fp8a8_experts writes it; else fp32)
cudaError_t launch_moe_combine(const void* y, const float* y_unit, const int32_t* row, const float* w, int T, int k, int D, const void* R, int r_bf16,
                               long ldr, void* Y, int y_bf16, int sms, cudaStream_t s);

// Routing by scores (route_scored.cu).
struct ScoredParams {
    const void* logits;  // [T][ldl] fp32 or bf16
    const float* bias;   // [E], or null
    const int32_t* live; // tokens from *live on have no experts (null: all T are live)
    long ldl;
    int l_bf16, T, E, k;
    int sigmoid;         // else softmax
    int groups, groups_kept, group_top;
    int group_size;      // E / groups, and 2^20 / group_size rounded up (set by the launcher)
    unsigned group_inv;
    int per_shift;       // lanes that share a group, as a power of two (set by the launcher)
    int renorm;
    float scale;
    int32_t* ids;        // [T][k]
    float* w;            // [T][k]
};
cudaError_t launch_route_scored(ScoredParams p, int sms, cudaStream_t s);

// Set the calling thread's message returned by qmm_last_error().
void set_last_error(const char* msg);
}  // namespace qmm
