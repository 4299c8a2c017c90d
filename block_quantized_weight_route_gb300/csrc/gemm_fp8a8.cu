// FP8 x FP8 products with block scales: which kernel takes which shape.
#include "qmm_internal.h"

namespace qmm {

// The kernel, tile and split with the least estimated time.  A launch's time is taken
// as waves x (start and end of a CTA + its K blocks x time of a K block), in
// microseconds, with the constants fitted to runs of one and of several waves at
// K = 2048 .. 17408 (the part that all kernels share, launch and memory, left out):
//   narrow kernel, 128 weight rows x tn tokens, K over cs CTAs, one CTA per SM
//   pair kernel, 256 tokens x bn columns, one pair per two SMs
// Measured at 5120 x 5120: 128 tokens narrow 128/3 10.5 us, pair 17.5; 300 tokens narrow
// 128/1 16.8, pair (192 columns) 20.9; 600 tokens 31 and 24; 1 token narrow 16/3 8.0, 16/1 13.3, 16/4 (more CTAs than
// SMs) 13.6; at 2000 x 1000, 128 tokens 32/4 6.4, 128/8 8.5.
Fp8a8Plan fp8a8_plan(int M, int K, int N, bool gated, int sms) {
    const int kbs = (K + 127) / 128;
    Fp8a8Plan best{};
    double least = 1e300;
    auto consider = [&](const Fp8a8Plan& pl, double tiles, double at_once, double ends, double kb, double per_kb) {
        const double waves = (double)(long)((tiles + at_once - 1) / at_once);
        const double t = waves * (ends + kb * per_kb);
        if (t < least) {
            least = t;
            best = pl;
        }
    };
    static const int tns[4] = {16, 32, 64, 128};
    static const double narrow_kb[2][4] = {{0.21, 0.23, 0.27, 0.30}, {0.27, 0.37, 0.50, 0.0}};
    for (int i = 0; i < (gated ? 3 : 4); ++i) {
        const double tiles = (double)((N + 127) / 128) * ((M + tns[i] - 1) / tns[i]);
        if (tiles > 8.0 * sms) continue;   // the pair kernel's
        for (int cs = 1; cs <= 8 && cs <= kbs; ++cs) {
            Fp8a8Plan pl{};
            pl.tn = tns[i];
            pl.cs = cs;
            const int at_once = fp8a8_narrow_at_once(cs);
            if (at_once < 1) continue;
            // (adding up costs a little for each CTA of a cluster)
            consider(pl, tiles, at_once, 2.2 + 0.1 * cs, (kbs + cs - 1) / cs, narrow_kb[gated][i]);
        }
    }
    static const int bns[3] = {256, 192, 128};
    static const double pair_ends[3] = {4.0, 2.9, 1.5}, pair_kb[3] = {0.43, 0.377, 0.30};
    for (int i = 0; i < (gated ? 1 : 3); ++i) {
        const double cols = gated ? 128 : bns[i];
        const double tiles = (double)((M + 255) / 256) * (double)(long)((N + cols - 1) / cols);
        Fp8a8Plan pl{};
        pl.pair = true;
        pl.bn = bns[i];
        consider(pl, tiles, sms / 2, pair_ends[i], kbs, pair_kb[i]);
    }
    return best;
}

}  // namespace qmm
