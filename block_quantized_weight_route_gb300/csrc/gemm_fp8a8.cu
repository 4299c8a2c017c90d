// FP8 x FP8 products with block scales: which kernel takes which shape.
#include <algorithm>
#include <cmath>

#include "qmm_internal.h"

namespace qmm {

namespace {

constexpr int kBn[3] = {256, 192, 128};
constexpr double kPairEnds[3] = {4.0, 2.9, 1.5}, kPairKb[3] = {0.42, 0.375, 0.245};
constexpr int kTn[4] = {16, 32, 64, 128};
constexpr double kNarrowKb[2][4] = {{0.21, 0.23, 0.27, 0.30}, {0.27, 0.37, 0.50, 0.65}};

constexpr double kSecondLaunch = 1.5;

// microseconds for what the tiles read through L2: `rows` operand rows of 128 bytes a K block
double traffic_time(long tiles, int kbs, int rows) { return (double)tiles * kbs * rows * 128 / 30e6; }

double pair_time(long tiles, long pairs, int i, int kbs) {
    return (double)((tiles + pairs - 1) / pairs) * (kPairEnds[i] + kbs * kPairKb[i]) + traffic_time(tiles, kbs, 256 + kBn[i]);
}

// The kernel, tile and split of K with the least estimated time for one launch over
// `cols` columns.  A launch's time is taken as waves x (start and end of a CTA + its K
// blocks x time of a K block), in microseconds, with the constants fitted to runs of one and of
// several waves at K = 2048 .. 17408 (the launch, which all share, left out), plus a charge
// for the operands' way through L2, which tells tilings of equal waves apart:
//   narrow kernel, 128 weight rows x tn tokens, K over cs CTAs
//   pair kernel, 256 tokens x bn columns, one pair per two SMs
// Measured at 5120 x 5120: 128 tokens narrow 128/3 11.1 us, pair (128 columns) 13.4; 300 tokens
// narrow 128/1 16.7, pair (192) 18.6; 600 tokens 32.4 and (256) 21.4; 1 token narrow 16/6 7.2,
// 16/3 8.0, 16/7 (more CTAs than fit at once) 12.9; at K = 2000, N = 1000, 128 tokens 32/4 6.2,
// 128/8 7.1, pair (128) 7.9; gate/up at 5120 x 17408, 100 tokens narrow 128/1 34.4, 64/1 61, pair 42;
// 300 tokens 94, 147 and 80.
// (A tiling that cannot be asked about is an error, not one tiling less.)
cudaError_t one_launch(int M, int kbs, int cols, bool gated, int sms, int dev, Fp8a8Plan* best, double* time) {
    *best = Fp8a8Plan{};
    *time = 1e300;
    auto consider = [&](const Fp8a8Plan& pl, double t) {
        if (t < *time) {
            *time = t;
            *best = pl;
        }
    };
    for (int i = 0; i < 4; ++i) {
        const long tiles = (long)((cols + 127) / 128) * ((M + kTn[i] - 1) / kTn[i]);
        if (tiles > 8L * sms) continue;   // the pair kernel's
        for (int cs = 1; cs <= 8 && cs <= kbs; ++cs) {
            int at_once = 0;
            const cudaError_t e = fp8a8_narrow_at_once(gated, kTn[i], cs, dev, &at_once);
            if (e != cudaSuccess) return e;
            if (at_once < 1) continue;   // clusters of cs do not fit this device
            Fp8a8Plan pl{};
            pl.tn = kTn[i];
            pl.cs = cs;
            // (adding up costs a little for each CTA of a cluster and for each token)
            consider(pl, (double)((tiles + at_once - 1) / at_once) *
                                 (2.0 + 0.1 * cs + 0.011 * kTn[i] * (gated ? 2 : 1) +
                                  (kbs + cs - 1) / cs * kNarrowKb[gated][i]) +
                             traffic_time(tiles, kbs, kTn[i] + (gated ? 256 : 128)));
        }
    }
    // Up to 16 tokens (the narrowest tile) the pair kernel takes only what the narrow one
    // cannot.  Its constants were fitted to waves of full tiles and leave out its start, so
    // that with K <= 640 the estimate favours it where it takes 3.1 us for 2.5 (1 x 16 x 128)
    // to 5.3 for 3.7 (1 x 400 x 5120); of 496 such shapes the narrow kernel was faster in 495, by
    // 14% in the mean.  With several hundred tokens the estimate is right (600 x 16 x 256:
    // 16-token tiles 34% slower).
    if (M <= kTn[0] && *time < 1e300) return cudaSuccess;
    for (int i = 0; i < (gated ? 1 : 3); ++i) {
        const int width = gated ? 128 : kBn[i];
        Fp8a8Plan pl{};
        pl.pair = true;
        pl.bn = kBn[i];
        consider(pl, pair_time((long)((M + 255) / 256) * ((cols + width - 1) / width), sms / 2, i, kbs));
    }
    return cudaSuccess;
}

}  // namespace

// One launch, or the columns of the whole waves of widest pair tiles in one and the rest
// in a second with a plan of its own, where that takes less by more than the second
// launch costs (2048 x 5120 x 5120: 152 tiles in two waves and 256 columns left).
cudaError_t fp8a8_plan(int M, int K, int N, bool gated, int sms, int dev, Fp8a8Plans* plans) {
    // (a model's calls come in the same few shapes: the last ones' plans are kept)
    struct Known {
        int M, K, N, gated, dev;
        Fp8a8Plans plans;
    };
    static thread_local Known known[16] = {};
    Known& slot = known[((unsigned)M * 2654435761u ^ (unsigned)K * 40503u ^ (unsigned)N * 9973u ^ (unsigned)gated) >> 7 & 15u];
    if (slot.M == M && slot.K == K && slot.N == N && slot.gated == gated && slot.dev == dev) {
        *plans = slot.plans;
        return cudaSuccess;
    }
    const int kbs = (K + 127) / 128;
    Fp8a8Plans r{};
    double least;
    cudaError_t e = one_launch(M, kbs, N, gated, sms, dev, &r.first, &least);
    if (e != cudaSuccess) return e;
    r.split = N;
    const long mt = (M + 255) / 256, pairs = sms / 2;
    const int width = gated ? 128 : kBn[0];
    const long waves = mt * ((N + width - 1) / width) / pairs;
    const long whole = waves * pairs / mt * width;
    if (M > kTn[0] && waves >= 1 && whole > 0 && whole < N) {
        double rest;
        Fp8a8Plan second;
        e = one_launch(M, kbs, N - (int)whole, gated, sms, dev, &second, &rest);
        if (e != cudaSuccess) return e;
        const double t = pair_time(mt * (whole / width), pairs, 0, kbs) + rest + kSecondLaunch;
        if (t < 0.97 * least) {
            r.first = Fp8a8Plan{};
            r.first.pair = true;
            r.first.bn = kBn[0];
            r.second = second;
            r.split = (int)whole;
        }
    }
    slot = Known{M, K, N, gated, dev, r};
    *plans = r;
    return cudaSuccess;
}

// The expert stage: the tile's tokens with the least estimated time of both products (the narrow
// kernel's constants above), for tokens that choose their experts evenly: the host does not
// know the rows of an expert.
cudaError_t moe_plan(int T, int D, int F, int E, int k, int sms, int dev, MoePlan* plan) {
    struct Known {
        int T, D, F, E, k, dev;
        MoePlan plan;
    };
    static thread_local Known known[8] = {};
    Known& slot = known[((unsigned)T * 2654435761u ^ (unsigned)D * 40503u ^ (unsigned)F * 9973u ^ (unsigned)(E * 31 + k)) >> 7 & 7u];
    if (slot.T == T && slot.D == D && slot.F == F && slot.E == E && slot.k == k && slot.dev == dev) {
        *plan = slot.plan;
        return cudaSuccess;
    }
    const double experts = E * (1.0 - std::pow(1.0 - (k < E ? (double)k / E : 1.0), T)), rows = (double)T * k / experts;
    // Many rows an expert: tiles of 128 x 256 (of H: 128) on persistent CTAs, a gather before them.  Few: the narrow
    // kernel; where its CTAs come in more than one wave each pays its start anew.  Neither is faster than the
    // weights' bytes come.  Measured with D = 2048, F = 768, k = 8, narrow / many, us: 128 experts, 32 tokens 110 / 110,
    // 301 167 / 135, 512 213 / 138; 64 experts, 64 tokens 74 / 77; 16 experts, 64 tokens 34 / 40; 8 experts, F = 2048, 200 tokens 84 / 51.
    const double weights_us = experts * D * (double)F / 5.9e6;   // of the down product; gate/up: twice
    auto many_time = [&](int kbs, int columns, double bytes_us) {
        const double tiles = experts * (rows / 128.0 < 0.5 ? 1.0 : rows / 128.0 + 0.5) * columns;
        return std::max(std::ceil(tiles / sms) * (2.5 + 0.42 * kbs), bytes_us);
    };
    double least = 6.0 + many_time((D + 127) / 128, F / 128, 2 * weights_us) + many_time(F / 128, (D + 255) / 256, weights_us);
    MoePlan best{true, 128, 1, 1};
    for (int i = 0; i < 4; ++i) {
        if ((long)T * k / kTn[i] + E > 65535) continue;   // (the tiles are a dimension of the grid)
        const double fill = rows / kTn[i], entries = experts * (fill < 0.5 ? 1.0 : fill + 0.5);
        MoePlan pl{false, kTn[i], 1, 1};
        double total = 0.0;
        for (int gated = 0; gated < 2; ++gated) {
            const int kbs = gated ? (D + 127) / 128 : F / 128, columns = gated ? F / 128 : (D + 127) / 128;
            double t_best = 1e300;
            for (int cs = 1; cs <= 8 && cs <= kbs; ++cs) {
                int at_once = 0;
                const cudaError_t e = fp8a8_narrow_at_once(gated, kTn[i], cs, dev, &at_once);
                if (e != cudaSuccess) return e;
                if (at_once < 1) continue;
                const double tiles = entries * columns, waves = tiles < at_once ? 1.0 : tiles / at_once;
                const double t = waves * ((waves > 1.0 ? 6.0 : 2.0) + 0.1 * cs + 0.011 * kTn[i] * (gated ? 2 : 1) +
                                          (kbs + cs - 1) / cs * kNarrowKb[gated][i]);
                if (t < t_best) {
                    t_best = t;
                    (gated ? pl.cs_gate_up : pl.cs_down) = cs;
                }
            }
            total += std::max(t_best, (gated ? 2 : 1) * weights_us);
        }
        if (total < least) {
            least = total;
            best = pl;
        }
    }
    slot = Known{T, D, F, E, k, dev, best};
    *plan = best;
    return cudaSuccess;
}

bool moe_plan_fits(const MoePlan& pl, int T, int D, int F, int E, int k) {
    if (pl.many) return pl.tn == 128;
    bool tile = false;
    for (int tn : kTn) tile |= pl.tn == tn;
    return tile && pl.cs_gate_up >= 1 && pl.cs_gate_up <= 8 && pl.cs_gate_up <= (D + 127) / 128 && pl.cs_down >= 1 && pl.cs_down <= 8 &&
           pl.cs_down <= F / 128 && (long)T * k / pl.tn + E <= 65535;
}

static bool plan_fits(const Fp8a8Plan& pl, int M, int kbs, int cols, bool gated) {
    if (pl.pair) {
        for (int i = 0; i < (gated ? 1 : 3); ++i)
            if (pl.bn == kBn[i]) return true;
        return false;
    }
    bool tile = false;
    for (int tn : kTn) tile |= pl.tn == tn;
    return tile && pl.cs >= 1 && pl.cs <= 8 && pl.cs <= kbs && (cols + 127) / 128 <= 65535 && (M + pl.tn - 1) / pl.tn <= 65535;
}

// Every CTA of a narrow tile's cluster has a K block, the grid is in range, and no tile of
// the first launch reaches into the second's columns, which start at a weight block.
bool fp8a8_plans_fit(const Fp8a8Plans& r, int M, int K, int N, bool gated) {
    const int kbs = (K + 127) / 128;
    if (r.split < 1 || r.split > N || !plan_fits(r.first, M, kbs, r.split, gated)) return false;
    if (r.split == N) return true;
    const int width = r.first.pair && !gated ? r.first.bn : 128;
    return r.split % 128 == 0 && r.split % width == 0 && plan_fits(r.second, M, kbs, N - r.split, gated);
}

}  // namespace qmm
