// group_norm_plan.cpp -- how a group norm call is laid out: groups, pixels and images a workgroup, and
// whether an image is held whole or in tiles.
#include <algorithm>

#include "block_launch.h"
#include "group_norm.h"

namespace cbr {
namespace gnorm {

Geo plan_group_norm(const cbr_group_norm_shape &s, bool backward)
{
    const int cpg = s.channels / s.groups, size = s.type == CBR_F32 ? 4 : 2;
    const int nv = split_of(cpg);
    // pixels a thread holds of images held whole
    const int most = (backward ? bwd_most(nv) : fwd_most(nv)) * 4 / size;
    const int64_t row = (int64_t)s.channels * size, limit = 0x7fffffff / row;   // pixels within 2^31 bytes
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    Geo best{};
    double least = 0;
    // Chunks of 1, 2, 4, ... groups, and of all (a call plans anew: few candidates).  Every chunk has eight
    // channels at least, if there are that many: else one of some groups more.
    auto fits = [&](int ng) {
        const int rest = s.groups % ng;
        return ng == s.groups || (ng * cpg >= 8 && (rest == 0 || rest * cpg >= 8));
    };
    for (int64_t want = 1;; want *= 2) {
        int ng = (int)std::min<int64_t>(want, s.groups);
        while (!fits(ng) && ng < 2 * want - 1) ++ng;
        const int V = (int)up((int64_t)ng * cpg, 8), chunks = (int)up(s.groups, ng);
        if (V > 1024 || (least > 0 && (int64_t)ng * cpg * size > 1024 && s.pixels > 8)) break;
        if (!fits(ng)) continue;
        const bool all = ng == s.groups, loose = cpg % 8 && ((int64_t)ng * cpg % 8 || s.channels % 8);
        const bool pow2 = (V & (V - 1)) == 0;
        for (int threads = 64; threads <= 1024; threads *= 2) {
            if (threads < V && threads < 1024) continue;
            Geo g{};
            g.V = V;
            g.ng = ng;
            g.chunks = chunks;
            g.P = std::max(1, threads / V);
            while (g.P > 1 && (g.P / 2 >= s.pixels || g.P > limit)) g.P = pow2 ? g.P / 2 : (g.P + 1) / 2;
            g.ipw = (int)std::max<int64_t>(1, std::min<int64_t>({threads / (V * g.P), s.images, limit / s.pixels}));
            const int64_t k = up(s.pixels, g.P);
            if (k <= most && g.ipw * s.pixels <= limit) {
                g.tiles = 1;
                g.k = (int)k;
            } else {
                // tiles for two workgroups a CU, of 64 pixels a thread at most
                g.ipw = 1;
                if (V * g.P < 64 || threads < 512) continue;
                const int64_t per = std::min(std::min<int64_t>(k, 64), std::max<int64_t>(1, limit / g.P));
                const int64_t tiles = std::max<int64_t>({2, up(s.pixels, g.P * per), std::min<int64_t>(k, up(512, s.images * chunks))});
                g.k = (int)up(s.pixels, tiles * g.P);
                g.tiles = (int)up(s.pixels, (int64_t)g.P * g.k);
                if (g.tiles < 2) continue;
            }
            g.pre = pow2 && V <= 64 && V * g.P % 64 == 0;
            if ((backward ? bwd_floats(g, cpg) : sum_floats(g, nv, 1)) > 40 * 1024) continue;   // floats: a CU's 160 KB
            // Expected time in us, fitted to measurements: 5 TB/s over all CUs and 60 GB/s for one; runs of a pixel's
            // channels shorter than 64 bytes cost; a workgroup that has its CU to itself (by its registers) loads, sums
            // and stores one after the other; SiLU's gradient is half as much arithmetic as loads and stores.
            const int t = V * g.P * g.ipw, f = 4 / size;
            const int waves = backward ? (g.k <= f ? 24 : g.k <= 2 * f ? 20 : 16) : g.k <= 2 * f ? 32 : g.k <= 4 * f ? 24 : 16;
            const int share = std::max(1, waves * 64 / std::max(t, 64));
            const double wgs = (double)up(s.images, g.ipw) * g.tiles * chunks, at_once = std::min(wgs, 256. * share);
            const double width = (double)ng * cpg * size, narrow = width >= 64 ? 1. : width >= 32 ? 1.2 : 1.6;
            const double values = (double)g.ipw * std::min<int64_t>(s.pixels, (int64_t)g.P * g.k) * ng * cpg;
            const double per_cu = std::max(1., at_once / 256.), rate = std::min(60e3, 5.0e6 / std::min(wgs, 256.));
            double one = per_cu * values * size * (backward ? 3 : 2) * narrow / rate;
            if (g.tiles > 1) {
                one *= backward ? 5. / 3. : 1.5;
            } else {
                if (share == 1) one *= 1.3;
                one += per_cu * values * (s.act == CBR_ACT_SILU ? (backward ? 0.35 : 0.1) : 0.05) / 4000.;
            }
            double time = (g.tiles > 1 ? 9. : 4.) + std::max(1., wgs / (256. * share)) * (1. + one) + (g.pre ? 0. : 1.);
            if (loose) time *= 1.1;
            if (least == 0 || time < least) {
                least = time;
                best = g;
            }
        }
        if (all) break;
    }
    return best;
}

}  // namespace gnorm
}  // namespace cbr
