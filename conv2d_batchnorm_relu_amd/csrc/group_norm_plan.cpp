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
    const int most = (backward ? 24 : 48) / size;   // vectors of x (and dy) a thread holds: 96 registers
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
            while (g.P > 1 && g.P / 2 >= s.pixels) g.P = pow2 ? g.P / 2 : (g.P + 1) / 2;
            g.ipw = (int)std::max<int64_t>(1, std::min<int64_t>(threads / (V * g.P), s.images));
            const int64_t k = up(s.pixels, g.P);
            if (k <= most) {
                g.tiles = 1;
                g.k = (int)k;
            } else {
                g.ipw = 1;
                if (V * g.P < 64 || threads < 512) continue;   // (fewer and larger tiles)
                const int64_t per = std::min<int64_t>(k, most / 2);
                g.tiles = (int)up(s.pixels, g.P * per);
                g.k = (int)up(s.pixels, (int64_t)g.tiles * g.P);
                g.tiles = (int)up(s.pixels, (int64_t)g.P * g.k);
            }
            g.pre = pow2 && V <= 64 && V * g.P % 64 == 0;
            if (lds_floats(g, cpg % 8 || backward ? 8 : 1, backward ? 2 : 1) > 40 * 1024) continue;   // of a CU's 160 KB
            const double wgs = (double)up(s.images, g.ipw) * g.tiles * chunks;
            const int t = g.V * g.P * g.ipw, share = std::max(1, (g.k > most / 2 ? 1024 : 2048) / std::max(t, 64));
            const double bytes = (double)g.ipw * std::min<int64_t>(s.pixels, (int64_t)g.P * g.k) * ng * cpg * size * (backward ? 3 : 2);
            const double width = (double)ng * cpg * size, narrow = width >= 128 ? 1. : width >= 64 ? 1.1 : width >= 32 ? 1.3 : 2.;   // of cache lines
            const double at_once = std::min(wgs, 256. * share), per_cu = std::max(1., at_once / 256.);
            const double rate = std::min(60e3, 5.0e6 / std::min(wgs, 256.));   // bytes a us and CU
            const double rounds = std::max(1., wgs / (256. * share));
            double time = 3. + rounds * (1.5 + per_cu * bytes * narrow / rate) + (g.pre ? 0. : 0.5);
            if (loose) time *= 1.1;
            if (g.tiles > 1) time = 4. + time * (backward ? 1.67 : 1.5);
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
